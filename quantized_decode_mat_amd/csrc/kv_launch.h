// kv_launch.h — internal launchers of the paged cache's kernels, called by the
// C ABI (kv_api.cpp) after it has validated every argument.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/xq.h"

namespace xq {

// Rows [n][heads][dim] of one type; strides in elements.
struct RowsView {
  void* data;
  int type;
  int64_t row, head;
};
// What n elements of a cache's type take (two of XQ_E2M1 share a byte), and a
// row's exponents there: a byte for 32 dims, in rows of 4 or 8.
inline int64_t cache_bytes(int64_t n, int32_t dtype) {
  return dtype == XQ_E2M1 ? n / 2 : dtype == XQ_E4M3 ? n : 2 * n;
}
inline int64_t exp_row_bytes(int64_t dim) { return dim <= 128 ? 4 : 8; }

struct TableView {
  const int32_t* data;
  int64_t width, stride;
};

// (Sequence, kv head, 16 of its heads) units, each at most a workgroup.
int64_t attn_decode_units(int64_t seqs, int64_t heads, const xq_kv& kv);
size_t attn_decode_workspace_bytes(int64_t seqs, int64_t heads, const xq_kv& kv, int64_t max_len,
                                   int64_t window, int64_t sinks);
hipError_t launch_attn_decode(const RowsView& out, const RowsView& q, int64_t seqs, int64_t heads,
                              const xq_kv& kv, const TableView& tables, const int32_t* lens,
                              float scale, int64_t window, int64_t sinks, int64_t max_len, void* ws,
                              hipStream_t stream);
int64_t attn_prefill_blocks(int64_t seqs, int64_t heads, const xq_kv& kv, int64_t max_chunk);
hipError_t launch_attn_prefill(const RowsView& out, const RowsView& q, int64_t rows, int64_t seqs,
                               int64_t heads, const xq_kv& kv, const TableView& tables,
                               const int32_t* lens, const int32_t* starts, int64_t max_chunk,
                               float scale, int64_t window, int64_t sinks, hipStream_t stream);
// Short chunks, whose (token, head) rows fill at most two workgroups of 16 a CU,
// run on the single-token kernel's form for rows (launch_attn_chunk).
bool chunk_in_rows(int64_t seqs, int64_t heads, const xq_kv& kv, int64_t max_chunk);
hipError_t launch_attn_chunk(const RowsView& out, const RowsView& q, int64_t rows, int64_t seqs,
                             int64_t heads, const xq_kv& kv, const TableView& tables,
                             const int32_t* lens, const int32_t* starts, int64_t max_chunk,
                             float scale, int64_t window, int64_t sinks, hipStream_t stream);
// kv (with k, v and slots) may be null: then only q is rotated.
hipError_t launch_rope(const RowsView& out, const RowsView& q, const RowsView* k, const RowsView* v,
                       int64_t tokens, int64_t heads, int64_t dim, const xq_kv* kv,
                       const int32_t* pos, int64_t pos_stride, const xq_rope_freqs& rope,
                       bool inverse, const int64_t* slots, hipStream_t stream);
hipError_t launch_cache_read(const RowsView& k_out, const RowsView& v_out, const xq_kv& kv,
                             const int64_t* slots, int64_t tokens, hipStream_t stream);
hipError_t launch_cache_copy(const xq_kv& kv, const int32_t* src, const int32_t* dst, int64_t n,
                             hipStream_t stream);
hipError_t launch_cache_free(const xq_kv& kv, int32_t* refs, int32_t* tables, int64_t slots,
                             int64_t width, int64_t stride, int32_t* lens, const int32_t* rows,
                             int64_t n, hipStream_t stream);
hipError_t launch_cache_fork(const xq_kv& kv, int32_t* refs, int32_t* tables, int64_t slots,
                             int64_t width, int64_t stride, int32_t* lens, const int32_t* parents,
                             const int32_t* children, int64_t n, int32_t* status, void* ws,
                             hipStream_t stream);
hipError_t launch_cache_compact(const xq_kv& kv, int32_t* refs, int32_t* tables, int64_t slots,
                                int64_t width, int64_t stride, int32_t* status, void* ws,
                                hipStream_t stream);
size_t cache_workspace_bytes(int64_t pages, int64_t slots);

}  // namespace xq
