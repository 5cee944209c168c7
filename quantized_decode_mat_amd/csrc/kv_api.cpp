// kv_api.cpp — the C ABI of the paged cache: attention, rotary positions,
// pages (include/xq.h). Gates in the order of xq_api.cpp: null pointers,
// shapes, alignment, then the device; nothing is launched after a refusal.
#include <cmath>

#include "kv_launch.h"
#include "xq_host.h"

using namespace xq::host;

namespace {

constexpr int64_t kMaxInt = 2147483647LL;
constexpr int64_t kMaxLen = 1LL << 30;
// Workgroups of 256 threads: a launch counts its threads in 32 bits, and more
// wrap round without an error.
constexpr int64_t kMaxBlocks = (1LL << 24) - 1;

int type_bytes(int32_t t) { return t == XQ_F32 ? 4 : t == XQ_E4M3 ? 1 : 2; }
bool row_type(int32_t t) { return t == XQ_F32 || t == XQ_BF16 || t == XQ_F16; }

// The struct itself; its alignment is kv_align's.
xq_status check_kv(const xq_kv* kv, bool one_layer) {
  if (!kv) return fail(XQ_E_NULL, "kv is NULL");
  if (!kv->k) return fail(XQ_E_NULL, "kv k is NULL");
  if (!kv->v) return fail(XQ_E_NULL, "kv v is NULL");
  if (kv->dtype != XQ_BF16 && kv->dtype != XQ_F16 && kv->dtype != XQ_E4M3)
    return fail(XQ_E_SHAPE, "kv dtype=%d is none of XQ_BF16, XQ_F16, XQ_E4M3", kv->dtype);
  // (layer, k or v, 1 of 64 parts) of a page is an int32 in the page moves.
  if (kv->layers < 1 || kv->layers > (1 << 24))
    return fail(XQ_E_SHAPE, "kv layers=%lld outside 1..2^24", (long long)kv->layers);
  if (one_layer && kv->layers != 1)
    return fail(XQ_E_SHAPE, "kv layers=%lld; this call takes one layer", (long long)kv->layers);
  if (kv->pages < 1 || kv->page < 1 || kv->pages > kMaxInt / kv->page)
    return fail(XQ_E_SHAPE, "kv pages=%lld of page=%lld tokens outside 1..2^31-1 tokens",
                (long long)kv->pages, (long long)kv->page);
  if (kv->kv_heads < 1 || kv->kv_heads > (1 << 20))
    return fail(XQ_E_SHAPE, "kv kv_heads=%lld outside 1..2^20", (long long)kv->kv_heads);
  if (kv->dim < 16 || kv->dim > 256 || kv->dim % 16)
    return fail(XQ_E_SHAPE, "kv dim=%lld not a multiple of 16 in 16..256", (long long)kv->dim);
  if (!(kv->k_scale > 0.f) || !(kv->v_scale > 0.f) || !std::isfinite(kv->k_scale) ||
      !std::isfinite(kv->v_scale))
    return fail(XQ_E_SHAPE, "kv scales %g, %g not finite and above 0", kv->k_scale, kv->v_scale);
  for (int i = 0; i < 4; ++i)
    if (kv->k_stride[i] < 0 || kv->v_stride[i] < 0)
      return fail(XQ_E_SHAPE, "kv stride %d is negative", i);
  return XQ_OK;
}

xq_status align_kv(const xq_kv* kv) {
  if (!aligned(kv->k, 16)) return fail(XQ_E_ALIGN, "kv k not 16-byte aligned");
  if (!aligned(kv->v, 16)) return fail(XQ_E_ALIGN, "kv v not 16-byte aligned");
  for (int i = 0; i < 4; ++i)
    if (kv->k_stride[i] * type_bytes(kv->dtype) % 16 || kv->v_stride[i] * type_bytes(kv->dtype) % 16)
      return fail(XQ_E_ALIGN, "kv stride %d not a multiple of 16 bytes", i);
  return XQ_OK;
}

xq_status check_tables(int64_t rows, int64_t width, int64_t stride) {
  if (width < 1 || width > kMaxInt)
    return fail(XQ_E_SHAPE, "table width=%lld outside 1..2^31-1", (long long)width);
  if (stride < (rows > 1 ? width : 0) || stride > (1LL << 40))
    return fail(XQ_E_SHAPE, "table stride=%lld below its width=%lld", (long long)stride,
                (long long)width);
  return XQ_OK;
}

// A tensor of rows for 16-byte accesses.
xq_status align_rows(const void* p, int64_t row, int64_t head, int32_t type, const char* what) {
  if (!aligned(p, 16)) return fail(XQ_E_ALIGN, "%s not 16-byte aligned", what);
  if (row * type_bytes(type) % 16 || head * type_bytes(type) % 16)
    return fail(XQ_E_ALIGN, "%s strides not multiples of 16 bytes", what);
  return XQ_OK;
}

xq_status check_attention(int64_t heads, const xq_kv* kv, float scale, int64_t window,
                          int64_t sinks) {
  if (heads < 1 || heads % kv->kv_heads)
    return fail(XQ_E_SHAPE, "heads=%lld not a multiple of kv_heads=%lld", (long long)heads,
                (long long)kv->kv_heads);
  if (heads / kv->kv_heads > 256)
    return fail(XQ_E_SHAPE, "heads/kv_heads=%lld above 256", (long long)(heads / kv->kv_heads));
  if (!std::isfinite(scale)) return fail(XQ_E_SHAPE, "scale=%g not finite", scale);
  // The kernels' exponents are of 2.
  if (!std::isfinite(scale * kv->k_scale * 1.44269504f))
    return fail(XQ_E_SHAPE, "scale=%g times k_scale=%g above f32's range", scale, kv->k_scale);
  for (const int64_t* st : {kv->k_stride, kv->v_stride}) {
    // The kernels find a token by its place within a head, in 16-byte units.
    const double last = static_cast<double>(kv->pages - 1) * static_cast<double>(st[1]) +
                        static_cast<double>(kv->page - 1) * static_cast<double>(st[3]);
    if (last * type_bytes(kv->dtype) >= 68719476736.0)
      return fail(XQ_E_SHAPE, "kv pages of one layer reach over 64 GiB");
  }
  if (window < 0 || window > kMaxLen)
    return fail(XQ_E_SHAPE, "window=%lld outside 0..2^30", (long long)window);
  if (sinks < 0 || sinks > kMaxLen)
    return fail(XQ_E_SHAPE, "sinks=%lld outside 0..2^30", (long long)sinks);
  return XQ_OK;
}

xq_status check_strides(int64_t row, int64_t head, const char* what) {
  if (row < 0 || head < 0) return fail(XQ_E_SHAPE, "%s has a negative stride", what);
  return XQ_OK;
}

xq_status check_decode(int64_t seqs, int64_t heads, const xq_kv* kv, float scale, int64_t window,
                       int64_t sinks, int64_t max_len) {
  if (xq_status s = check_kv(kv, true)) return s;
  if (xq_status s = check_attention(heads, kv, scale, window, sinks)) return s;
  if (seqs < 1 || seqs > (1 << 20) / kv->kv_heads)
    return fail(XQ_E_SHAPE, "seqs*kv_heads = %lld*%lld outside 1..2^20", (long long)seqs,
                (long long)kv->kv_heads);
  if (max_len < 1 || max_len > kMaxLen)
    return fail(XQ_E_SHAPE, "max_len=%lld outside 1..2^30", (long long)max_len);
  if (xq::attn_decode_units(seqs, heads, *kv) > kMaxBlocks)
    return fail(XQ_E_SHAPE, "seqs and heads give too many workgroups for one launch");
  return XQ_OK;
}

}  // namespace

extern "C" {

xq_status xq_attn_decode(void *out, const void *q, int32_t io, int64_t seqs, int64_t heads,
                         int64_t out_row, int64_t out_head, int64_t q_row, int64_t q_head,
                         const xq_kv *kv, const int32_t *tables, int64_t table_width,
                         int64_t table_stride, const int32_t *lens, float scale, int64_t window,
                         int64_t sinks, int64_t max_len, void *workspace, size_t workspace_bytes,
                         void *stream) {
  if (!out) return fail(XQ_E_NULL, "out is NULL");
  if (!q) return fail(XQ_E_NULL, "q is NULL");
  if (!tables) return fail(XQ_E_NULL, "tables is NULL");
  if (!lens) return fail(XQ_E_NULL, "lens is NULL");
  if (!row_type(io)) return fail(XQ_E_SHAPE, "io=%d is none of XQ_F32, XQ_BF16, XQ_F16", io);
  if (xq_status s = check_decode(seqs, heads, kv, scale, window, sinks, max_len)) return s;
  if (xq_status s = check_strides(out_row, out_head, "out")) return s;
  if (xq_status s = check_strides(q_row, q_head, "q")) return s;
  if (xq_status s = check_tables(seqs, table_width, table_stride)) return s;
  const size_t need = xq::attn_decode_workspace_bytes(seqs, heads, *kv, max_len, window, sinks);
  if (xq_status s = check_workspace(workspace, workspace_bytes, need,
                                    "xq_attn_decode_workspace_bytes"))
    return s;
  if (xq_status s = align_rows(out, out_row, out_head, io, "out")) return s;
  if (xq_status s = align_rows(q, q_row, q_head, io, "q")) return s;
  if (xq_status s = align_kv(kv)) return s;
  if (!aligned(tables, 4)) return fail(XQ_E_ALIGN, "tables not 4-byte aligned");
  if (!aligned(lens, 4)) return fail(XQ_E_ALIGN, "lens not 4-byte aligned");
  if (xq_status s = check_workspace_align(workspace, need)) return s;
  if (xq_status s = check_device()) return s;
  return launched(xq::launch_attn_decode(xq::RowsView{out, io, out_row, out_head},
                                         xq::RowsView{const_cast<void*>(q), io, q_row, q_head},
                                         seqs, heads, *kv,
                                         xq::TableView{tables, table_width, table_stride}, lens,
                                         scale, window, sinks, max_len, workspace,
                                         static_cast<hipStream_t>(stream)),
                  "xq_attn_decode");
}

size_t xq_attn_decode_workspace_bytes(int64_t seqs, int64_t heads, const xq_kv *kv,
                                      int64_t max_len, int64_t window, int64_t sinks) {
  if (check_decode(seqs, heads, kv, 1.f, window, sinks, max_len)) return 0;
  return xq::attn_decode_workspace_bytes(seqs, heads, *kv, max_len, window, sinks);
}

xq_status xq_attn_prefill(void *out, const void *q, int32_t io, int64_t rows, int64_t seqs,
                          int64_t heads, int64_t out_row, int64_t out_head, int64_t q_row,
                          int64_t q_head, const xq_kv *kv, const int32_t *tables,
                          int64_t table_width, int64_t table_stride, const int32_t *lens,
                          const int32_t *starts, int64_t max_chunk, float scale, int64_t window,
                          int64_t sinks, void *stream) {
  if (!out) return fail(XQ_E_NULL, "out is NULL");
  if (!q) return fail(XQ_E_NULL, "q is NULL");
  if (!tables) return fail(XQ_E_NULL, "tables is NULL");
  if (!lens) return fail(XQ_E_NULL, "lens is NULL");
  if (!starts) return fail(XQ_E_NULL, "starts is NULL");
  if (io != XQ_BF16 && io != XQ_F16)
    return fail(XQ_E_SHAPE, "io=%d is neither XQ_BF16 nor XQ_F16", io);
  if (xq_status s = check_kv(kv, true)) return s;
  if (kv->dtype != io && kv->dtype != XQ_E4M3)
    return fail(XQ_E_SHAPE, "kv dtype=%d is neither io=%d nor XQ_E4M3", kv->dtype, io);
  if (xq_status s = check_attention(heads, kv, scale, window, sinks)) return s;
  if (rows < 1 || rows > kMaxInt / heads)
    return fail(XQ_E_SHAPE, "rows*heads = %lld*%lld outside 1..2^31-1", (long long)rows,
                (long long)heads);
  if (seqs < 1 || seqs > (1 << 16))
    return fail(XQ_E_SHAPE, "seqs=%lld outside 1..2^16", (long long)seqs);
  if (max_chunk < 1 || max_chunk > rows)
    return fail(XQ_E_SHAPE, "max_chunk=%lld outside 1..rows=%lld", (long long)max_chunk,
                (long long)rows);
  if (xq::attn_prefill_blocks(seqs, heads, *kv, max_chunk) > kMaxBlocks)
    return fail(XQ_E_SHAPE, "seqs, heads and max_chunk give too many workgroups for one launch");
  if (xq_status s = check_strides(out_row, out_head, "out")) return s;
  if (xq_status s = check_strides(q_row, q_head, "q")) return s;
  if (xq_status s = check_tables(seqs, table_width, table_stride)) return s;
  if (xq_status s = align_rows(out, out_row, out_head, io, "out")) return s;
  if (xq_status s = align_rows(q, q_row, q_head, io, "q")) return s;
  if (xq_status s = align_kv(kv)) return s;
  if (!aligned(tables, 4)) return fail(XQ_E_ALIGN, "tables not 4-byte aligned");
  if (!aligned(lens, 4)) return fail(XQ_E_ALIGN, "lens not 4-byte aligned");
  if (!aligned(starts, 4)) return fail(XQ_E_ALIGN, "starts not 4-byte aligned");
  if (xq_status s = check_device()) return s;
  return launched(xq::launch_attn_prefill(xq::RowsView{out, io, out_row, out_head},
                                          xq::RowsView{const_cast<void*>(q), io, q_row, q_head},
                                          rows, seqs, heads, *kv,
                                          xq::TableView{tables, table_width, table_stride}, lens,
                                          starts, max_chunk, scale, window, sinks,
                                          static_cast<hipStream_t>(stream)),
                  "xq_attn_prefill");
}

static xq_status check_rope(const xq_rope_freqs* rope, int64_t tokens, int64_t heads, int64_t dim,
                            int64_t pos_stride) {
  if (dim < 8 || dim > 1024 || dim % 8)
    return fail(XQ_E_SHAPE, "dim=%lld not a multiple of 8 in 8..1024", (long long)dim);
  if (rope->rot < 8 || rope->rot > dim || rope->rot % 8)
    return fail(XQ_E_SHAPE, "rope rot=%lld not a multiple of 8 in 8..dim", (long long)rope->rot);
  if (rope->axes < 1 || rope->axes > 4)
    return fail(XQ_E_SHAPE, "rope axes=%lld outside 1..4", (long long)rope->axes);
  if (rope->adjacent != 0 && rope->adjacent != 1)
    return fail(XQ_E_SHAPE, "rope adjacent=%lld is neither 0 nor 1", (long long)rope->adjacent);
  int64_t pairs = 0;
  for (int i = 0; i < rope->axes; ++i) {
    if (rope->sections[i] < 0 || rope->sections[i] > rope->rot / 2)
      return fail(XQ_E_SHAPE, "rope sections[%d]=%lld outside 0..rot/2", i,
                  (long long)rope->sections[i]);
    pairs += rope->sections[i];
  }
  if (pairs != rope->rot / 2)
    return fail(XQ_E_SHAPE, "rope sections sum to %lld, not rot/2=%lld", (long long)pairs,
                (long long)(rope->rot / 2));
  if (tokens < 1 || heads < 1 || tokens > kMaxInt / heads)
    return fail(XQ_E_SHAPE, "tokens*heads = %lld*%lld outside 1..2^31-1", (long long)tokens,
                (long long)heads);
  if (pos_stride < 0) return fail(XQ_E_SHAPE, "pos has a negative stride");
  return XQ_OK;
}

static xq_status align_elems(const void* p, int32_t type, const char* what) {
  if (!aligned(p, type_bytes(type)))
    return fail(XQ_E_ALIGN, "%s not aligned to its elements", what);
  return XQ_OK;
}

xq_status xq_rope(void *out, int32_t out_type, int64_t out_row, int64_t out_head, const void *x,
                  int32_t x_type, int64_t x_row, int64_t x_head, int64_t tokens, int64_t heads,
                  int64_t dim, const int32_t *pos, int64_t pos_stride, const xq_rope_freqs *rope,
                  int32_t inverse, void *stream) {
  if (!out) return fail(XQ_E_NULL, "out is NULL");
  if (!x) return fail(XQ_E_NULL, "x is NULL");
  if (!pos) return fail(XQ_E_NULL, "pos is NULL");
  if (!rope) return fail(XQ_E_NULL, "rope is NULL");
  if (!rope->freq) return fail(XQ_E_NULL, "rope freq is NULL");
  if (!row_type(out_type))
    return fail(XQ_E_SHAPE, "out_type=%d is none of XQ_F32, XQ_BF16, XQ_F16", out_type);
  if (!row_type(x_type))
    return fail(XQ_E_SHAPE, "x_type=%d is none of XQ_F32, XQ_BF16, XQ_F16", x_type);
  if (inverse != 0 && inverse != 1)
    return fail(XQ_E_SHAPE, "inverse=%d is neither 0 nor 1", inverse);
  if (xq_status s = check_rope(rope, tokens, heads, dim, pos_stride)) return s;
  if (xq_status s = check_strides(out_row, out_head, "out")) return s;
  if (xq_status s = check_strides(x_row, x_head, "x")) return s;
  if (xq_status s = align_elems(out, out_type, "out")) return s;
  if (xq_status s = align_elems(x, x_type, "x")) return s;
  if (!aligned(pos, 4)) return fail(XQ_E_ALIGN, "pos not 4-byte aligned");
  if (!aligned(rope->freq, 8)) return fail(XQ_E_ALIGN, "rope freq not 8-byte aligned");
  if (xq_status s = check_device()) return s;
  return launched(xq::launch_rope(xq::RowsView{out, out_type, out_row, out_head},
                                  xq::RowsView{const_cast<void*>(x), x_type, x_row, x_head},
                                  nullptr, nullptr, tokens, heads, dim, nullptr, pos, pos_stride,
                                  *rope, inverse != 0, nullptr, static_cast<hipStream_t>(stream)),
                  "xq_rope");
}

xq_status xq_rope_append(void *q_out, int32_t out_type, int64_t out_row, int64_t out_head,
                         const xq_kv *kv, const void *q, int64_t q_row, int64_t q_head,
                         const void *k, int64_t k_row, int64_t k_head, const void *v,
                         int64_t v_row, int64_t v_head, int32_t x_type, int64_t tokens,
                         int64_t heads, const int32_t *pos, int64_t pos_stride,
                         const xq_rope_freqs *rope, const int64_t *slots, void *stream) {
  if (!q_out) return fail(XQ_E_NULL, "q_out is NULL");
  if (!q) return fail(XQ_E_NULL, "q is NULL");
  if (!k) return fail(XQ_E_NULL, "k is NULL");
  if (!v) return fail(XQ_E_NULL, "v is NULL");
  if (!pos) return fail(XQ_E_NULL, "pos is NULL");
  if (!rope) return fail(XQ_E_NULL, "rope is NULL");
  if (!rope->freq) return fail(XQ_E_NULL, "rope freq is NULL");
  if (!slots) return fail(XQ_E_NULL, "slots is NULL");
  if (!row_type(out_type))
    return fail(XQ_E_SHAPE, "out_type=%d is none of XQ_F32, XQ_BF16, XQ_F16", out_type);
  if (!row_type(x_type))
    return fail(XQ_E_SHAPE, "x_type=%d is none of XQ_F32, XQ_BF16, XQ_F16", x_type);
  if (xq_status s = check_kv(kv, true)) return s;
  if (heads < 1 || heads > kMaxInt - 2 * kv->kv_heads)
    return fail(XQ_E_SHAPE, "heads=%lld outside 1..2^31-1", (long long)heads);
  if (xq_status s = check_rope(rope, tokens, heads + 2 * kv->kv_heads, kv->dim, pos_stride)) return s;
  if (xq_status s = check_strides(out_row, out_head, "q_out")) return s;
  if (xq_status s = check_strides(q_row, q_head, "q")) return s;
  if (xq_status s = check_strides(k_row, k_head, "k")) return s;
  if (xq_status s = check_strides(v_row, v_head, "v")) return s;
  if (xq_status s = align_elems(q_out, out_type, "q_out")) return s;
  if (xq_status s = align_elems(q, x_type, "q")) return s;
  if (xq_status s = align_elems(k, x_type, "k")) return s;
  if (xq_status s = align_elems(v, x_type, "v")) return s;
  if (xq_status s = align_kv(kv)) return s;
  if (!aligned(pos, 4)) return fail(XQ_E_ALIGN, "pos not 4-byte aligned");
  if (!aligned(rope->freq, 8)) return fail(XQ_E_ALIGN, "rope freq not 8-byte aligned");
  if (!aligned(slots, 8)) return fail(XQ_E_ALIGN, "slots not 8-byte aligned");
  if (xq_status s = check_device()) return s;
  const xq::RowsView kr{const_cast<void*>(k), x_type, k_row, k_head};
  const xq::RowsView vr{const_cast<void*>(v), x_type, v_row, v_head};
  return launched(xq::launch_rope(xq::RowsView{q_out, out_type, out_row, out_head},
                                  xq::RowsView{const_cast<void*>(q), x_type, q_row, q_head}, &kr,
                                  &vr, tokens, heads, kv->dim, kv, pos, pos_stride, *rope, false,
                                  slots, static_cast<hipStream_t>(stream)),
                  "xq_rope_append");
}

xq_status xq_cache_copy(const xq_kv *kv, const int32_t *src, const int32_t *dst, int64_t n,
                        void *stream) {
  if (!src && n != 0) return fail(XQ_E_NULL, "src is NULL");
  if (!dst && n != 0) return fail(XQ_E_NULL, "dst is NULL");
  if (xq_status s = check_kv(kv, false)) return s;
  if (n < 0 || n > kMaxInt) return fail(XQ_E_SHAPE, "n=%lld outside 0..2^31-1", (long long)n);
  if (xq_status s = align_kv(kv)) return s;
  if (!aligned(src, 4)) return fail(XQ_E_ALIGN, "src not 4-byte aligned");
  if (!aligned(dst, 4)) return fail(XQ_E_ALIGN, "dst not 4-byte aligned");
  if (n == 0) return ok();
  if (xq_status s = check_device()) return s;
  return launched(xq::launch_cache_copy(*kv, src, dst, n, static_cast<hipStream_t>(stream)),
                  "xq_cache_copy");
}

static xq_status check_cache(const xq_kv* kv, const int32_t* refs, const int32_t* tables,
                             int64_t slots, int64_t width, int64_t stride) {
  if (!refs) return fail(XQ_E_NULL, "refs is NULL");
  if (!tables) return fail(XQ_E_NULL, "tables is NULL");
  if (xq_status s = check_kv(kv, false)) return s;
  if (slots < 1 || slots > (1 << 20))
    return fail(XQ_E_SHAPE, "slots=%lld outside 1..2^20", (long long)slots);
  return check_tables(slots, width, stride);
}

static xq_status align_cache(const xq_kv* kv, const int32_t* refs, const int32_t* tables) {
  if (xq_status s = align_kv(kv)) return s;
  if (!aligned(refs, 4)) return fail(XQ_E_ALIGN, "refs not 4-byte aligned");
  if (!aligned(tables, 4)) return fail(XQ_E_ALIGN, "tables not 4-byte aligned");
  return XQ_OK;
}

xq_status xq_cache_free(const xq_kv *kv, int32_t *refs, int32_t *tables, int64_t slots,
                        int64_t width, int64_t stride, int32_t *lens, const int32_t *rows,
                        int64_t n, void *stream) {
  if (!lens) return fail(XQ_E_NULL, "lens is NULL");
  if (!rows && n != 0) return fail(XQ_E_NULL, "rows is NULL");
  if (xq_status s = check_cache(kv, refs, tables, slots, width, stride)) return s;
  if (n < 0 || n > (1 << 20)) return fail(XQ_E_SHAPE, "n=%lld outside 0..2^20", (long long)n);
  if (xq_status s = align_cache(kv, refs, tables)) return s;
  if (!aligned(lens, 4)) return fail(XQ_E_ALIGN, "lens not 4-byte aligned");
  if (!aligned(rows, 4)) return fail(XQ_E_ALIGN, "rows not 4-byte aligned");
  if (n == 0) return ok();
  if (xq_status s = check_device()) return s;
  return launched(xq::launch_cache_free(*kv, refs, tables, slots, width, stride, lens, rows, n,
                                        static_cast<hipStream_t>(stream)),
                  "xq_cache_free");
}

xq_status xq_cache_fork(const xq_kv *kv, int32_t *refs, int32_t *tables, int64_t slots,
                        int64_t width, int64_t stride, int32_t *lens, const int32_t *parents,
                        const int32_t *children, int64_t n, int32_t *status, void *workspace,
                        size_t workspace_bytes, void *stream) {
  if (!lens) return fail(XQ_E_NULL, "lens is NULL");
  if (!parents && n != 0) return fail(XQ_E_NULL, "parents is NULL");
  if (!children && n != 0) return fail(XQ_E_NULL, "children is NULL");
  if (!status) return fail(XQ_E_NULL, "status is NULL");
  if (xq_status s = check_cache(kv, refs, tables, slots, width, stride)) return s;
  if (n < 0 || n > slots)
    return fail(XQ_E_SHAPE, "n=%lld outside 0..slots=%lld", (long long)n, (long long)slots);
  const size_t need = xq::cache_workspace_bytes(kv->pages, slots);
  if (xq_status s = check_workspace(workspace, workspace_bytes, need, "xq_cache_workspace_bytes"))
    return s;
  if (xq_status s = align_cache(kv, refs, tables)) return s;
  if (!aligned(lens, 4)) return fail(XQ_E_ALIGN, "lens not 4-byte aligned");
  if (!aligned(parents, 4)) return fail(XQ_E_ALIGN, "parents not 4-byte aligned");
  if (!aligned(children, 4)) return fail(XQ_E_ALIGN, "children not 4-byte aligned");
  if (!aligned(status, 4)) return fail(XQ_E_ALIGN, "status not 4-byte aligned");
  if (xq_status s = check_workspace_align(workspace, need)) return s;
  if (xq_status s = check_device()) return s;
  return launched(xq::launch_cache_fork(*kv, refs, tables, slots, width, stride, lens, parents,
                                        children, n, status, workspace,
                                        static_cast<hipStream_t>(stream)),
                  "xq_cache_fork");
}

xq_status xq_cache_compact(const xq_kv *kv, int32_t *refs, int32_t *tables, int64_t slots,
                           int64_t width, int64_t stride, int32_t *status, void *workspace,
                           size_t workspace_bytes, void *stream) {
  if (!status) return fail(XQ_E_NULL, "status is NULL");
  if (xq_status s = check_cache(kv, refs, tables, slots, width, stride)) return s;
  const size_t need = xq::cache_workspace_bytes(kv->pages, slots);
  if (xq_status s = check_workspace(workspace, workspace_bytes, need, "xq_cache_workspace_bytes"))
    return s;
  if (xq_status s = align_cache(kv, refs, tables)) return s;
  if (!aligned(status, 4)) return fail(XQ_E_ALIGN, "status not 4-byte aligned");
  if (xq_status s = check_workspace_align(workspace, need)) return s;
  if (xq_status s = check_device()) return s;
  return launched(xq::launch_cache_compact(*kv, refs, tables, slots, width, stride, status,
                                           workspace, static_cast<hipStream_t>(stream)),
                  "xq_cache_compact");
}

size_t xq_cache_workspace_bytes(int64_t pages, int64_t slots) {
  if (pages < 1 || pages > kMaxInt || slots < 1 || slots > (1 << 20)) return 0;
  return xq::cache_workspace_bytes(pages, slots);
}

}  // extern "C"
