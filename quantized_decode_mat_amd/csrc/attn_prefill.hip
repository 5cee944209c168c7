// attn_prefill.hip — attention of chunks of new tokens over a paged cache.
//
//   out_i = sum_j exp(s_ij - m_i) v_scale v_j / sum_j exp(s_ij - m_i),
//   s_ij = scale * k_scale * (q_i . k_j), over the tokens j that row i sees:
//   j <= p_i, and with a window j > p_i - window or j < sinks.
//
// What bounds it: the matrix instructions, 4 * dim operations per visible
// (row, token) pair, and beside them the exponentials. Rows are (token, head)
// pairs of one kv head, the heads of a token next to each other: a workgroup
// takes 128 rows (32 per wave) and walks over the tokens that any of them
// sees, 64 at a time, so a kv head's keys and values are read once for all its
// heads, and short chunks still fill their tiles. K and V of the next tile are
// fetched into registers while the present one is worked on out of LDS, and
// put into the other half of a double buffer after it: one barrier per tile.
//  - S^T = K Q^T (32x32x16): lane l holds row l % 32 and 16 tokens of each 32,
//    so a row's maximum and sum are local to the lane but for one exchange
//    between the wave's halves.
//  - O^T = V^T P^T: P goes from S^T's registers straight into the instruction;
//    its V operand comes from LDS by transposing loads (4 tokens of one dim
//    per lane), in the same order of the summed index. O^T's column is again
//    row l % 32: rescaling is local to the lane.
// LDS rows are padded by 16 bytes, so 8 rows of a 16-byte column hit 32
// different banks.
//
// Precision: S, the softmax and O are f32; q enters in its own 16 bits, an
// 8-bit cache is widened exactly; p is rounded to 16 bits, as the product
// needs.
#include <algorithm>

#include "kv_device.h"
#include "kv_launch.h"

namespace xq {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kRows = 32 * kWaves;  // rows of a workgroup
constexpr int kTile = 64;           // tokens of a step
constexpr float kLog2e = 1.44269504088896340736f;

struct PrefillArgs {
  KvView kv;
  const uint8_t* q;
  uint8_t* out;
  const int32_t* tables;
  const int32_t* lens;
  const int32_t* starts;
  int64_t q_row, q_head, out_row, out_head;  // bytes
  int64_t table_stride, table_tokens;
  FastDiv group;
  int rows, seqs, kv_heads, dim, max_chunk, window, sinks, tiles;
  float c, v_scale;
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
// Four tokens of one dim: lanes 4r .. 4r+3 of each 16 point at token r's 16
// dims, and lane i receives dim i of the four.
__device__ __forceinline__ u32x2 load_transposed(const uint8_t* p) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_bit_cast(
      u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                 (lds_s16x4*)(__attribute__((address_space(3))) uint8_t*)(p)));
}

// Each lane's value and that of the lane 32 away, the lower lane's first.
__device__ __forceinline__ f32x2 both_halves(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t x = s[0], y = s[1];  // a bit cast of s[1] itself takes s[0]
  return f32x2{__builtin_bit_cast(float, x), __builtin_bit_cast(float, y)};
}
__device__ __forceinline__ float halves_max(float v) {
  const f32x2 s = both_halves(v);
  return fmaxf(s.x, s.y);
}
__device__ __forceinline__ float halves_sum(float v) {
  const f32x2 s = both_halves(v);
  return s.x + s.y;
}

// MT: q's and out's type. CT: the cache's, MT or kE4M3. DP: dim rounded up.
template <int MT, int CT, int DP>
__global__ __launch_bounds__(kThreads, DP <= 128 ? 2 : 1) void attn_prefill_kernel(PrefillArgs a) {
  constexpr int EB = CT == kE4M3 ? 1 : 2;
  constexpr int RB = DP * 2 + 16;            // bytes of a row in LDS
  constexpr int CH = DP / 8;                 // 8-dim pieces of a row
  constexpr int PER = kTile * CH / kThreads; // of a thread, K and V each
  constexpr int DT = DP / 32;
  constexpr uint32_t kInf2 = MT == kBF16 ? 0x7f80u : 0x7c00u;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ int64_t offs[3][2][kTile];      // of a tile's tokens in k and v, -1: none
  __shared__ int odd[3];                     // a masked tile's V holds infinities or NaN

  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int l32 = lane % 32, lh = lane / 32;
  // Units (sequence, kv head) go to the XCDs in turn, so that one's keys and
  // values stay in one L2; the late tiles, which see most, start first.
  const int units = a.seqs * a.kv_heads;
  int unit, tile;
  if (units % 8 == 0) {
    const int x = blockIdx.x % 8, y = blockIdx.x / 8, per = units / 8;
    unit = x + 8 * (y % per);
    tile = a.tiles - 1 - y / per;
  } else {
    unit = blockIdx.x % units;
    tile = a.tiles - 1 - blockIdx.x / units;
  }
  const int seq = unit / a.kv_heads, kvh = unit % a.kv_heads;

  const int first = min(max(a.starts[seq], 0), a.rows);
  const int count = min(min(max(a.starts[seq + 1], first), a.rows) - first, a.max_chunk);
  const int group = a.group.d;
  const int row0 = tile * kRows;
  if (row0 >= count * group) return;
  const int n = static_cast<int>(min(static_cast<int64_t>(max(0, a.lens[seq])), a.table_tokens));
  const int base = n - count;  // position of the chunk's first token; may be below 0

  // This lane's row.
  const int r = row0 + wave * 32 + l32;
  const bool mine = r < count * group;
  const int tok = mine ? div_by(r, a.group) : 0;
  const int head = kvh * group + (r - tok * group);
  const int pos = mine ? base + tok : -1;
  const int from = a.window ? pos - a.window : -1;  // sees j > from, or j < sinks
  const int sinks = a.window ? a.sinks : 0;

  // The workgroup's tokens: the sinks' tiles, then those from `lo` on.
  const int pmin = base + div_by(row0, a.group);
  const int pmax = base + div_by(min(row0 + kRows, count * group) - 1, a.group);
  const int lo = a.window ? max(0, pmin - a.window + 1) / kTile * kTile : 0;
  const int ns = min(sinks, lo);
  const int sink_tiles = (ns + kTile - 1) / kTile;
  const int tiles = sink_tiles + (pmax + 1 > lo ? (pmax + 1 - lo + kTile - 1) / kTile : 0);
  auto tile_begin = [&](int t) { return t < sink_tiles ? t * kTile : lo + (t - sink_tiles) * kTile; };
  auto tile_end = [&](int t) { return t < sink_tiles ? min(ns, (t + 1) * kTile) : min(pmax + 1, tile_begin(t) + kTile); };

  u32x4 qf[DP / 16];
  {
    const uint8_t* qr = a.q + (first + tok) * a.q_row + head * a.q_head;
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) {
      const int d0 = s * 16 + lh * 8;
      qf[s] = u32x4{0, 0, 0, 0};
      if (mine && d0 < a.dim) qf[s] = *reinterpret_cast<const u32x4*>(qr + d0 * 2);
    }
  }

  const uint8_t* kb = a.kv.k + kvh * a.kv.k_head;
  const uint8_t* vb = a.kv.v + kvh * a.kv.v_head;
  const int32_t* table = a.tables + seq * a.table_stride;
  // The first 64 threads look up a tile's tokens.
  auto page_of = [&](int t) {
    const int j = tile_begin(t) + tid;
    return t < tiles && tid < kTile && j < tile_end(t) ? table[div_by(j, a.kv.page)] : -1;
  };
  auto place = [&](int t, int page) {
    if (tid < kTile) {
      const uint32_t j = tile_begin(t) + tid;
      const bool ok = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.kv.pages);
      const uint32_t slot = j - div_by(j, a.kv.page) * a.kv.page.d;
      offs[t % 3][0][tid] = ok ? page * a.kv.k_page + slot * a.kv.k_tok : -1;
      offs[t % 3][1][tid] = ok ? page * a.kv.v_page + slot * a.kv.v_tok : -1;
    }
  };
  u32x4 kr[PER], vr[PER];
  auto load = [&](int t, int which, const uint8_t* from, u32x4(&reg)[PER]) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = tid + i * kThreads, row = at / CH, d0 = (at % CH) * 8;
      const int64_t off = offs[t % 3][which][row];
      reg[i] = u32x4{0, 0, 0, 0};
      if (off >= 0 && d0 < a.dim) {
        if constexpr (EB == 2) {
          reg[i] = *reinterpret_cast<const u32x4*>(from + off + d0 * 2);
        } else {
          const u32x2 w = *reinterpret_cast<const u32x2*>(from + off + d0);
          reg[i] = u32x4{w.x, w.y, 0, 0};
        }
      }
    }
  };
  auto widen = [&](u32x4 w) {
    if constexpr (EB == 2) {
      return w;
    } else {
      const u32x2 x = widen4<MT>(w.x), y = widen4<MT>(w.y);
      return u32x4{x.x, x.y, y.x, y.y};
    }
  };
  // Whether every row of the workgroup sees every token of tile t (its own
  // lookups aside).
  auto plain_tile = [&](int t) {
    const int b = tile_begin(t), e = b + kTile;
    if (e > tile_end(t) || e - 1 > pmin || (a.window && b <= pmax - a.window && e > sinks)) return false;
    return true;
  };
  auto put = [&](int t) {
    uint8_t* kl = smem + (t % 2) * (2 * kTile * RB);
    uint8_t* vl = kl + kTile * RB;
    const bool all = plain_tile(t);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = tid + i * kThreads, row = at / CH, c = at % CH;
      *reinterpret_cast<u32x4*>(kl + row * RB + c * 16) = widen(kr[i]);
      u32x4 w = widen(vr[i]);
      if (!all) {
        // 0 * infinity must not reach a row that does not see the token: such
        // values are left out here and added to the rows that do.
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool x = (w[e] & kInf2) == kInf2, y = ((w[e] >> 16) & kInf2) == kInf2;
          if (x || y) odd[t % 3] = 1;
          w[e] &= (x ? 0u : 0xffffu) | (y ? 0u : 0xffff0000u);
        }
      }
      *reinterpret_cast<u32x4*>(vl + row * RB + c * 16) = w;
    }
  };

  f32x16 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  float m = -INFINITY, l = 0.f;

  if (tid < 3) odd[tid] = 0;
  place(0, page_of(0));
  place(1, page_of(1));
  __syncthreads();
  if (tiles > 0) {
    load(0, 0, kb, kr);
    load(0, 1, vb, vr);
    put(0);
  }
  __syncthreads();

  for (int t = 0; t < tiles; ++t) {
    const int page = page_of(t + 2);
    if (tid == 0) odd[(t + 2) % 3] = 0;  // last read before the barrier, next set after the coming one
    if (t + 1 < tiles) {
      load(t + 1, 0, kb, kr);
      load(t + 1, 1, vb, vr);
    }
    const uint8_t* kl = smem + (t % 2) * (2 * kTile * RB);
    const uint8_t* vl = kl + kTile * RB;

    f32x16 st[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 16; ++i) st[h][i] = 0.f;
#pragma unroll
      for (int s = 0; s < DP / 16; ++s) {
        const u32x4 kf = *reinterpret_cast<const u32x4*>(kl + (h * 32 + l32) * RB + (s * 16 + lh * 8) * 2);
        st[h] = mfma32<MT>(kf, qf[s], st[h]);
      }
    }

    // A tile whose pages are all there and that every row sees needs no mask.
    const int b = tile_begin(t), e = tile_end(t);
    const uint64_t there = __ballot(offs[t % 3][0][lane] >= 0);
    const bool masked = !plain_tile(t) || there != ~0ull;
    float top = -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float x = st[h][i] * a.c;
        if (masked) {
          const int k = h * 32 + 8 * (i / 4) + 4 * lh + i % 4, j = b + k;
          const bool sees = ((there >> k) & 1) && j < e && j <= pos && (j > from || j < sinks);
          if (!sees) x = -INFINITY;
        }
        st[h][i] = x;
        top = fmaxf(top, x);
      }
    top = fmaxf(m, halves_max(top));
    const float ref = top == -INFINITY ? 0.f : top;
    const float alpha = exp2_fast(m - ref);
    m = top;
    float sum = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        st[h][i] = exp2_fast(st[h][i] - ref);
        sum += st[h][i];
      }
    l = l * alpha + sum;
    if (__ballot(alpha != 1.f)) {
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= alpha;
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      u32x4 pf;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        pf[i] = pack2<MT>(st[s / 2][(s % 2) * 8 + 2 * i], st[s / 2][(s % 2) * 8 + 2 * i + 1]);
      const uint8_t* vp = vl + (16 * s + 4 * lh + (lane % 16) / 4) * RB +
                          (16 * ((lane / 16) % 2) + (lane % 4) * 4) * 2;
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const u32x2 x = load_transposed(vp + d * 64), y = load_transposed(vp + 8 * RB + d * 64);
        o[d] = mfma32<MT>(u32x4{x.x, x.y, y.x, y.y}, pf, o[d]);
      }
    }
    if (odd[t % 3]) {
      // Infinities and NaN of this tile, for the rows that see them.
      for (int k = 0; k < kTile; ++k) {
        const int64_t off = offs[t % 3][1][k];
        const int j = b + k;
        if (off < 0) continue;
        const bool sees = j < e && j <= pos && (j > from || j < sinks);
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int dim = d * 32 + 8 * (i / 4) + 4 * lh + i % 4;
            if (sees && dim < a.dim) {
              float x;
              if constexpr (EB == 2) {
                x = load_as_f32(vb + off, MT, dim);
              } else {
                x = unpack2<MT>(widen4<MT>(vb[off + dim]).x).x;
              }
              if (!(fabsf(x) < INFINITY)) o[d][i] += x;
            }
          }
      }
    }

    if (t + 1 < tiles) put(t + 1);
    if (t + 2 < tiles) place(t + 2, page);
    __syncthreads();
  }

  l = halves_sum(l);
  const float inv = l == 0.f ? 0.f : a.v_scale / l;
  if (mine) {
    uint8_t* row = a.out + (first + tok) * a.out_row + head * a.out_head;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int dim = d * 32 + 8 * (i / 4) + 4 * lh;
        if (dim < a.dim)
          *reinterpret_cast<u32x2*>(row + dim * 2) =
              u32x2{pack2<MT>(o[d][i] * inv, o[d][i + 1] * inv), pack2<MT>(o[d][i + 2] * inv, o[d][i + 3] * inv)};
      }
  }
}

int64_t row_tiles(int64_t heads, const xq_kv& kv, int64_t max_chunk) {
  return (max_chunk * (heads / kv.kv_heads) + kRows - 1) / kRows;
}

template <int MT, int CT, int DP>
hipError_t launch(const PrefillArgs& a, uint32_t blocks, hipStream_t stream) {
  constexpr int lds = 2 * 2 * kTile * (DP * 2 + 16);
  auto kernel = attn_prefill_kernel<MT, CT, DP>;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  kernel<<<dim3(blocks), dim3(kThreads), lds, stream>>>(a);
  return hipGetLastError();
}

template <int MT, int CT>
hipError_t launch_dim(const PrefillArgs& a, uint32_t blocks, hipStream_t stream) {
  if (a.dim <= 64) return launch<MT, CT, 64>(a, blocks, stream);
  if (a.dim <= 96) return launch<MT, CT, 96>(a, blocks, stream);
  if (a.dim <= 128) return launch<MT, CT, 128>(a, blocks, stream);
  if (a.dim <= 192) return launch<MT, CT, 192>(a, blocks, stream);
  return launch<MT, CT, 256>(a, blocks, stream);
}

}  // namespace

int64_t attn_prefill_blocks(int64_t seqs, int64_t heads, const xq_kv& kv, int64_t max_chunk) {
  return seqs * kv.kv_heads * row_tiles(heads, kv, max_chunk);
}

hipError_t launch_attn_prefill(const RowsView& out, const RowsView& q, int64_t rows, int64_t seqs,
                               int64_t heads, const xq_kv& kv, const TableView& tables,
                               const int32_t* lens, const int32_t* starts, int64_t max_chunk,
                               float scale, int64_t window, int64_t sinks, hipStream_t stream) {
  const int eb = elem_bytes(kv.dtype);
  PrefillArgs a;
  a.kv = KvView{static_cast<uint8_t*>(kv.k), static_cast<uint8_t*>(kv.v),
                kv.k_stride[1] * eb, kv.k_stride[2] * eb, kv.k_stride[3] * eb,
                kv.v_stride[1] * eb, kv.v_stride[2] * eb, kv.v_stride[3] * eb,
                fast_div(static_cast<uint32_t>(kv.page)), static_cast<int>(kv.pages)};
  a.q = static_cast<const uint8_t*>(q.data);
  a.out = static_cast<uint8_t*>(out.data);
  a.tables = tables.data;
  a.lens = lens;
  a.starts = starts;
  a.q_row = q.row * 2;
  a.q_head = q.head * 2;
  a.out_row = out.row * 2;
  a.out_head = out.head * 2;
  a.table_stride = tables.stride;
  // Positions stay below 2^30.
  a.table_tokens = std::min<int64_t>(tables.width * kv.page, 1 << 30);
  a.group = fast_div(static_cast<uint32_t>(heads / kv.kv_heads));
  a.rows = static_cast<int>(rows);
  a.seqs = static_cast<int>(seqs);
  a.kv_heads = static_cast<int>(kv.kv_heads);
  a.dim = static_cast<int>(kv.dim);
  a.max_chunk = static_cast<int>(max_chunk);
  a.window = static_cast<int>(window);
  a.sinks = static_cast<int>(sinks);
  a.tiles = static_cast<int>(row_tiles(heads, kv, max_chunk));
  a.c = scale * kv.k_scale * kLog2e;
  a.v_scale = kv.v_scale;
  const uint32_t blocks = static_cast<uint32_t>(attn_prefill_blocks(seqs, heads, kv, max_chunk));
  if (q.type == kBF16)
    return kv.dtype == kBF16 ? launch_dim<kBF16, kBF16>(a, blocks, stream)
                             : launch_dim<kBF16, kE4M3>(a, blocks, stream);
  return kv.dtype == kF16 ? launch_dim<kF16, kF16>(a, blocks, stream)
                          : launch_dim<kF16, kE4M3>(a, blocks, stream);
}

}  // namespace xq
