// attn_decode.hip — attention of one new token per sequence over a paged cache.
//
//   s_j = scale * k_scale * (q . k_j),  out = sum_j exp(s_j - m) v_scale v_j / sum_j exp(s_j - m)
//
// over a sequence's visible tokens. One pass: a wave keeps the running maximum
// m, the sum l and the unnormalised output o of the tokens it has seen; a new
// maximum m' scales l and o by exp(m - m'). Partial results (m, l, o) of the
// waves of a workgroup, and of workgroups that split a long sequence, are
// joined by the same rule.
//
// What bounds it: the cache's bytes. A wave takes 32 tokens at a time for all
// the heads that share one kv head (up to 16 are one matrix instruction's
// columns), so each byte is read once, straight from memory into the registers
// of the matrix instructions:
//  - S^T = K Q^T, 16 tokens x 16 heads per instruction. K's operand wants 8
//    consecutive dims of one token per lane: a 16-byte load. Lane l gets head
//    l % 16, tokens 4 * (l / 16) + i of each 16.
//  - O^T = V^T P^T over the 32 tokens. The order of the summed index is free
//    as long as both operands agree, so P goes from S^T's registers straight
//    into the instruction: element i of lane group g is token 4g + i of the
//    first 16, element 4 + i of the second. V's operand wants one dim of those
//    eight tokens: a lane loads 8 consecutive dims of each of its 8 tokens (16
//    lanes cover a whole row) and turns the 8 x 8 block around with byte
//    permutes. Both m and l belong to head l % 16, which is also the lane's
//    column of O^T, so rescaling is local to the lane.
// The next tile's K is asked for before this tile's softmax, its V right after
// this tile's product, the page numbers one tile earlier.
//
// Precision: q and the weights p enter the 16-bit matrix instructions as sums
// of pieces (each the rounded remainder of the one before). For a 16-bit
// output: q exactly, p in two pieces (2^-16 or better). For an f32 output: as
// many pieces as f32 has bits (three of bf16's 8, two of f16's 11). The
// instructions wait on memory, so the pieces cost no time.
#include <algorithm>

#include "kv_device.h"
#include "kv_launch.h"

namespace xq {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kTile = 32;                   // tokens of a wave's step
constexpr int kStep = kTile * kWaves;       // tokens of a workgroup's step
constexpr int kHeadTile = 16;               // heads of one workgroup
constexpr int kCounterStride = 32;          // ints: a 128-byte line per arrival counter
constexpr int64_t kMaxSplitUnits = 768;     // 96 KiB of counters, at the same place in every plan
constexpr int kMaxSplits = 256;
constexpr int kWaitVm0 = 0x0f70;            // s_waitcnt vmcnt(0), others untouched
constexpr float kLog2e = 1.44269504088896340736f;

struct DecodeArgs {
  KvView kv;
  const uint8_t* q;
  uint8_t* out;
  const int32_t* tables;
  const int32_t* lens;
  float* part;
  int32_t* count;
  int64_t q_row, q_head, out_row, out_head;  // bytes
  int64_t table_stride, table_tokens;        // table_width * page
  int kv_heads, group, dim, io, max_len, window, sinks, chunk, splits, head_tiles;
  float c;        // scale * k_scale * log2(e)
  float v_scale;
};

// Sum and maximum over the four lanes that hold one head.
__device__ __forceinline__ float heads_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, kWave));
  return fmaxf(v, __shfl_xor(v, 32, kWave));
}
__device__ __forceinline__ float heads_sum(float v) {
  v += __shfl_xor(v, 16, kWave);
  return v + __shfl_xor(v, 32, kWave);
}

template <int BYTES>
__device__ __forceinline__ u32x4 load_words(const uint8_t* p) {
  if constexpr (BYTES == 16) {
    return *reinterpret_cast<const u32x4*>(p);
  } else if constexpr (BYTES == 8) {
    const u32x2 v = *reinterpret_cast<const u32x2*>(p);
    return u32x4{v.x, v.y, 0, 0};
  } else {
    return u32x4{*reinterpret_cast<const uint32_t*>(p), 0, 0, 0};
  }
}

// CT: the cache's type. DP: dim rounded up to 64, 128, 192 or 256. NQ, NP:
// pieces of q and of p.
template <int CT, int DP, int NQ, int NP>
__global__ __launch_bounds__(kThreads, DP <= 128 ? 2 : 1) void attn_decode_kernel(DecodeArgs a) {
  constexpr int MT = CT == kBF16 ? kBF16 : kF16;   // the matrix instruction's type
  constexpr int EB = CT == kE4M3 ? 1 : 2;
  constexpr int QS = DP / 32;                      // instructions of S^T along dim
  // One K load gives KL instructions their operand: an 8-bit row's 16 bytes
  // are 16 dims, two instructions' worth.
  constexpr int KL = CT == kE4M3 ? 2 : 1;
  constexpr int KN = QS / KL;
  constexpr int VE = DP == 64 ? 4 : 8;             // dims of a lane's V load
  constexpr int VC = (DP + 16 * VE - 1) / (16 * VE);
  constexpr int OS = DP + 4;                       // floats of a joined row in LDS
  extern __shared__ float lds[];

  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int l16 = lane % 16, lg = lane / 16;
  const int unit = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
  const int ht = unit % a.head_tiles;
  const int kvh = (unit / a.head_tiles) % a.kv_heads;
  const int seq = unit / a.head_tiles / a.kv_heads;
  const int heads = min(kHeadTile, a.group - ht * kHeadTile);  // of this workgroup
  const int head0 = kvh * a.group + ht * kHeadTile;

  // The visible tokens as one run: `ns` sinks, then lo .. n-1.
  const int n = static_cast<int>(
      min(static_cast<int64_t>(max(0, min(a.lens[seq], a.max_len))), a.table_tokens));
  const int lo = a.window && n > a.window ? n - a.window : 0;
  const int ns = min(a.sinks, lo);
  const int nv = n - lo + ns;
  const int n_splits = max(1, (nv + a.chunk - 1) / a.chunk);
  if (split >= n_splits) return;
  const int begin = split * a.chunk, end = min(nv, begin + a.chunk);

  const uint8_t* kb = a.kv.k + kvh * a.kv.k_head;
  const uint8_t* vb = a.kv.v + kvh * a.kv.v_head;
  const int32_t* table = a.tables + seq * a.table_stride;

  // q as the B operand: head l16, dims of step s. An f16 operand is scaled by
  // a power of two that brings the head's largest |q| to 2^14..2^15, so that
  // no piece of an f32 or bf16 q leaves f16's range.
  u32x4 qf[QS][NQ];
  float qs = a.c;
  {
    float x[QS][8];
    float top = 0.f;
    const uint8_t* qr = a.q + seq * a.q_row + (head0 + l16) * a.q_head;
#pragma unroll
    for (int s = 0; s < QS; ++s) {
      const int d0 = KL == 1 ? s * 32 + lg * 8 : (s / 2) * 64 + lg * 16 + (s % 2) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[s][e] = l16 < heads && d0 < a.dim ? load_as_f32(qr, a.io, d0 + e) : 0.f;
        top = fmaxf(top, fabsf(x[s][e]));
      }
    }
    float mul = 1.f;
    if constexpr (MT == kF16) {
      top = heads_max(top);
      if (top > 0.f && top < INFINITY) {
        const int e = ilogbf(top);
        mul = ldexpf(1.f, min(127, 14 - e));
        qs = a.c * ldexpf(1.f, max(-127, e - 14));
      }
    }
#pragma unroll
    for (int s = 0; s < QS; ++s)
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        float u = x[s][e] * mul, w = x[s][e + 1] * mul;
#pragma unroll
        for (int p = 0; p < NQ; ++p) {
          const uint32_t h = pack2<MT>(u, w);
          qf[s][p][e / 2] = h;
          const f32x2 back = unpack2<MT>(h);
          u -= back.x;
          w -= back.y;
        }
      }
  }

  const f32x4 zero4 = {0.f, 0.f, 0.f, 0.f};
  f32x4 o[VC][VE];
#pragma unroll
  for (int c = 0; c < VC; ++c)
#pragma unroll
    for (int j = 0; j < VE; ++j) o[c][j] = zero4;
  float m = -INFINITY, l = 0.f;

  // The page of this lane's token (l % 32) of a tile, and its place.
  auto token_of = [&](int u) { return u < ns ? u : lo + (u - ns); };
  auto page_of = [&](int u0) {
    const int u = u0 + lane % kTile;
    return u < end ? table[div_by(token_of(u), a.kv.page)] : -1;
  };
  int64_t koff, voff;
  uint32_t live;  // bit t: token t of the tile is there
  auto place = [&](int u0, int page) {
    const int u = u0 + lane % kTile;
    const bool ok = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.kv.pages);
    const uint32_t j = token_of(u);
    const uint32_t slot = j - div_by(j, a.kv.page) * a.kv.page.d;
    // A token that is not there reads page 0, which always is; its score is
    // hidden and its v is cleared.
    koff = ok ? page * a.kv.k_page + slot * a.kv.k_tok : 0;
    voff = ok ? page * a.kv.v_page + slot * a.kv.v_tok : 0;
    live = static_cast<uint32_t>(__ballot(ok));
  };
  u32x4 kr[2][KN], vr[VC][8];
  auto load_k = [&]() {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint8_t* p = kb + __shfl(koff, t * 16 + l16, kWave);
#pragma unroll
      for (int s = 0; s < KN; ++s) {
        const int d0 = s * 32 * KL + lg * 8 * KL;
        kr[t][s] = u32x4{0, 0, 0, 0};
        if (d0 < a.dim) kr[t][s] = load_words<16>(p + d0 * EB);
      }
    }
  };
  auto load_v = [&]() {
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const uint8_t* p = vb + __shfl(voff, (t / 4) * 16 + lg * 4 + t % 4, kWave);
#pragma unroll
      for (int c = 0; c < VC; ++c) {
        const int d0 = (c * 16 + l16) * VE;
        vr[c][t] = u32x4{0, 0, 0, 0};
        if (d0 < a.dim) vr[c][t] = load_words<VE * EB>(p + d0 * EB);
      }
    }
  };

  auto widen_v = [&](const u32x4(&r)[8], u32x4(&w)[8]) {
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if constexpr (CT == kE4M3) {
        const u32x2 x = widen4<MT>(r[t].x), y = widen4<MT>(r[t].y);
        w[t] = u32x4{x.x, x.y, y.x, y.y};
      } else {
        w[t] = r[t];
      }
    }
  };
  // Dim j of the lane's eight tokens (`flip` is 0).
  auto turned = [&](const u32x4(&w)[8], int j, uint32_t flip) {
    const uint32_t sel = (j % 2 ? 0x07060302u : 0x05040100u) + flip;
    u32x4 f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __builtin_amdgcn_perm(w[2 * i + 1][j / 2], w[2 * i][j / 2], sel);
    return f;
  };

  int u0 = begin + wave * kTile;
  int page = -1;
  if (u0 < end) {
    page = page_of(u0);
    place(u0, page);
    page = page_of(u0 + kStep);
    load_k();
    load_v();
  }
  while (u0 < end) {  // wave-uniform
    const uint32_t here = live;
    const int next = u0 + kStep;
    if (next < end) {
      place(next, page);
      page = page_of(next + kStep);
    }

    f32x4 st[2] = {zero4, zero4};
#pragma unroll
    for (int s = 0; s < QS; ++s)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        u32x4 kf;
        if constexpr (KL == 2) {
          const u32x4 w = kr[t][s / 2];
          const u32x2 x = widen4<MT>(w[(s % 2) * 2]), y = widen4<MT>(w[(s % 2) * 2 + 1]);
          kf = u32x4{x.x, x.y, y.x, y.y};
        } else {
          kf = kr[t][s];
        }
#pragma unroll
        for (int p = 0; p < NQ; ++p) st[t] = mfma16<MT>(kf, qf[s][p], st[t]);
      }
    if (next < end) load_k();

    float s[8];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[i] = st[i / 4][i % 4] * qs;
      if (!((here >> ((i / 4) * 16 + lg * 4 + i % 4)) & 1)) s[i] = -INFINITY;
      top = fmaxf(top, s[i]);
    }
    top = fmaxf(m, heads_max(top));
    const float base = top == -INFINITY ? 0.f : top;
    const float alpha = exp2_fast(m - base);
    m = top;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[i] = exp2_fast(s[i] - base);
      sum += s[i];
    }
    l = l * alpha + sum;
    if (__ballot(alpha != 1.f)) {
#pragma unroll
      for (int c = 0; c < VC; ++c)
#pragma unroll
        for (int j = 0; j < VE; ++j) o[c][j] *= alpha;
    }
    u32x4 pf[NP];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      // f16 pieces of weights up to 2^14, so that small ones keep their bits
      // (the join divides the factor out).
      float u = s[i], w = s[i + 1];
      if constexpr (MT == kF16) {
        u *= 16384.f;
        w *= 16384.f;
      }
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const uint32_t h = pack2<MT>(u, w);
        pf[p][i / 2] = h;
        const f32x2 back = unpack2<MT>(h);
        u -= back.x;
        w -= back.y;
      }
    }
    if (here != 0xffffffffu) {
      // What lies in a place without a token may be anything, NaN too.
#pragma unroll
      for (int t = 0; t < 8; ++t)
        if (!((here >> ((t / 4) * 16 + lg * 4 + t % 4)) & 1))
#pragma unroll
          for (int c = 0; c < VC; ++c) vr[c][t] = u32x4{0, 0, 0, 0};
    }
    // Whether the tile's V has an infinity or NaN: an exponent of all ones
    // carries into the sign's place. (An 8-bit V has no infinity, and NaN needs
    // no care.)
    bool odd = false;
    if constexpr (CT != kE4M3) {
      constexpr uint32_t kOne = CT == kBF16 ? 0x00800080u : 0x04000400u;
      uint32_t carry = 0;
#pragma unroll
      for (int c = 0; c < VC; ++c)
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int i = 0; i < VE / 2; ++i) carry |= (vr[c][t][i] & 0x7fff7fffu) + kOne;
      odd = __ballot(carry & 0x80008000u) != 0;
    }
    if (!odd) {
#pragma unroll
      for (int c = 0; c < VC; ++c) {
        u32x4 vw[8];
        widen_v(vr[c], vw);
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const u32x4 vf = turned(vw, j, 0);
#pragma unroll
          for (int p = 0; p < NP; ++p) o[c][j] = mfma16<MT>(vf, pf[p], o[c][j]);
        }
      }
    } else {
      // An infinity times p's first piece is the infinity it should be; times
      // a further piece, which may be 0 or below, it is not. (The zero that the
      // compiler does not know keeps this path's turning of V its own: shared
      // with the other path's it is done ahead of both and spills.)
      uint32_t flip = 0;
      asm volatile("" : "+s"(flip));
#pragma unroll
      for (int c = 0; c < VC; ++c) {
        u32x4 vw[8];
        widen_v(vr[c], vw);
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const u32x4 vf = turned(vw, j, flip);
          f32x4 x = zero4;
#pragma unroll
          for (int p = 1; p < NP; ++p) x = mfma16<MT>(vf, pf[p], x);
          o[c][j] = mfma16<MT>(vf, pf[0], o[c][j]);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (fabsf(x[i]) < INFINITY) o[c][j][i] += x[i];
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    if (next < end) load_v();
    u0 = next;
  }

  // Join the waves: LDS rows [wave][head] of o, then m and l.
  l = heads_sum(l);
  float* lm = lds + kWaves * heads * OS;
  if (l16 < heads) {
    float* row = lds + (wave * heads + l16) * OS;
#pragma unroll
    for (int c = 0; c < VC; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d0 = (c * 16 + lg * 4 + i) * VE;
        if (d0 >= DP) continue;
#pragma unroll
        for (int j = 0; j < VE; j += 4)
          *reinterpret_cast<f32x4*>(row + d0 + j) =
              f32x4{o[c][j][i], o[c][j + 1][i], o[c][j + 2][i], o[c][j + 3][i]};
      }
    if (lg == 0) {
      lm[wave * heads + l16] = m;
      lm[(kWaves + wave) * heads + l16] = l;
    }
  }
  __syncthreads();

  constexpr float kPScale = MT == kF16 ? 1.f / 16384.f : 1.f;
  const bool whole = n_splits == 1;
  float* po = a.part + (static_cast<int64_t>(unit) * a.splits) * kHeadTile * (DP + 2);
  for (int i = tid; i < heads * DP; i += kThreads) {
    const int r = i / DP, d = i % DP;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, lm[w * heads + r]);
    const float base = top == -INFINITY ? 0.f : top;
    float x = 0.f, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float f = exp2_fast(lm[w * heads + r] - base);
      x += f * lds[(w * heads + r) * OS + d];
      sum += f * lm[(kWaves + w) * heads + r];
    }
    x *= kPScale;
    if (whole) {
      if (d < a.dim)
        store_from_f32(a.out + seq * a.out_row + (head0 + r) * a.out_head, a.io, d,
                       sum == 0.f ? 0.f : x / sum * a.v_scale);
    } else {
      float* mine = po + split * heads * (DP + 2);
      __hip_atomic_store(mine + i, x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (d == 0) {
        __hip_atomic_store(mine + heads * DP + r, top, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(mine + heads * DP + heads + r, sum, __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
      }
    }
  }
  if (whole) return;

  // The last split to arrive joins them all. The partials and the counter are
  // agent-scope atomics, which bypass the per-XCD L2's non-coherent state; each
  // wave waits for its stores' acknowledgement before the barrier, so whoever
  // sees the last count sees every partial.
  __shared__ int last;
  __builtin_amdgcn_s_waitcnt(kWaitVm0);
  __syncthreads();
  if (tid == 0)
    last = __hip_atomic_fetch_add(a.count + static_cast<int64_t>(unit) * kCounterStride, 1,
                                  __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == n_splits - 1;
  __syncthreads();
  if (!last) return;  // workgroup-uniform
  if (tid == 0)
    __hip_atomic_store(a.count + static_cast<int64_t>(unit) * kCounterStride, 0, __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
  // Each split's factor per head, exp(m - max m) / sum, in LDS.
  for (int r = wave; r < heads; r += kWaves) {
    float sm[kMaxSplits / kWave], sl[kMaxSplits / kWave];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kMaxSplits / kWave; ++i) {
      const int sp = i * kWave + lane;
      sm[i] = -INFINITY;
      sl[i] = 0.f;
      if (sp < n_splits) {
        const float* p = po + sp * heads * (DP + 2) + heads * DP + r;
        sm[i] = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        sl[i] = __hip_atomic_load(p + heads, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      top = fmaxf(top, sm[i]);
    }
    top = wave_max(top);
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxSplits / kWave; ++i) {
      sm[i] = exp2_fast(sm[i] - base);
      sum += sm[i] * sl[i];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < kMaxSplits / kWave; ++i) {
      const int sp = i * kWave + lane;
      if (sp < n_splits) lds[r * kMaxSplits + sp] = sum == 0.f ? 0.f : sm[i] / sum * a.v_scale;
    }
  }
  __syncthreads();
  for (int i = tid; i < heads * DP; i += kThreads) {
    const int r = i / DP, d = i % DP;
    float x = 0.f;
#pragma unroll 8
    for (int sp = 0; sp < n_splits; ++sp)
      x += lds[r * kMaxSplits + sp] * __hip_atomic_load(po + sp * heads * (DP + 2) + i,
                                                        __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (d < a.dim)
      store_from_f32(a.out + seq * a.out_row + (head0 + r) * a.out_head, a.io, d, x);
  }
}

int dim_pad(int64_t dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : dim <= 192 ? 192 : 256; }

struct Plan {
  int64_t head_tiles, units, chunk, splits;
};
// How many tokens a workgroup takes. The card holds 512 of these workgroups at
// once; a split is worth its join from 128 tokens (one step) on.
Plan plan(int64_t seqs, int64_t heads, const xq_kv& kv, int64_t max_len, int64_t window,
          int64_t sinks) {
  Plan p;
  const int64_t group = heads / kv.kv_heads;
  p.head_tiles = (group + kHeadTile - 1) / kHeadTile;
  p.units = seqs * kv.kv_heads * p.head_tiles;
  const int64_t most = window && window + sinks < max_len ? window + sinks : max_len;
  const int64_t want = p.units > kMaxSplitUnits ? 1 : std::max<int64_t>(1, 1024 / p.units);
  int64_t chunk = (most + want - 1) / want;
  chunk = std::max<int64_t>(chunk, want == 1 ? most : (most + kMaxSplits - 1) / kMaxSplits);
  p.chunk = std::max<int64_t>(1, (chunk + kStep - 1) / kStep) * kStep;
  p.splits = (most + p.chunk - 1) / p.chunk;
  return p;
}

constexpr size_t kCounterBytes = kMaxSplitUnits * kCounterStride * 4;

template <int CT, int DP, int NQ, int NP>
hipError_t launch(const DecodeArgs& a, const Plan& p, hipStream_t stream) {
  const int heads = std::min(kHeadTile, a.group);
  size_t lds = static_cast<size_t>(kWaves) * heads * (DP + 4 + 2) * 4;
  if (p.splits > 1) lds = std::max(lds, static_cast<size_t>(heads) * kMaxSplits * 4);
  auto kernel = attn_decode_kernel<CT, DP, NQ, NP>;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(lds));
    if (e != hipSuccess) return e;
  }
  kernel<<<dim3(static_cast<uint32_t>(p.units * p.splits)), dim3(kThreads), lds, stream>>>(a);
  return hipGetLastError();
}

template <int CT, int NQ, int NP>
hipError_t launch_dim(const DecodeArgs& a, const Plan& p, hipStream_t stream) {
  switch (dim_pad(a.dim)) {
    case 64: return launch<CT, 64, NQ, NP>(a, p, stream);
    case 128: return launch<CT, 128, NQ, NP>(a, p, stream);
    case 192: return launch<CT, 192, NQ, NP>(a, p, stream);
    default: return launch<CT, 256, NQ, NP>(a, p, stream);
  }
}

}  // namespace

size_t attn_decode_workspace_bytes(int64_t seqs, int64_t heads, const xq_kv& kv, int64_t max_len,
                                   int64_t window, int64_t sinks) {
  const Plan p = plan(seqs, heads, kv, max_len, window, sinks);
  if (p.splits == 1) return 0;
  return kCounterBytes + static_cast<size_t>(p.units) * p.splits * kHeadTile *
                                (dim_pad(kv.dim) + 2) * 4;
}

hipError_t launch_attn_decode(const RowsView& out, const RowsView& q, int64_t seqs, int64_t heads,
                              const xq_kv& kv, const TableView& tables, const int32_t* lens,
                              float scale, int64_t window, int64_t sinks, int64_t max_len, void* ws,
                              hipStream_t stream) {
  const Plan p = plan(seqs, heads, kv, max_len, window, sinks);
  const int eb = elem_bytes(kv.dtype), ib = elem_bytes(q.type);
  DecodeArgs a;
  a.kv = KvView{static_cast<uint8_t*>(kv.k), static_cast<uint8_t*>(kv.v),
                kv.k_stride[1] * eb, kv.k_stride[2] * eb, kv.k_stride[3] * eb,
                kv.v_stride[1] * eb, kv.v_stride[2] * eb, kv.v_stride[3] * eb,
                fast_div(static_cast<uint32_t>(kv.page)), static_cast<int>(kv.pages)};
  a.q = static_cast<const uint8_t*>(q.data);
  a.out = static_cast<uint8_t*>(out.data);
  a.tables = tables.data;
  a.lens = lens;
  a.count = static_cast<int32_t*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kCounterBytes);
  a.q_row = q.row * ib;
  a.q_head = q.head * ib;
  a.out_row = out.row * ib;
  a.out_head = out.head * ib;
  a.table_stride = tables.stride;
  a.table_tokens = tables.width * kv.page;
  a.kv_heads = static_cast<int>(kv.kv_heads);
  a.group = static_cast<int>(heads / kv.kv_heads);
  a.dim = static_cast<int>(kv.dim);
  a.io = q.type;
  a.max_len = static_cast<int>(max_len);
  a.window = static_cast<int>(window);
  a.sinks = static_cast<int>(sinks);
  a.chunk = static_cast<int>(p.chunk);
  a.splits = static_cast<int>(p.splits);
  a.head_tiles = static_cast<int>(p.head_tiles);
  a.c = scale * kv.k_scale * kLog2e;
  a.v_scale = kv.v_scale;
  switch (kv.dtype) {
    case kBF16:
      return q.type == kBF16 ? launch_dim<kBF16, 1, 2>(a, p, stream)
                             : launch_dim<kBF16, 3, 3>(a, p, stream);
    case kF16:
      return q.type == kF32 ? launch_dim<kF16, 2, 2>(a, p, stream)
                            : launch_dim<kF16, 1, 2>(a, p, stream);
    default:
      return q.type == kF32 ? launch_dim<kE4M3, 2, 2>(a, p, stream)
                            : launch_dim<kE4M3, 1, 2>(a, p, stream);
  }
}

}  // namespace xq
