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
//
// Measured: 4096 tokens, 32 heads of 128 dims on 8 kv heads, bf16: 168-196 us by
// card, 701-818 TFLOP/s (56-66% of a large library product's rate); of the
// cycles MFMA are busy in 37%, VALU in 46%, LDS in 55%, and a third of the waves'
// time is waits. The tile's ceiling is LDS: every wave reads the whole of K and V
// for its 32 rows, as many cycles as its matrix instructions take, and writes
// are a quarter on top. 8192 tokens with a window of 2048, f16: 323-341 us. What
// made it so: operands read ahead of
// the matrix instructions (256 -> 230 us with the lagging reference, 199 with
// both), wave priority over them (183). Few rows run elsewhere: chunk_in_rows.
//
// Precision: S, the softmax and O are f32; q enters in its own 16 bits, an
// 8-bit cache is widened exactly; p is rounded to 16 bits, as the product
// needs (bf16 to 2^-8; f16 to 2^-11 down to 2^-26 of the row's maximum).
#include <algorithm>
#include <cmath>
#include <type_traits>

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
  uint32_t k_page16, k_tok16, v_page16, v_tok16;  // in 16-byte units
  int flip;       // q's sign is turned, for a negative scale
  int zero;       // q counts as 0, for a scale of 0 (c is 1 then: -infinity hides a score only if c > 0)
  float c;        // |scale| * k_scale * log2(e)
  float v_scale;
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
  // (clang's bit cast of a vector's element reads the vector's start: that of
  // s[1] itself would be s[0]'s.)
  const uint32_t x = s[0], y = s[1];
  return f32x2{__builtin_bit_cast(float, x), __builtin_bit_cast(float, y)};
}
__device__ __forceinline__ float halves_max(float v) {
  const f32x2 s = both_halves(v);
  return fmaxf(s.x, s.y);
}
// Bits 0 .. n-1.
__device__ __forceinline__ uint64_t below(int n) {
  return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1;
}
// The largest of 16, or NaN if there is one: v_maximum3_f32. (fmaxf, which
// drops NaN, would quiet each value first.)
__device__ __forceinline__ float max16(f32x16 x) {
  float r = x[0];
#pragma unroll
  for (int i = 1; i < 15; i += 2)
    r = __builtin_elementwise_maximum(__builtin_elementwise_maximum(x[i], x[i + 1]), r);
  return __builtin_elementwise_maximum(r, x[15]);
}
__device__ __forceinline__ float halves_sum(float v) {
  const f32x2 s = both_halves(v);
  return s.x + s.y;
}

// MT: q's and out's type. CT: the cache's, MT or kE4M3. DP: dim rounded up to
// 64, 96, 128, 192 or 256; FULL: dim is DP.
template <int MT, int CT, int DP, bool FULL>
__global__ __launch_bounds__(kThreads, DP <= 128 ? 2 : 1) void attn_prefill_kernel(PrefillArgs a) {
  constexpr int EB = CT == kE4M3 ? 1 : 2;
  // Bytes of a row in LDS. A row of K begins 4 banks past the one before, so 8
  // rows of a 16-byte column hit 32 banks; a row of V 8 banks (of 32 mod 128
  // bytes), so the 4 rows x 32 bytes of a transposing load do.
  constexpr int KB = DP * 2 + 16, VB = DP * 2 + 32;
  constexpr int STAGE = kTile * (KB + VB);
  constexpr int CH = DP / 8;                 // 8-dim pieces of a row
  constexpr int PER = kTile * CH / kThreads; // of a thread, K and V each
  constexpr int DT = DP / 32;
  constexpr uint32_t kInf2 = MT == kBF16 ? 0x7f80u : 0x7c00u;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ uint32_t places[3][2][kTile];   // of a tile's tokens in k and v, in 16-byte units
  __shared__ uint64_t found[3];              // bit t: token t of the tile is there
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
  const int end = a.starts[seq + 1];
  const int count = min(min(max(end, first), a.rows) - first, a.max_chunk);
  const int group = a.group.d;
  const int row0 = tile * kRows;
  if (row0 >= count * group) return;
  const int n = static_cast<int>(min(static_cast<int64_t>(max(0, a.lens[seq])), a.table_tokens));
  // Position of row first + t: the chunk's last row, whether it is done or left
  // out, is the sequence's last token. One below 0 sees nothing. (end > first
  // >= 0 here, so nothing leaves 32 bits; 64 would leave the scalar unit.)
  const int base = n - (end - first);
  auto position = [&](int t) { return max(base + t, -1); };

  // This lane's row.
  const int r = row0 + wave * 32 + l32;
  const bool mine = r < count * group;
  const int tok = mine ? div_by(r, a.group) : 0;
  const int head = kvh * group + (r - tok * group);
  const int pos = mine ? position(tok) : -1;
  const int from = a.window ? pos - a.window : -1;  // sees j > from, or j < sinks
  const int sinks = a.window ? a.sinks : 0;

  // The workgroup's tokens: the sinks' tiles, then those from `lo` on.
  const int pmin = position(div_by(row0, a.group));
  const int pmax = position(div_by(min(row0 + kRows, count * group) - 1, a.group));
  const int lo = a.window ? max(0, pmin - a.window + 1) / kTile * kTile : 0;
  const int ns = min(sinks, lo);
  const int sink_tiles = (ns + kTile - 1) / kTile;
  const int tiles = sink_tiles + (pmax + 1 > lo ? (pmax + 1 - lo + kTile - 1) / kTile : 0);
  auto tile_begin = [&](int t) { return t < sink_tiles ? t * kTile : lo + (t - sink_tiles) * kTile; };
  auto tile_end = [&](int t) { return t < sink_tiles ? min(ns, (t + 1) * kTile) : min(pmax + 1, tile_begin(t) + kTile); };

  u32x4 qf[DP / 16];
  {
    const uint8_t* qr = a.q + (first + tok) * a.q_row + head * a.q_head;
    const bool reads = mine && !a.zero;
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) {
      const int d0 = s * 16 + lh * 8;
      qf[s] = u32x4{0, 0, 0, 0};
      if (reads && (FULL || d0 < a.dim)) qf[s] = *reinterpret_cast<const u32x4*>(qr + d0 * 2);
      if (a.flip) qf[s] ^= u32x4{0x80008000u, 0x80008000u, 0x80008000u, 0x80008000u};
    }
  }

  const uint8_t* kb = a.kv.k + kvh * a.kv.k_head;
  const uint8_t* vb = a.kv.v + kvh * a.kv.v_head;
  const int32_t* table = a.tables + seq * a.table_stride;
  // The first wave looks up a tile's tokens. One that is not there reads the
  // start of page 0, which always is; its score is hidden.
  auto page_of = [&](int t) {
    const int j = tile_begin(t) + lane;
    const bool in = t < tiles && j < tile_end(t);
    const int page = table[in ? div_by(j, a.kv.page) : 0];
    return in ? page : -1;
  };
  auto place = [&](int t, int page) {
    const uint32_t j = tile_begin(t) + lane;
    const bool ok = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.kv.pages);
    const uint32_t slot = j - div_by(j, a.kv.page) * a.kv.page.d;
    places[t % 3][0][lane] = ok ? page * a.k_page16 + slot * a.k_tok16 : 0;
    places[t % 3][1][lane] = ok ? page * a.v_page16 + slot * a.v_tok16 : 0;
    const uint64_t all = __ballot(ok);
    if (lane == 0) found[t % 3] = all;
  };
  using Raw = std::conditional_t<EB == 2, u32x4, u32x2>;
  Raw kr[PER], vr[PER];
  auto load = [&](int t) {
    uint32_t at[2][PER];
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int i = 0; i < PER; ++i) at[w][i] = places[t % 3][w][(tid + i * kThreads) / CH];
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int d0 = (tid + i * kThreads) % CH * 8;
        const uint8_t* p = (w ? vb : kb) + static_cast<uint64_t>(at[w][i]) * 16 +
                           (FULL || d0 < a.dim ? d0 : 0) * EB;
        (w ? vr[i] : kr[i]) = *reinterpret_cast<const Raw*>(p);
      }
  };
  auto widen = [&](Raw w) {
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
    uint8_t* kl = smem + (t % 2) * STAGE;
    uint8_t* vl = kl + kTile * KB;
    const bool masked = !plain_tile(t) || found[t % 3] != ~0ull;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = tid + i * kThreads, row = at / CH, c = at % CH;
      u32x4 w = widen(kr[i]);
      // q is 0 past the end, but 0 * infinity is not.
      if (!FULL && c * 8 >= a.dim) w = u32x4{0, 0, 0, 0};
      *reinterpret_cast<u32x4*>(kl + row * KB + c * 16) = w;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = tid + i * kThreads, row = at / CH, c = at % CH;
      u32x4 w = widen(vr[i]);
      if (masked) {
        // 0 * infinity must not reach a row that does not see the token: such
        // values are left out here and added to the rows that do.
        bool any = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool x = (w[e] & kInf2) == kInf2, y = ((w[e] >> 16) & kInf2) == kInf2;
          any |= x || y;
          w[e] &= (x ? 0u : 0xffffu) | (y ? 0u : 0xffff0000u);
        }
        if (any) odd[t % 3] = 1;
      }
      *reinterpret_cast<u32x4*>(vl + row * VB + c * 16) = w;
      // (Widened one after the other: registers are short.)
      if constexpr (EB == 1) __builtin_amdgcn_sched_barrier(0);
    }
  };

  f32x16 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  // Weights are exp2(c s - ref). A new ref makes the row's maximum so far weigh
  // 2^kLift, and stays until one weighs over 2^(kLift + kLag): the f32 sums do
  // not mind, and are seldom rescaled. `limit` is the score that ends a ref,
  // -infinity before the row's first token. In f16 the lift keeps small weights'
  // bits: none is above 2^15, and those down to 2^-26 of the row's maximum are
  // normal numbers. (Without it 131072 tokens of 2^-26 each, 2^-9 of the sum,
  // added nothing to the product.)
  constexpr float kLag = MT == kF16 ? 3.f : 8.f, kLift = MT == kF16 ? 12.f : 0.f;
  float ref = 0.f, limit = -INFINITY, l = 0.f;

  if (tid < 3) odd[tid] = 0;
  if (wave == 0) {
    place(0, page_of(0));
    place(1, page_of(1));
  }
  __syncthreads();
  if (tiles > 0) {
    load(0);
    put(0);
  }
  __syncthreads();

  for (int t = 0; t < tiles; ++t) {
    int page = -1;
    if (wave == 0) page = page_of(t + 2);
    if (tid == 0) odd[(t + 2) % 3] = 0;  // last read before the barrier, next set after the coming one
    load(t + 1 < tiles ? t + 1 : t);
    const uint8_t* kl = smem + (t % 2) * STAGE;
    const uint8_t* vl = kl + kTile * KB;

    f32x16 st[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 16; ++i) st[h][i] = 0.f;
    // K goes through registers GS steps of 16 dims at a time, the next group's
    // reads under way while one is worked on. (The fences keep that order; left
    // to itself the compiler waits for each read.)
    constexpr int GS = 2, GN = DP / 16 / GS;
    u32x4 kf[2][GS][2];
    auto read_k = [&](int g) {
#pragma unroll
      for (int s = 0; s < GS; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          kf[g % 2][s][h] = *reinterpret_cast<const u32x4*>(
              kl + (h * 32 + l32) * KB + ((g * GS + s) * 16 + lh * 8) * 2);
    };
    __builtin_amdgcn_s_setprio(1);
    read_k(0);
#pragma unroll
    for (int g = 0; g < GN; ++g) {
      if (g + 1 < GN) read_k(g + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int s = 0; s < GS; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) st[h] = mfma32<MT>(kf[g % 2][s][h], qf[g * GS + s], st[h]);
      __builtin_amdgcn_sched_barrier(0);
    }
    // V's operands for 16 tokens, read 16 tokens ahead.
    u32x4 vf[2][DT];
    auto read_v = [&](int s) {
      const uint8_t* vp = vl + (16 * s + 4 * lh + (lane % 16) / 4) * VB +
                          (16 * ((lane / 16) % 2) + (lane % 4) * 4) * 2;
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const u32x2 x = load_transposed(vp + d * 64), y = load_transposed(vp + 8 * VB + d * 64);
        vf[s % 2][d] = u32x4{x.x, x.y, y.x, y.y};
      }
    };
    read_v(0);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(0);

    // A tile whose pages are all there and that every row sees needs no mask.
    const int b = tile_begin(t), e = tile_end(t);
    const uint64_t there = found[t % 3];
    // Else bit k of `vis` says whether the lane's row sees the tile's token k.
    uint64_t vis = ~0ull;
    if (!plain_tile(t) || there != ~0ull) {
      vis = there & below(min(pos + 1, e) - b) & (~below(from + 1 - b) | below(sinks - b));
      const uint64_t mine = vis >> (4 * lh);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t bits = static_cast<uint32_t>(mine >> (32 * h));
        // A select, not a branch: set under a branch of several conditions,
        // element 0 of a vector went wrong in the compiler's back end (the block
        // that sets it came out empty; its store had moved ahead of a copy that
        // undid it), and tokens 0 and 4 of a tile stayed visible.
#pragma unroll
        for (int i = 0; i < 16; ++i) st[h][i] = bits & (1u << (8 * (i / 4) + i % 4)) ? st[h][i] : -INFINITY;
      }
    }
    const float top = halves_max(fmaxf(max16(st[0]), max16(st[1]))) * a.c;
    if (__ballot(top > limit)) {
      const float to = top > limit ? top - kLift : ref;
      const float alpha = limit == -INFINITY ? 0.f : exp2_fast(ref - to);
      if (top > limit) {
        ref = to;
        limit = top + kLag;
      }
      l *= alpha;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= alpha;
    }
    // The weights of 16 tokens are formed while the matrix instructions of the
    // 16 before run.
    float sums[4] = {0.f, 0.f, 0.f, 0.f};
    u32x4 pf[2];
    auto weigh = [&](int s) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const int k = (s % 2) * 8 + i;
        const float x = exp2_fast(fmaf(st[s / 2][k], a.c, -ref));
        const float y = exp2_fast(fmaf(st[s / 2][k + 1], a.c, -ref));
        sums[i / 2] += x + y;
        // (Here, beside the matrix instructions, not after them all.)
        asm volatile("" : "+v"(sums[i / 2]));
        pf[s % 2][i / 2] = pack2<MT>(x, y);
      }
    };
    weigh(0);
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s < 3) read_v(s + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] = mfma32<MT>(vf[s % 2][d], pf[s % 2], o[d]);
      if (s < 3) {
        weigh(s + 1);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x402, (28 + DT - 1) / DT, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_setprio(0);
    l += (sums[0] + sums[1]) + (sums[2] + sums[3]);
    if (odd[t % 3]) {
      // Infinities and NaN of this tile, for the rows that see them. (What the
      // compiler knows of this lane's dims it would work out ahead of the loop
      // over tiles, and keep in registers that there are none of.)
      int first_dim = 4 * lh;
      asm volatile("" : "+v"(first_dim));
#pragma unroll 1
      for (int k = 0; k < kTile; ++k) {
        if (!((there >> k) & 1)) continue;
        const uint8_t* row = vb + static_cast<int64_t>(places[t % 3][1][k]) * 16;
        const bool sees = (vis >> k) & 1;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const int dim = d * 32 + 8 * (i / 4) + first_dim;
            const uint8_t* p = row + (FULL || dim < a.dim ? dim : 0) * EB;
            u32x2 w;
            if constexpr (EB == 2) w = *reinterpret_cast<const u32x2*>(p);
            else w = widen4<MT>(*reinterpret_cast<const uint32_t*>(p));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const f32x2 pair = unpack2<MT>(w[e / 2]);
              const float x = e % 2 ? pair.y : pair.x;
              o[d][i + e] += sees && !(fabsf(x) < INFINITY) ? x : 0.f;
            }
            __builtin_amdgcn_sched_barrier(0);  // few loads under way: registers are short
          }
      }
    }

    if (t + 1 < tiles) put(t + 1);
    if (wave == 0) place(t + 2, page);
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

template <int MT, int CT, int DP, bool FULL>
hipError_t launch(const PrefillArgs& a, uint32_t blocks, hipStream_t stream) {
  constexpr int lds = 2 * kTile * (2 * DP * 2 + 48);
  auto kernel = attn_prefill_kernel<MT, CT, DP, FULL>;
  if (lds > 48 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  kernel<<<dim3(blocks), dim3(kThreads), lds, stream>>>(a);
  return hipGetLastError();
}

template <int MT, int CT, int DP>
hipError_t launch_full(const PrefillArgs& a, uint32_t blocks, hipStream_t stream) {
  return a.dim == DP ? launch<MT, CT, DP, true>(a, blocks, stream)
                     : launch<MT, CT, DP, false>(a, blocks, stream);
}

template <int MT, int CT>
hipError_t launch_dim(const PrefillArgs& a, uint32_t blocks, hipStream_t stream) {
  if (a.dim <= 64) return launch_full<MT, CT, 64>(a, blocks, stream);
  if (a.dim <= 96) return launch_full<MT, CT, 96>(a, blocks, stream);
  if (a.dim <= 128) return launch_full<MT, CT, 128>(a, blocks, stream);
  if (a.dim <= 192) return launch_full<MT, CT, 192>(a, blocks, stream);
  return launch_full<MT, CT, 256>(a, blocks, stream);
}

}  // namespace

int64_t attn_prefill_blocks(int64_t seqs, int64_t heads, const xq_kv& kv, int64_t max_chunk) {
  return seqs * kv.kv_heads * row_tiles(heads, kv, max_chunk);
}

hipError_t launch_attn_prefill(const RowsView& out, const RowsView& q, int64_t rows, int64_t seqs,
                               int64_t heads, const xq_kv& kv, const TableView& tables,
                               const int32_t* lens, const int32_t* starts, int64_t max_chunk,
                               float scale, int64_t window, int64_t sinks, hipStream_t stream) {
  if (chunk_in_rows(seqs, heads, kv, max_chunk))
    return launch_attn_chunk(out, q, rows, seqs, heads, kv, tables, lens, starts, max_chunk, scale, window, sinks,
                             stream);
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
  a.k_page16 = static_cast<uint32_t>(a.kv.k_page / 16);
  a.k_tok16 = static_cast<uint32_t>(a.kv.k_tok / 16);
  a.v_page16 = static_cast<uint32_t>(a.kv.v_page / 16);
  a.v_tok16 = static_cast<uint32_t>(a.kv.v_tok / 16);
  a.flip = scale < 0.f;
  a.c = std::fabs(scale) * kv.k_scale * kLog2e;
  a.zero = a.c == 0.f;
  if (a.zero) a.c = 1.f;
  a.v_scale = kv.v_scale;
  const uint32_t blocks = static_cast<uint32_t>(attn_prefill_blocks(seqs, heads, kv, max_chunk));
  if (q.type == kBF16)
    return kv.dtype == kBF16 ? launch_dim<kBF16, kBF16>(a, blocks, stream)
                             : launch_dim<kBF16, kE4M3>(a, blocks, stream);
  return kv.dtype == kF16 ? launch_dim<kF16, kF16>(a, blocks, stream)
                          : launch_dim<kF16, kE4M3>(a, blocks, stream);
}

}  // namespace xq
