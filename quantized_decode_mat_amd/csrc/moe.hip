// moe.hip — a mixture-of-experts layer for a few tokens: the router, and the
// chosen experts' feed-forward on Q4_K weights.
//
//   logits = R x;  ids, weights: the `used` highest of their scores
//   h[t,k] = silu(G_e x^) * (U_e x^),  x^ = q8_K(x),  e = ids[t][k]
//   y[t]   = sum_k weights[t][k] * (D_e q8_K(h[t,k]))
//
// What bounds it: the chosen experts' bytes, each read once; for one token the
// launches beside them (tens of MB are 6 us). So a token's layer is two launches:
// gate and up with the product of their results, then down with the sum over the
// slots. Each workgroup of the first quantizes x for itself, and each of the
// second the h that it needs, while its first weights are on their way. Where
// many tokens share experts the work is an expert's: the pairs (token, slot) that
// chose it share one pass over its rows.
//
// A row's dot is the mat-vec's (q4k_row.h): four lanes a super-block. Rows of
// at most 8 or 4 blocks take a half or a quarter of a wave, which then holds
// two or four rows, gate's and up's next to each other.
//
// Measured, router and experts together: one token, 8 of 64 experts, 2048 x 1536:
// 21.8 us (43 MB; 5.9 at a streaming read's rate); five tokens, 6 of 64, 2048 x
// 1280: 38.8 (110 MB, 15); 16 tokens, 2 of 8, 4096 x 14336: 202 to 217 us by card
// (785 MB, 108).
//
// Precision: the products are whole numbers up to the scales, sums over blocks
// and slots f32. The activations go to q8_K twice, as the mat-vecs' do; h stays
// f32 in between.
#include <algorithm>

#include "kv_device.h"
#include "moe_launch.h"
#include "q4k_row.h"
#include "q8k_block.h"
#include "xq_launch.h"

namespace xq {
namespace {

constexpr int kWaitVm0 = 0x0f70;  // s_waitcnt vmcnt(0), others untouched
constexpr size_t kCounterRegion = 96 * 1024;
constexpr int kCounterStride = 32;  // ints: a 128-byte line

__device__ __forceinline__ float4 load_x4(const uint8_t* row, int type, int at) {
  if (type == kF32) return *reinterpret_cast<const float4*>(row + at * 4);
  const u32x2 w = *reinterpret_cast<const u32x2*>(row + at * 2);
  const f32x2 a = type == kBF16 ? unpack2<kBF16>(w.x) : unpack2<kF16>(w.x);
  const f32x2 b = type == kBF16 ? unpack2<kBF16>(w.y) : unpack2<kF16>(w.y);
  return make_float4(a.x, a.y, b.x, b.y);
}

// ---------------------------------------------------------------- router

constexpr int kRouteThreads = 512;
constexpr int kRouteWaves = kRouteThreads / kWave;
constexpr int kRouteExperts = 4;  // of a workgroup

struct RouteArgs {
  const uint8_t* x;
  const uint8_t* router;
  const float* bias;
  int32_t* ids;
  float* weights;
  float* logits;   // workspace, [tokens][experts]
  int32_t* count;  // an arrival counter for each tile of tokens
  int64_t x_row;   // bytes
  int x_type, router_type, tokens, experts, used, k, expert_tiles, sigmoid, normalize;
  float scale;
};

__device__ __forceinline__ int wave_max_int(int v) {
  v = max(v, dpp<kDppQuadSwap1>(v));
  v = max(v, dpp<kDppQuadSwap2>(v));
  v = max(v, dpp<kDppRowHalfMirror>(v));
  v = max(v, dpp<kDppRowMirror>(v));
  return max(max(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16)),
             max(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48)));
}

// Whole numbers in the order of the floats; NaN below all of them.
constexpr int kAbsent = -2147483647 - 1;
__device__ __forceinline__ int ordered(float v) {
  if (v != v) return kAbsent + 1;
  v += 0.f;  // -0 is 0
  const int b = __builtin_bit_cast(int, v);
  return b < 0 ? static_cast<int>(0x80000000u - static_cast<uint32_t>(b)) : b;
}

struct Row8 {
  float v[8];
};
__device__ __forceinline__ Row8 load_x8(const uint8_t* row, int type, int at) {
  Row8 r;
  const float4 a = load_x4(row, type, at), b = load_x4(row, type, at + 4);
  r.v[0] = a.x, r.v[1] = a.y, r.v[2] = a.z, r.v[3] = a.w;
  r.v[4] = b.x, r.v[5] = b.y, r.v[6] = b.z, r.v[7] = b.w;
  return r;
}

// What bounds it is latency: one read of the router's rows (0.3 to 8 MB), the sums
// through LDS, an arrival, the ranking. Four experts a workgroup put 16 workgroups
// on 64 experts, whose x stays in registers for all four; 512 threads cover 4096
// columns at once. Measured: 64 experts of 2048 columns, one token 6.0 us, five
// tokens 8.9.
//
// A workgroup has four experts' rows against NT tokens; its waves share the
// columns, and LDS adds up their sums. The last workgroup of a tile of tokens to
// arrive ranks them, a wave a token: the highest key `used` times over, the
// lowest index among equals. PER: experts of a lane there.
template <int NT, int PER>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(RouteArgs a) {
  __shared__ float sums[kRouteWaves * 4][kRouteExperts * NT];
  __shared__ int last;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int tile = blockIdx.x / a.expert_tiles, e0 = blockIdx.x % a.expert_tiles * kRouteExperts;
  const int t0 = tile * NT, tokens = min(NT, a.tokens - t0);
  const int64_t r_row = static_cast<int64_t>(a.k) * (a.router_type == kF32 ? 4 : 2);
  float sum[kRouteExperts][NT] = {};
  for (int k = threadIdx.x * 8; k < a.k; k += kRouteThreads * 8) {
    Row8 r[kRouteExperts];
#pragma unroll
    for (int e = 0; e < kRouteExperts; ++e)
      r[e] = load_x8(a.router + min(e0 + e, a.experts - 1) * r_row, a.router_type, k);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const Row8 x = load_x8(a.x + (t0 + min(t, tokens - 1)) * a.x_row, a.x_type, k);
#pragma unroll
      for (int e = 0; e < kRouteExperts; ++e)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[e][t] = fmaf(r[e].v[i], x.v[i], sum[e][t]);
    }
  }
#pragma unroll
  for (int e = 0; e < kRouteExperts; ++e)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float v = row16_sum(sum[e][t]);
      if (lane % 16 == 0) sums[threadIdx.x / 16][e * NT + t] = v;
    }
  __syncthreads();
  if (threadIdx.x < kRouteExperts * NT) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kRouteWaves * 4; ++w) v += sums[w][threadIdx.x];
    const int e = e0 + threadIdx.x / NT, t = threadIdx.x % NT;
    if (e < a.experts && t < tokens)
      __hip_atomic_store(a.logits + static_cast<int64_t>(t0 + t) * a.experts + e, v, __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
  }
  __builtin_amdgcn_s_waitcnt(kWaitVm0);  // the logits are where all can see them
  __syncthreads();
  if (threadIdx.x == 0)
    last = __hip_atomic_fetch_add(a.count + tile * kCounterStride, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
           a.expert_tiles - 1;
  __syncthreads();
  if (!last) return;  // workgroup-uniform
  if (threadIdx.x == 0)
    __hip_atomic_store(a.count + tile * kCounterStride, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);

  for (int t = wave; t < tokens; t += kRouteWaves) {
    const float* logits = a.logits + static_cast<int64_t>(t0 + t) * a.experts;
    float score[PER];
    int key[PER];
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = j * kWave + lane;
      score[j] = e < a.experts ? __hip_atomic_load(logits + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : -INFINITY;
      top = fmaxf(top, score[j]);
    }
    float all = 1.f;
    if (!a.sigmoid) {
      top = wave_max(top);
      all = 0.f;
#pragma unroll
      for (int j = 0; j < PER; ++j) all += j * kWave + lane < a.experts ? expf(score[j] - top) : 0.f;
      all = wave_sum(all);
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = j * kWave + lane;
      const float logit = score[j];
      score[j] = a.sigmoid ? 1.f / (1.f + expf(-logit)) : expf(logit - top) / all;
      // (Softmax keeps the logits' order: without a bias they rank by those, also
      // where scores underflow or round to one. Sigmoid ranks by its scores.)
      const float rank = a.bias ? score[j] + (e < a.experts ? a.bias[e] : 0.f) : a.sigmoid ? score[j] : logit;
      key[j] = e < a.experts ? ordered(rank) : kAbsent;
    }
    int my_id = 0;
    float my_score = 0.f, chosen = 0.f;
    for (int k = 0; k < a.used; ++k) {
      int best = key[0], at = 0;
      float s = score[0];
#pragma unroll
      for (int j = 1; j < PER; ++j)
        if (key[j] > best) best = key[j], at = j, s = score[j];
      const int high = wave_max_int(best);
      // Of the lanes that have it the one with the lowest index.
      const uint64_t have = __ballot(best == high);
      int id = __builtin_ctzll(have);
      if constexpr (PER > 1) {
        if (have & (have - 1)) id = -wave_max_int(best == high ? -(at * kWave + lane) : kAbsent + 1);
        else id += __builtin_amdgcn_readlane(at, id) * kWave;
      }
      const float v = readlane(s, id % kWave);
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (j * kWave + lane == id) key[j] = kAbsent;
      if (lane == k) my_id = id, my_score = v;
      chosen += v;
    }
    if (lane < a.used) {
      const int64_t at = static_cast<int64_t>(t0 + t) * a.used + lane;
      a.ids[at] = my_id;
      a.weights[at] = (a.normalize ? (chosen == 0.f ? 0.f : my_score / chosen) : my_score) * a.scale;
    }
  }
}

// ---------------------------------------------------------------- experts

struct MoeArgs {
  const uint8_t* x;        // the rows that go in, of type x_type (or packed)
  int64_t x_row;           // bytes
  const float* xs;         // packed rows' scales, [rows][nb]
  const uint8_t* w[2];     // gate and up, or down
  const int32_t* ids;
  const float* weights;
  float* out;              // f32 [pairs][rows]
  uint8_t* y;
  int64_t y_row;           // bytes
  int type, x_type, tokens, used, experts, rows, nb;
  int by_pair;             // a row that goes in is a pair's, not a token's
  int groups;              // of rows, that a wave walks over
  FastDiv used_div, nb_div;
};

constexpr int kMaxPairs = 512;

// The pairs that chose pair `first`'s expert e, in order, into `list`; 0 if one
// before it did, whose workgroup then does the work. (By every wave alike; the
// list is wave 0's to write.)
__device__ __forceinline__ int pairs_of(const int32_t* ids, int pairs, int first, int e, uint16_t* list) {
  const int lane = threadIdx.x % kWave;
  int count = 0;
  for (int p = 0; p < pairs; p += kWave) {
    const uint64_t same = __ballot(p + lane < pairs && ids[min(p + lane, pairs - 1)] == e);
    if (p <= first) {
      const uint64_t before = p + kWave <= first ? ~0ull : (1ull << (first - p)) - 1;
      if (same & before) return 0;
    }
    if (threadIdx.x < kWave && (same >> lane & 1))
      list[count + __builtin_popcountll(same & ((1ull << lane) - 1))] = static_cast<uint16_t>(p + lane);
    count += __builtin_popcountll(same);
  }
  return count;
}

__device__ __forceinline__ float silu(float g) { return g / (1.f + expf(-g)); }

// ---- Few pairs an expert: mat-vecs.

// Rows of weights that a wave's lanes have in flight, and rows of h that they make.
constexpr int kUpSteps = 4;
constexpr int up_rows(int lpr) { return kUpSteps * (kWave / lpr) / 2; }

// Gate and up, and silu(gate) * up, of one pair. LPR: lanes of a row (nb <= LPR / 4
// where it is below 64). A workgroup has W waves, each `groups` times R rows of h
// of pair blockIdx.y.
//
// What bounds it: the weights' bytes, and with 10 to 25 KB a wave in all the start
// of that stream (ids, then the first weights; x is quantized meanwhile). Four
// rows of weights in flight hide it; nothing around the loads is conditional, so
// that the compiler lets them pass the dots before them. Pairs of one expert are
// not brought together: they run at the same time, a row's workgroup on the same
// XCD (the grid's width is a multiple of 8), whose L2 has the second one's reads.
// (Two pairs a pass, with two rows in flight, were slower but for none: the experts'
// call with 10 tokens, 6 of 64 experts of 2048 x 1280 67 -> 51 us, 16 tokens, 8 of
// 128 of 2048 x 768 81 -> 60, 4 tokens, 2 of 8 of 4096 x 14336 160 -> 137; without the
// multiple of 8 53, 62 and 143.) Measured: 8 pairs, 2 x 1536 rows of 2048 columns, 28
// MB: 8.0 to 9.9 us; 30 pairs, 2 x 1280 rows, 73 MB: 17.6, 4.2 TB/s.
template <int LPR, int W>
__global__ __launch_bounds__(W * kWave, 3) void moe_up_kernel(MoeArgs a) {
  constexpr int SEG = kWave / LPR;            // rows of weights of a wave at a time
  constexpr int STEPS = kUpSteps;
  constexpr int R = up_rows(LPR);
  constexpr int UB = LPR / 4;                 // blocks of a unit
  extern __shared__ __attribute__((aligned(16))) uint8_t act[];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int pair = blockIdx.y, from = blockIdx.x * a.groups * W * R;
  if (from >= a.rows) return;  // (the width's rounding)
  // x does not wait for the choice of experts. (Two blocks a wave; more than 8
  // blocks, 2048 columns, take another turn.)
  constexpr int XE = 2;
  const uint8_t* x = a.x + div_by(pair, a.used_div) * a.x_row;
  float4 xe[XE];
#pragma unroll
  for (int i = 0; i < XE; ++i) xe[i] = load_x4(x, a.x_type, min(wave + i * W, a.nb - 1) * 256 + lane * 4);
  const int e = a.ids[pair];
  if (e < 0 || e >= a.experts) return;

  const LaneGeom L = lane_geom(lane);
  const int seg = lane / LPR, bsub = lane % LPR / 4;
  const int first = from + wave * R;          // group g's rows begin at first + g * W * R
  const int64_t row_bytes = static_cast<int64_t>(a.nb) * kQ4KBytes;
  const int units = LPR < kWave ? 1 : (a.nb + UB - 1) / UB;
  auto load = [&](int g, int u, Nib(&n)[STEPS], uint4(&h)[STEPS]) {
    const int b = min(u * UB + bsub, a.nb - 1);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int item = s * SEG + seg, row = min(first + g * W * R + item / 2, a.rows - 1);
      const uint8_t* blk = (item % 2 ? a.w[1] : a.w[0]) +
                           (static_cast<int64_t>(e) * a.rows + row) * row_bytes + b * kQ4KBytes;
      n[s] = load_group(blk, L);
      h[s] = *reinterpret_cast<const uint4*>(blk);
    }
  };
  Nib n0[STEPS], n1[STEPS];
  uint4 h0[STEPS], h1[STEPS];
  load(0, 0, n0, h0);
#pragma unroll
  for (int i = 0; i < XE; ++i)
    if (wave + i * W < a.nb) q8k_block_wave<true>(xe[i], act + (wave + i * W) * kQ8KBytes, lane);
  for (int i = wave + XE * W; i < a.nb; i += W)
    q8k_block_wave<true>(load_x4(x, a.x_type, i * 256 + lane * 4), act + i * kQ8KBytes, lane);
  __syncthreads();

  float acc[STEPS] = {};
  auto add = [&](int u, const Nib(&n)[STEPS], const uint4(&h)[STEPS]) {
    const int bb = u * UB + bsub, b = min(bb, a.nb - 1);
    const TokenSlice t = token_slice(act, b, L);
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const float v = chunk_token_slice(chunk_decode(n[s], h[s], L), t);
      acc[s] += bb < a.nb ? v : 0.f;
    }
  };
  // A row's sum in the mat-vec's order, each to the lane that stores it.
  auto finish = [&](int g) {
    float mine = 0.f, up = 0.f, sums[STEPS * SEG];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const float v = row16_sum(acc[s]);
      acc[s] = 0.f;
      if constexpr (LPR == 64) {
        sums[s] = (readlane(v, 0) + readlane(v, 16)) + (readlane(v, 32) + readlane(v, 48));
      } else if constexpr (LPR == 32) {
        sums[s * 2] = readlane(v, 0) + readlane(v, 16);
        sums[s * 2 + 1] = readlane(v, 32) + readlane(v, 48);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) sums[s * 4 + i] = readlane(v, 16 * i);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mine = lane == r ? sums[2 * r] : mine;
      up = lane == r ? sums[2 * r + 1] : up;
    }
    mine = silu(mine) * up;
    const int row = first + g * W * R + lane;
    if (lane < R && row < a.rows) a.out[static_cast<int64_t>(pair) * a.rows + row] = mine;
  };
  // Groups of rows, and units of a row, one after the other; the next one's
  // weights are on their way while one is worked on.
  int g = 0, u = 0;
  auto step = [&](Nib(&n)[STEPS], uint4(&h)[STEPS], Nib(&nn)[STEPS], uint4(&hh)[STEPS]) {
    const int g1 = u + 1 < units ? g : g + 1, u1 = u + 1 < units ? u + 1 : 0;
    const bool more = g1 < a.groups && first + g1 * W * R < a.rows;  // wave-uniform
    if (more) load(g1, u1, nn, hh);
    add(u, n, h);
    if (u + 1 == units) finish(g);
    g = g1;
    u = u1;
    return more;
  };
  while (step(n0, h0, n1, h1) && step(n1, h1, n0, h0)) {
  }
}

// Down for a token by itself: a wave's row of y is one sum over the blocks of
// all its slots' rows, four lanes a block, 16 blocks at a time; `groups` rows one
// after the other. The workgroup quantizes the token's h, used * nb blocks, while
// its first weights load.
// PF: steps of 16 blocks under way, all of a row's up to four.
//
// What bounds it: for one token the chain ids -> weights and h -> codes -> LDS ahead
// of 14 MB; one row of all slots a wave keeps the sum over the slots in registers
// (no h of a pair is read twice, no partial sums to add). Measured: 2048 rows of
// 8 x 1536 columns, 14 MB: 8.2 us; five tokens, 6 x 1280: 14 us.
template <int W, int PF>
__global__ __launch_bounds__(W * kWave) void moe_down_kernel(MoeArgs a) {
  constexpr int QB = 3;     // blocks of a wave quantized side by side
  extern __shared__ __attribute__((aligned(16))) uint8_t act[];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int token = blockIdx.y;
  const LaneGeom L = lane_geom(lane);
  const int blocks = a.used * a.nb, steps = (blocks + kUnitBlocks - 1) / kUnitBlocks;
  const int batches = (steps + PF - 1) / PF;
  const int64_t row_bytes = static_cast<int64_t>(a.nb) * kQ4KBytes;
  struct Batch {
    Nib nib[PF];
    uint4 hdr[PF];
  };
  const int first = blockIdx.x * a.groups * W + wave;
  // A lane's blocks of a batch: which slot's, of which expert, its weight.
  int place[PF], expert[PF];
  float weight[PF];
  auto look_up = [&](int bt) {
#pragma unroll
    for (int p = 0; p < PF; ++p) {
      const int i = (bt * PF + p) * kUnitBlocks + L.bsub, k = div_by(min(i, blocks - 1), a.nb_div);
      const int e = a.ids[token * a.used + k];
      weight[p] = a.weights[token * a.used + k];
      expert[p] = i < blocks && e >= 0 && e < a.experts ? e : -1;
      place[p] = min(i, blocks - 1) - k * a.nb;
    }
  };
  auto load = [&](int row, Batch& b) {
#pragma unroll
    for (int p = 0; p < PF; ++p) {
      b.nib[p] = zero_group();
      b.hdr[p] = make_uint4(0, 0, 0, 0);
      if (expert[p] >= 0 && row < a.rows) {
        const uint8_t* blk = a.w[0] + (static_cast<int64_t>(expert[p]) * a.rows + row) * row_bytes + place[p] * kQ4KBytes;
        b.nib[p] = load_group(blk, L);
        b.hdr[p] = *reinterpret_cast<const uint4*>(blk);
      }
    }
  };
  look_up(0);
  Batch b0, b1;
  load(first, b0);
  const float* h = reinterpret_cast<const float*>(a.x) + static_cast<int64_t>(token) * blocks * 256;
  for (int i0 = wave; i0 < blocks; i0 += QB * W) {
    float4 v[QB];
    bool ok[QB];  // (the h of a slot that is left out was not written)
#pragma unroll
    for (int q = 0; q < QB; ++q) {
      const int i = min(i0 + q * W, blocks - 1), e = a.ids[token * a.used + div_by(i, a.nb_div)];
      ok[q] = i0 + q * W < blocks && e >= 0 && e < a.experts;
      v[q] = ok[q] ? *reinterpret_cast<const float4*>(h + i * 256 + lane * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int q = 0; q < QB; ++q)
      if (ok[q]) q8k_block_wave<true>(v[q], act + (i0 + q * W) * kQ8KBytes, lane);
  }
  __syncthreads();
  float acc = 0.f;
  auto add = [&](int bt, const Batch& b) {
#pragma unroll
    for (int p = 0; p < PF; ++p) {
      const int i = min((bt * PF + p) * kUnitBlocks + L.bsub, blocks - 1);
      const float v = unit_partial(b.nib[p], b.hdr[p], act, i, L);
      if (expert[p] >= 0) acc = fmaf(weight[p], v, acc);
    }
  };
  auto store = [&](int row) {
    const float sum = wave_sum(acc);
    acc = 0.f;
    if (lane == 0 && row < a.rows) store_from_f32(a.y + token * a.y_row, a.type, row, sum);
  };
  if (PF < 4 || batches == 1) {
    // The next row's weights load while one is worked on.
    for (int g = 0; g < a.groups; g += 2) {
      const int row = first + g * W;
      if (g + 1 < a.groups) load(row + W, b1);
      add(0, b0);
      store(row);
      if (g + 1 >= a.groups) break;
      if (g + 2 < a.groups) load(row + 2 * W, b0);
      add(0, b1);
      store(row + W);
    }
  } else {
    for (int g = 0; g < a.groups; ++g) {
      const int row = first + g * W;
      for (int bt = 0; bt < batches; ++bt) {
        if (g > 0 || bt > 0) {
          look_up(bt);
          load(row, b0);
        }
        add(bt, b0);
      }
      store(row);
    }
  }
}

// ---- Many pairs an expert: matrix instructions.
//
// 16 rows of weights against 16 pairs, a super-block at a time: a code times its
// sub-block's 6-bit scale is a whole number below 2^10, exact in f16, and so are
// the activation's codes, so the f16 instruction's f32 sums are the integer
// route's up to f32's rounding. Lane l has row l % 16 and nibble group l / 16 of
// the block, whose scales are then its own: 16 codes of a dword become eight f16
// pairs by or-ing a 2^10 over them (1024 + q, or 1024 + 16 q) and one fused
// multiply-add that takes it off again. The mins ride on a ninth instruction,
// against sums of eight codes. The pairs' rows come packed in that order.
//
// What bounds it: bytes, read once an expert whatever its pairs, and next to them
// the VALU work that widens a weight once per 16 pairs. (int8 instructions take
// the codes without widening, but their sums need a scale per 32 columns: more
// VALU work than this.) Measured, 16 tokens, 2 of 8 experts of 4096 x 14336: gate and
// up 528 MB 125 to 135 us, 4.1 TB/s; down 264 MB 65 to 72 us; packing 2 x 4.8, the
// sum over slots 4.7.

constexpr int kPackHalves = 288;               // of a block: 256 codes, 32 sums of eight
constexpr int kPackBytes = kPackHalves * 2;
constexpr int kPackRow = kPackBytes + 16;      // in LDS: 8 rows of 16-byte reads hit all banks
constexpr int kTileWaves = 4;
constexpr int kTilePairs = 16;
constexpr int kChunk = 2;                      // blocks between two barriers
// A wave's rows of weights of a chunk go through LDS: loaded as they lie, 18
// lanes a row next to each other, read back a lane a row. (Loaded a lane a row,
// four lanes of a quad touch four rows' cache lines in each of three loads: the
// loads alone took 124 us for 528 MB.)
constexpr int kRowBytes = kChunk * kQ4KBytes, kRowWords = kRowBytes / 16;
constexpr int kRowPitch = kRowBytes + 16;      // 8 rows of 16-byte reads hit all banks
constexpr int kRowLoads = (16 * kRowWords + kWave - 1) / kWave;

// Rows of any type to packed blocks and their scales, a wave a block. (A launch:
// 4.8 us for 16 rows of 4096 as for 32 of 14336.)
__global__ __launch_bounds__(256) void moe_pack_kernel(uint8_t* packed, float* scales, const uint8_t* x, int64_t x_row,
                                                       int type, FastDiv nb, int blocks) {
  const int i = blockIdx.x * 4 + threadIdx.x / kWave, lane = threadIdx.x % kWave;
  if (i >= blocks) return;
  const int row = div_by(i, nb), b = i - row * nb.d;
  const Q8KLane q = q8k_block_lane<true>(load_x4(x + row * x_row, type, b * 256 + lane * 4));
  auto code = [&](int k) { return static_cast<float>(static_cast<int8_t>(q.packed >> (8 * k))); };
  // Elements 4l .. 4l + 3 in the order 0, 2, 1, 3.
  uint8_t* out = packed + static_cast<int64_t>(i) * kPackBytes;
  reinterpret_cast<u32x2*>(out)[lane] = u32x2{pack2<kF16>(code(0), code(2)), pack2<kF16>(code(1), code(3))};
  float sum = (code(0) + code(1)) + (code(2) + code(3));
  sum += dppf<kDppQuadSwap1>(sum);
  if (lane % 2 == 0) reinterpret_cast<uint16_t*>(out + 512)[lane / 2] = static_cast<uint16_t>(pack2<kF16>(sum, 0.f));
  if (lane == 0) scales[i] = q.d;
}

// MATS 2: a wave's 16 rows of gate and of up; 1: of down.
template <int MATS>
__global__ __launch_bounds__(kTileWaves * kWave, 2) void moe_tile_kernel(MoeArgs a) {
  constexpr int kThreads = kTileWaves * kWave;
  constexpr int kWords = kPackBytes / 16;                                     // 16-byte words of a packed block
  constexpr int kPer = (kTilePairs * kChunk * kWords + kThreads - 1) / kThreads;
  __shared__ __attribute__((aligned(16))) uint8_t act[2][kChunk][kTilePairs * kPackRow];
  __shared__ __attribute__((aligned(16))) uint8_t rows[kTileWaves][MATS][16 * kRowPitch];
  __shared__ __attribute__((aligned(16))) float scale[2][kChunk][kTilePairs];
  __shared__ uint16_t members[kMaxPairs];
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, l16 = lane % 16, lg = lane / 16;
  const int pair = blockIdx.y;
  const int e = a.ids[pair];
  if (e < 0 || e >= a.experts) return;
  const int count = pairs_of(a.ids, a.tokens * a.used, pair, e, members);
  if (count == 0) return;  // workgroup-uniform
  const LaneGeom L{0, lg, lg >= 2 ? ~0u : 0u, 16 * (lg & 1)};
  const int row0 = (blockIdx.x * kTileWaves + wave) * 16;
  const int row_bytes = a.nb * kQ4KBytes;
  const int64_t rows_at = (static_cast<int64_t>(e) * a.rows + min(row0, a.rows - 1)) * row_bytes;
  const int chunks = (a.nb + kChunk - 1) / kChunk;
  // This lane's words of the wave's rows: word i is row i / kRowWords's. Rows past
  // the matrix's last are that one again, words past a row's end its last.
  uint32_t word_from[kRowLoads], word_in[kRowLoads], word_to[kRowLoads];
#pragma unroll
  for (int j = 0; j < kRowLoads; ++j) {
    const int i = min(lane + j * kWave, 16 * kRowWords - 1), r = i / kRowWords;
    word_in[j] = i % kRowWords * 16;
    word_from[j] = max(min(r, a.rows - 1 - row0), 0) * row_bytes;
    word_to[j] = r * kRowPitch + word_in[j];
  }
  u32x4 raw[MATS][kRowLoads];
  auto load = [&](int c) {
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
      for (int j = 0; j < kRowLoads; ++j) {
        const uint32_t in = min(static_cast<uint32_t>(c * kRowBytes) + word_in[j], static_cast<uint32_t>(row_bytes - 16));
        raw[m][j] = *reinterpret_cast<const u32x4*>(a.w[m] + rows_at + (word_from[j] + in));
      }
  };
  auto lay_out = [&]() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
      for (int j = 0; j < kRowLoads; ++j) *reinterpret_cast<u32x4*>(&rows[wave][m][word_to[j]]) = raw[m][j];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
  };
  for (int m0 = 0; m0 < count; m0 += kTilePairs) {
    const int here = min(kTilePairs, count - m0);
    load(0);
    __syncthreads();  // the members are listed; the pass before is done with the activations
    // A thread's words of a chunk: word i is pair i / kChunk / kWords's. Nothing
    // here is conditional, so that the compiler knows how many loads are under
    // way: past the last word it is that one again, past the last chunk too. (Rows of
    // pairs past the last stay as they are; what they give nothing reads. The
    // block after a row of an odd number is the workspace's, and not used.)
    const int words = here * kChunk * kWords;
    auto row_of = [&](int t) {
      const int p = members[m0 + t];
      return static_cast<uint32_t>((a.by_pair ? p : static_cast<int>(div_by(p, a.used_div))) * a.nb);
    };
    uint32_t from[kPer], to[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = min(tid + j * kThreads, words - 1);
      const int t = i / (kChunk * kWords), r = i % (kChunk * kWords);
      from[j] = row_of(t) * kPackBytes + r * 16;
      to[j] = (r / kWords * kTilePairs + t) * kPackRow + r % kWords * 16;
    }
    const int mine = min(tid, here * kChunk - 1);
    const uint32_t scale_from = row_of(mine / kChunk) + mine % kChunk;
    u32x4 st[kPer];
    float ss;
    auto fetch = [&](int c) {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        st[j] = *reinterpret_cast<const u32x4*>(a.x + (from[j] + static_cast<uint32_t>(c * kChunk * kPackBytes)));
      ss = a.xs[scale_from + c * kChunk];
    };
    auto put = [&](int c) {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        *reinterpret_cast<u32x4*>(act[c % 2][0] + to[j]) = st[j];
      scale[c % 2][mine % kChunk][mine / kChunk] = ss;
    };
    fetch(0);
    put(0);
    __syncthreads();

    f32x4 total[MATS];
#pragma unroll
    for (int m = 0; m < MATS; ++m) total[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto add = [&](int c) {
#pragma unroll
      for (int k = 0; k < kChunk; ++k) {
        if (c * kChunk + k >= a.nb) break;  // workgroup-uniform
        const uint8_t* x = &act[c % 2][k][l16 * kPackRow + lg * 128];
        f32x4 s[MATS], low[MATS];
        u32x4 sc[MATS];  // pairs of f16: the scales, and what takes the 2^10 off, of low and high nibbles
        ChunkDecode d[MATS];
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
          s[m] = low[m] = f32x4{0.f, 0.f, 0.f, 0.f};
          const uint8_t* blk = &rows[wave][m][l16 * kRowPitch + k * kQ4KBytes];
          d[m] = chunk_decode(load_group(blk, L), *reinterpret_cast<const uint4*>(blk), L);
          const float s0 = static_cast<float>(d[m].sc0), s1 = static_cast<float>(d[m].sc1);
          sc[m] = u32x4{pack2<kF16>(s0, s0), pack2<kF16>(-1024.f * s0, -1024.f * s0),
                        pack2<kF16>(s1 * 0.0625f, s1 * 0.0625f), pack2<kF16>(-64.f * s1, -64.f * s1)};
          const float m0f = static_cast<float>(d[m].m0), m1f = static_cast<float>(d[m].m1);
          const uint32_t p0 = pack2<kF16>(m0f, m0f), p1 = pack2<kF16>(m1f, m1f);
          const u32x4 sums = *reinterpret_cast<const u32x4*>(&act[c % 2][k][l16 * kPackRow + 512 + lg * 16]);
          low[m] = mfma16<kF16>(sums, u32x4{p0, p0, p1, p1}, low[m]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const u32x4 xf = *reinterpret_cast<const u32x4*>(x + j * 16);
#pragma unroll
          for (int m = 0; m < MATS; ++m) {
            const uint4 q4 = j % 4 < 2 ? d[m].nib.a : d[m].nib.b;
            const uint32_t q0 = j % 2 ? q4.z : q4.x, q1 = j % 2 ? q4.w : q4.y;
            const uint32_t mask = j < 4 ? 0x000f000fu : 0x00f000f0u;
            const f16x2 mul = __builtin_bit_cast(f16x2, j < 4 ? sc[m].x : sc[m].z);
            const f16x2 off = __builtin_bit_cast(f16x2, j < 4 ? sc[m].y : sc[m].w);
            auto pairs = [&](uint32_t q) {
              const f16x2 v = __builtin_bit_cast(f16x2, (q & mask) | 0x64006400u);
              return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(v, mul, off));
            };
            s[m] = mfma16<kF16>(xf, u32x4{pairs(q0), pairs(q0 >> 8), pairs(q1), pairs(q1 >> 8)}, s[m]);
          }
        }
        const f32x4 xs = *reinterpret_cast<const f32x4*>(&scale[c % 2][k][lg * 4]);
#pragma unroll
        for (int m = 0; m < MATS; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            total[m][i] = fmaf(xs[i], fmaf(-d[m].dmin, low[m][i], d[m].d * s[m][i]), total[m][i]);
      }
    };
    // The next chunk's loads are under way while one is worked on.
    for (int c = 0; c < chunks; ++c) {
      const int after = min(c + 1, chunks - 1);
      lay_out();
      fetch(after);
      load(after);
      add(c);
      put(c + 1);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = lg * 4 + i;
      float v = total[0][i];
      if constexpr (MATS == 2) v = silu(v) * total[1][i];
      if (t < here && row0 + l16 < a.rows) a.out[static_cast<int64_t>(members[m0 + t]) * a.rows + row0 + l16] = v;
    }
  }
}

// y[t] = sum over its slots of weight * (down's row of the pair), in the slots'
// order whichever workgroup wrote them: no atomics. 16 x 4096 of 2 slots: 4.7 us.
__global__ __launch_bounds__(256) void moe_sum_kernel(MoeArgs a) {
  const int row = blockIdx.x * 256 + threadIdx.x, token = blockIdx.y;
  if (row >= a.rows) return;
  float sum = 0.f;
  for (int k = 0; k < a.used; ++k) {
    const int64_t p = static_cast<int64_t>(token) * a.used + k;
    const int e = a.ids[p];
    if (e >= 0 && e < a.experts) sum = fmaf(a.weights[p], a.out[p * a.rows + row], sum);
  }
  store_from_f32(a.y + token * a.y_row, a.type, row, sum);
}

template <int LPR>
hipError_t launch_up(MoeArgs a, hipStream_t stream) {
  constexpr int W = 4, R = up_rows(LPR);
  const size_t lds = static_cast<size_t>(a.nb) * kQ8KBytes;  // (of 128 blocks at most, 40 KiB)
  const int64_t pairs = static_cast<int64_t>(a.tokens) * a.used;
  // So many groups a wave that all workgroups are on the card at once, three a CU,
  // or two where the busiest CU has less to do then: five tokens, 6 of 64 experts
  // of 2048 x 1280, are 600 workgroups of 4 groups or 480 of 5, 33.5 and 30.3 us.
  const int64_t tiles = (a.rows + W * R - 1) / (W * R);
  int64_t blocks = 0, least = 0;
  for (int64_t per_cu = 3; per_cu >= 2; --per_cu) {
    const int64_t room = std::max<int64_t>(8, 256 * per_cu / pairs / 8 * 8), groups = (tiles + room - 1) / room;
    const int64_t used = (tiles + groups - 1) / groups, busiest = groups * ((used * pairs + 255) / 256);
    if (blocks && busiest >= least) continue;
    least = busiest;
    a.groups = static_cast<int>(groups);
    blocks = (used + 7) / 8 * 8;
  }
  moe_up_kernel<LPR, W><<<dim3(static_cast<uint32_t>(blocks), static_cast<uint32_t>(pairs)), dim3(W * kWave), lds, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_up_of(const MoeArgs& a, hipStream_t stream) {
  if (a.nb <= 4) return launch_up<16>(a, stream);
  if (a.nb <= 8) return launch_up<32>(a, stream);
  return launch_up<64>(a, stream);
}

template <int MATS>
hipError_t launch_tiles(const MoeArgs& a, hipStream_t stream) {
  const int64_t blocks = (a.rows + 16 * kTileWaves - 1) / (16 * kTileWaves);
  moe_tile_kernel<MATS><<<dim3(static_cast<uint32_t>(blocks), static_cast<uint32_t>(a.tokens * a.used)),
                          dim3(kTileWaves * kWave), 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_pack(uint8_t* packed, float* scales, const uint8_t* x, int64_t x_row, int type, int64_t rows, int64_t nb,
                       hipStream_t stream) {
  const int64_t blocks = rows * nb;
  moe_pack_kernel<<<dim3(static_cast<uint32_t>((blocks + 3) / 4)), dim3(256), 0, stream>>>(
      packed, scales, x, x_row, type, fast_div(static_cast<uint32_t>(nb)), static_cast<int>(blocks));
  return hipGetLastError();
}

constexpr int kDownWaves = 8;
constexpr int kMostDownLds = 80 * 1024;  // two workgroups a CU
template <int PF>
hipError_t launch_down(MoeArgs a, hipStream_t stream) {
  const size_t lds = static_cast<size_t>(a.used) * a.nb * kQ8KBytes;
  auto kernel = moe_down_kernel<kDownWaves, PF>;
  // (The same bound from every call, so that calls of several threads do not
  // lower one another's.)
  if (lds > 48 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, kMostDownLds);
    if (e != hipSuccess) return e;
  }
  // So many rows a wave that all workgroups are on the card at once, one a CU.
  const int per_token = std::max(1, 256 / a.tokens);
  a.groups = (a.rows + per_token * kDownWaves - 1) / (per_token * kDownWaves);
  const int blocks = (a.rows + a.groups * kDownWaves - 1) / (a.groups * kDownWaves);
  kernel<<<dim3(static_cast<uint32_t>(blocks), static_cast<uint32_t>(a.tokens)), dim3(kDownWaves * kWave), lds, stream>>>(a);
  return hipGetLastError();
}

// Mat-vecs, pair by pair and token by token, where they read hardly more than each
// expert once, or where what they read again (from the caches) is less than the
// tiles' launches and passes cost; and a token's h has to fit a workgroup's LDS.
// The experts' call alone, mat-vecs against tiles, us, by tokens:
//   8 experts of 4096 x 14336, 2 used: 2 87 / 109, 4 138 / 147, 5 172 / 153, 8 246 / 182
//   64 experts of 2048 x 1280, 6 used: 8 41 / 67, 16 69 / 90, 24 104 / 104, 48 163 / 122
//   128 experts of 2048 x 768, 8 used: 16 60 / 90, 32 103 / 126, 64 170 / 165
//   8 experts of 2048 x 4096, 2 used: 4 23 / 40, 8 33 / 47, 16 52 / 49, 32 90 / 50
//   16 experts of 1024 x 1024, 4 used: 4 13 / 22, 16 21 / 28, 32 31 / 29
// (The rule turns to tiles at 5, 25, 45, 11 and 34 tokens. An expert costs the tiles a
// start and a tile that is not full, beside what every call costs.)
// Past 80 KiB of LDS, one workgroup of down a CU, rows would still be ahead where
// pairs are no more than experts: one token, 8 used of 4096 x 14336 188 against 197
// us, 8 of 2048 x 11264 89 against 97, 4 of 1024 x 28672 83 against 121; that step
// is not taken.
bool by_rows(int64_t tokens, int64_t used, int64_t experts, int64_t hidden, int64_t ffn) {
  const int64_t pairs = tokens * used, bytes = 3 * (hidden / 256) * ffn * kQ4KBytes;
  return (pairs <= experts || (pairs - experts) * bytes <= 150000000 + experts * 3500000) &&
         used * (ffn / 256) * kQ8KBytes <= kMostDownLds;
}

struct Layout {
  size_t h, xp, xs, hp, hs, out, bytes;
};
// (For any number of experts: the most that a call needs.)
Layout layout(int64_t tokens, int64_t used, int64_t hidden, int64_t ffn) {
  size_t at = kCounterRegion;
  auto take = [&](size_t n) {
    const size_t was = at;
    at += (n + 255) / 256 * 256;
    return was;
  };
  const size_t pairs = static_cast<size_t>(tokens * used), xb = static_cast<size_t>(tokens * (hidden / 256));
  Layout l = {};
  l.h = take(pairs * ffn * 4);
  l.xp = take(xb * kPackBytes);
  l.xs = take(xb * 4);
  l.hp = take(pairs * (ffn / 256) * kPackBytes);
  l.hs = take(pairs * (ffn / 256) * 4);
  l.out = take(pairs * hidden * 4);
  l.bytes = at;
  return l;
}

}  // namespace

size_t moe_route_workspace_bytes(int64_t tokens, int64_t experts) {
  return kCounterRegion + static_cast<size_t>(tokens * experts) * 4;
}

hipError_t launch_moe_route(int32_t* ids, float* weights, const void* x, int x_type, int64_t x_row,
                            const void* router, int router_type, const float* bias, int64_t tokens,
                            int64_t experts, int64_t used, int64_t k, bool sigmoid, bool normalize,
                            float scale, void* ws, hipStream_t stream) {
  RouteArgs a = {};
  a.x = static_cast<const uint8_t*>(x);
  a.router = static_cast<const uint8_t*>(router);
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  a.count = static_cast<int32_t*>(ws);
  a.logits = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kCounterRegion);
  a.x_row = x_row * elem_bytes(x_type);
  a.x_type = x_type;
  a.router_type = router_type;
  a.tokens = static_cast<int>(tokens);
  a.experts = static_cast<int>(experts);
  a.used = static_cast<int>(used);
  a.k = static_cast<int>(k);
  a.expert_tiles = static_cast<int>((experts + kRouteExperts - 1) / kRouteExperts);
  a.sigmoid = sigmoid;
  a.normalize = normalize;
  a.scale = scale;
  auto launch = [&](auto kernel, int64_t nt) {
    const int64_t tiles = (tokens + nt - 1) / nt;
    kernel<<<dim3(static_cast<uint32_t>(tiles * a.expert_tiles)), dim3(kRouteThreads), 0, stream>>>(a);
    return hipGetLastError();
  };
  if (experts <= 64)
    return tokens == 1 ? launch(route_kernel<1, 1>, 1) : launch(route_kernel<4, 1>, 4);
  if (experts <= 128)
    return tokens == 1 ? launch(route_kernel<1, 2>, 1) : launch(route_kernel<4, 2>, 4);
  return tokens == 1 ? launch(route_kernel<1, 16>, 1) : launch(route_kernel<4, 16>, 4);
}

size_t moe_q4k_workspace_bytes(int64_t tokens, int64_t used, int64_t hidden, int64_t ffn) {
  return layout(tokens, used, hidden, ffn).bytes;
}

hipError_t launch_moe_q4k(void* y, int64_t y_row, const void* x, int64_t x_row, int io, const void* gate,
                          const void* up, const void* down, const int32_t* ids, const float* weights,
                          int64_t tokens, int64_t used, int64_t experts, int64_t hidden, int64_t ffn, void* ws,
                          hipStream_t stream) {
  const Layout l = layout(tokens, used, hidden, ffn);
  uint8_t* w = static_cast<uint8_t*>(ws);
  MoeArgs a = {};
  a.x = static_cast<const uint8_t*>(x);
  a.x_row = x_row * elem_bytes(io);
  a.w[0] = static_cast<const uint8_t*>(gate);
  a.w[1] = static_cast<const uint8_t*>(up);
  a.ids = ids;
  a.weights = weights;
  a.out = reinterpret_cast<float*>(w + l.h);
  a.y = static_cast<uint8_t*>(y);
  a.y_row = y_row * elem_bytes(io);
  a.type = io;
  a.x_type = io;
  a.tokens = static_cast<int>(tokens);
  a.used = static_cast<int>(used);
  a.experts = static_cast<int>(experts);
  a.rows = static_cast<int>(ffn);
  a.nb = static_cast<int>(hidden / 256);
  a.used_div = fast_div(static_cast<uint32_t>(used));
  a.nb_div = fast_div(static_cast<uint32_t>(a.nb));
  MoeArgs d = a;
  d.w[0] = static_cast<const uint8_t*>(down);
  d.rows = static_cast<int>(hidden);
  d.nb = static_cast<int>(ffn / 256);
  d.nb_div = fast_div(static_cast<uint32_t>(d.nb));
  d.x = w + l.h;
  hipError_t e;
  if (by_rows(tokens, used, experts, hidden, ffn)) {
    if ((e = launch_up_of(a, stream)) != hipSuccess) return e;
    const int64_t steps = (used * d.nb + kUnitBlocks - 1) / kUnitBlocks;
    if (steps == 1) return launch_down<1>(d, stream);
    if (steps == 2) return launch_down<2>(d, stream);
    if (steps == 3) return launch_down<3>(d, stream);
    return launch_down<4>(d, stream);
  }
  a.xs = reinterpret_cast<const float*>(w + l.xs);
  if ((e = launch_pack(w + l.xp, reinterpret_cast<float*>(w + l.xs), a.x, a.x_row, io, tokens, a.nb, stream)) != hipSuccess)
    return e;
  a.x = w + l.xp;
  if ((e = launch_tiles<2>(a, stream)) != hipSuccess) return e;
  if ((e = launch_pack(w + l.hp, reinterpret_cast<float*>(w + l.hs), d.x, ffn * 4, kF32, tokens * used, d.nb, stream)) !=
      hipSuccess)
    return e;
  d.x = w + l.hp;
  d.xs = reinterpret_cast<const float*>(w + l.hs);
  d.by_pair = 1;
  d.out = reinterpret_cast<float*>(w + l.out);
  if ((e = launch_tiles<1>(d, stream)) != hipSuccess) return e;
  moe_sum_kernel<<<dim3(static_cast<uint32_t>((hidden + 255) / 256), static_cast<uint32_t>(tokens)), dim3(256), 0, stream>>>(d);
  return hipGetLastError();
}

}  // namespace xq
