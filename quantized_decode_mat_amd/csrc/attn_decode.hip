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
// The next tile's K is asked for right after this tile's S^T, its V right after
// this tile's product, the page numbers one tile earlier. (Tiles two ahead, in
// twice the registers, or K turned round in LDS after whole-row loads, were
// both slower.)
//
// Measured: 2 sequences of up to 131072, 32 heads of 128 dims on 8 kv heads, bf16
// cache: 163-172 us, 6.0-6.3 TB/s (a streaming read: 7.3); 64 windows of 8192 of
// 8 bits 131-134 us; one sequence of 517 11.0 us, of which the join is 3.6.
//
// Precision: q and the weights p enter the 16-bit matrix instructions as sums
// of pieces (each the rounded remainder of the one before). For a 16-bit
// output: q exactly, p in two pieces (2^-16 or better). For an f32 output: as
// many pieces as f32 has bits (three of bf16's 8, two of f16's 11). The
// instructions wait on memory, so the pieces cost no time.
#include <algorithm>

#include "kv_device.h"
#include "kv_lanes.h"
#include "kv_launch.h"

namespace xq {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kTile = 32;                   // tokens of a wave's step
constexpr int kStep = kTile * kWaves;       // tokens of a workgroup's step
constexpr int kHeadTile = 16;               // heads of one workgroup
constexpr int kCounterStride = 32;          // ints: a 128-byte line per arrival counter
constexpr int kMaxGroups = 768;             // workgroups that share: 96 KiB of counters in every plan
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
  uint32_t k_page16, k_tok16, v_page16, v_tok16;  // in 16-byte units
  int kv_heads, group, dim, max_len, window, sinks, seqs, head_tiles;
  int shared;     // workgroups share all the work evenly; else one takes one unit
  const int32_t* starts;  // of a chunk's rows
  int rows, max_chunk;
  FastDiv group_div;
  FastDiv ranges;  // parts that the sequences' steps are shared out to
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

// A wave's lanes see what they have left for each other in LDS. (No
// instruction: a wave's LDS accesses keep their order; this keeps the
// compiler's.)
__device__ __forceinline__ void lanes_meet() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// Bits 0 .. n-1.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0 : n >= 32 ? ~0u : (1u << n) - 1; }

// V's loads are whole rows that nothing reads again: non-temporal ones take
// 131072 tokens x 2 from 190 to 174 us. K's take part of a row's line each, and
// lose by it (32768 tokens x 8 stored token by token, 88 against 103 us).
template <int BYTES>
__device__ __forceinline__ u32x4 load_words(const uint8_t* p) {
  if constexpr (BYTES == 16) {
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  } else if constexpr (BYTES == 8) {
    const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
    return u32x4{v.x, v.y, 0, 0};
  } else {
    return u32x4{__builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p)), 0, 0, 0};
  }
}

// Workgroups that a CU is given at most, its SIMDs one wave of each. Twice as
// many of 128 dims and more of a 16-bit cache, each with half the work, are
// slower: 131072 tokens x 2 195 against 174 us. Of 64 dims they are faster (115
// -> 95 us), and of an 8-bit cache of up to 128, whose widening then overlaps
// the loads: 64 windows of 8192 150 -> 138 us, 32 sequences of up to 4099 40 ->
// 33.5. (With pages stored token by token, where a workgroup's rows lie apart,
// the latter lose: 131072 tokens x 2 89 -> 100 us; those take one.)
constexpr int groups_per_cu(int ct, int dp) { return dp == 64 || (ct == kE4M3 && dp == 128) ? 2 : 1; }

// CT: the cache's type. IO: q's and out's. DP: dim rounded up to 64, 128, 192
// or 256; FULL: dim is DP. CHUNK: several new tokens per sequence; a
// workgroup's 16 columns are then 16 of a sequence's (token, head) rows, which
// see different tokens.
template <int CT, int IO, int DP, bool FULL, bool CHUNK>
__global__ __launch_bounds__(kThreads, groups_per_cu(CT, DP)) void attn_decode_kernel(DecodeArgs a) {
  constexpr int MT = CT == kBF16 ? kBF16 : kF16;   // the matrix instruction's type
  constexpr int EB = CT == kE4M3 ? 1 : 2;
  constexpr int IB = IO == kF32 ? 4 : 2;
  // Pieces of q and of p.
  constexpr int NQ = MT == kBF16 ? (IO == kBF16 ? 1 : 3) : (IO == kF32 ? 2 : 1);
  constexpr int NP = MT == kBF16 && IO == kF32 ? 3 : 2;
  constexpr int QS = DP / 32;                      // instructions of S^T along dim
  // 16 bytes of K give KL instructions their operand: an 8-bit row's are 16
  // dims, two instructions' worth.
  constexpr int KL = CT == kE4M3 ? 2 : 1;
  constexpr int KN = decode_k_loads(DP, EB);       // K loads of a lane per token
  static_assert(KN * KL == QS);
  constexpr int VE = decode_v_dims(DP);            // dims of a lane's V load
  constexpr int VC = decode_v_loads(DP);
  constexpr int OS = DP + 4;                       // floats of a joined row in LDS
  extern __shared__ float lds[];
  __shared__ __attribute__((aligned(16))) uint32_t places[kWaves][2][kTile];

  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int l16 = lane % 16, lg = lane / 16;
  const int per_seq = a.kv_heads * a.head_tiles;  // units of a sequence
  // A sequence's visible tokens as one run: `ns` sinks, then lo .. n-1.
  auto length_of = [&](int len) {
    return static_cast<int>(min(static_cast<int64_t>(max(0, min(len, a.max_len))), a.table_tokens));
  };
  auto low_of = [&](int n) { return a.window && n > a.window ? n - a.window : 0; };
  auto steps_of = [&](int n) {
    const int lo = low_of(n);
    return max(1, (n - lo + min(a.sinks, lo) + kStep - 1) / kStep);
  };

  // This workgroup's unit (kv head and 16 of its heads), and its part of every
  // sequence's steps laid end to end: [at, stop), `at` lying in sequence `seq`,
  // which begins at `seq0`. Workgroups next to each other have one part and the
  // sequence's units: they walk over the same pages at the same time, and a
  // page's heads, which are neighbours in memory, are read together.
  const int unit = blockIdx.x % per_seq, range = blockIdx.x / per_seq;
  int seq, n, steps, at, stop, seq0, each;
  if (a.shared) {
    // Every wave adds up the sequences' steps for itself, 64 sequences at a
    // time; with more, the second pass stops where `at` lies.
    int n_l, steps_l, begin_l, before = 0, chunk = 0;
    auto add_up = [&](int b) {
      n_l = b + lane < a.seqs ? length_of(a.lens[b + lane]) : 0;
      steps_l = b + lane < a.seqs ? steps_of(n_l) : 0;
      int x = steps_l;
#pragma unroll
      for (int d = 1; d < kWave; d <<= 1) {
        const int y = __shfl_up(x, d, kWave);
        if (lane >= d) x += y;
      }
      begin_l = before + x - steps_l;
      before += __builtin_amdgcn_readlane(x, kWave - 1);
    };
    for (int b = 0; b < a.seqs; b += kWave) add_up(b);
    const int all = before;
    each = div_by(all + a.ranges.d - 1, a.ranges);
    at = range * each;
    stop = min(all, at + each);
    if (at >= stop) return;
    if (a.seqs > kWave) {
      before = 0;
      for (;; chunk += kWave) {
        add_up(chunk);
        if (before > at) break;
      }
    }
    // The last lane whose sequence begins at or before `at`.
    const int l = kWave - 1 - __builtin_clzll(__ballot(steps_l > 0 && begin_l <= at));
    seq = chunk + l;
    n = __builtin_amdgcn_readlane(n_l, l);
    steps = __builtin_amdgcn_readlane(steps_l, l);
    seq0 = __builtin_amdgcn_readlane(begin_l, l);
  } else {
    seq = range;
    n = length_of(a.lens[seq]);
    steps = CHUNK ? 1 : steps_of(n);
    at = seq0 = 0;
    stop = each = steps;
  }
  const int ht = unit % a.head_tiles, kvh = unit / a.head_tiles;
  // This workgroup's heads, or rows: `heads` of them, the first head0. Row r of
  // a chunk is its token r / group, and head r % group of the kv head's.
  int heads, head0, first_row = 0, pos = 0, pmin = 0, pmax = 0;
  if constexpr (CHUNK) {
    first_row = min(max(a.starts[seq], 0), a.rows);
    const int end = a.starts[seq + 1];
    const int count = min(min(max(end, first_row), a.rows) - first_row, a.max_chunk);
    head0 = ht * kHeadTile;
    heads = min(kHeadTile, count * a.group - head0);
    if (heads <= 0) return;
    // The chunk's last row, whether it is done or left out, is the sequence's
    // last token. A position below 0 sees nothing. (end > first_row >= 0 here.)
    const int base = n - (end - first_row);
    auto position = [&](int r) { return max(base + static_cast<int>(div_by(head0 + r, a.group_div)), -1); };
    pos = position(min(l16, heads - 1));
    pmin = position(0);
    pmax = position(heads - 1);
  } else {
    heads = min(kHeadTile, a.group - ht * kHeadTile);
    head0 = kvh * a.group + ht * kHeadTile;
  }
  const int sinks = a.window ? a.sinks : 0;
  // Byte offset of this workgroup's row r, given a tensor's strides.
  auto row_at = [&](int r, int64_t row_stride, int64_t head_stride) {
    if constexpr (CHUNK) {
      const int t = div_by(head0 + r, a.group_div);
      return (first_row + t) * row_stride + (kvh * a.group + head0 + r - t * a.group) * head_stride;
    } else {
      return seq * row_stride + (head0 + r) * head_stride;
    }
  };

  for (bool first = true; at < stop; first = false) {
  const int begin_step = at - seq0, end_step = min(steps, stop - seq0);
  // The tokens that any row sees.
  const int lo = CHUNK ? (a.window ? max(0, pmin - a.window + 1) : 0) : low_of(n), ns = min(sinks, lo);
  const int begin = begin_step * kStep;
  const int end = CHUNK ? max(0, pmax + 1 - lo) + ns : min(n - lo + ns, end_step * kStep);

  const uint8_t* kb = a.kv.k + kvh * a.kv.k_head;
  const uint8_t* vb = a.kv.v + kvh * a.kv.v_head;
  const int32_t* table = a.tables + seq * a.table_stride;

  const f32x4 zero4 = {0.f, 0.f, 0.f, 0.f};
  constexpr uint32_t kSigns = EB == 1 ? 0x80808080u : 0x80008000u;
  constexpr uint32_t kOne = EB == 1 ? 0x01010101u : CT == kBF16 ? 0x00800080u : 0x04000400u;
  f32x4 o[VC][VE];
#pragma unroll
  for (int c = 0; c < VC; ++c)
#pragma unroll
    for (int j = 0; j < VE; ++j) o[c][j] = zero4;
  float m = -INFINITY, l = 0.f;

  // The lanes look up a tile's tokens (lane l token l % 32) and leave their
  // places, in 16-byte units, in the wave's corner of LDS. Lane l's K loads
  // need those of tokens l % 16 and 16 + l % 16, its V loads those of 4g .. 4g+3
  // and 16 + those.
  auto token_of = [&](int u) { return u < ns ? u : lo + (u - ns); };
  auto page_of = [&](int u0) {
    const int u = u0 + lane % kTile;
    const int page = table[u < end ? div_by(token_of(u), a.kv.page) : 0];
    return u < end ? page : -1;
  };
  uint32_t live;  // bit t: token t of the tile is there
  uint32_t k_at = 0, v_at = 0;
  auto place = [&](int u0, int page) {
    const int u = u0 + lane % kTile;
    const bool ok = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.kv.pages);
    const uint32_t j = token_of(u);
    const uint32_t slot = j - div_by(j, a.kv.page) * a.kv.page.d;
    // A token that is not there reads what was read last in its stead, at
    // first the start of page 0, which is always there; its score is hidden
    // and its v is cleared.
    k_at = ok ? page * a.k_page16 + slot * a.k_tok16 : k_at;
    v_at = ok ? page * a.v_page16 + slot * a.v_tok16 : v_at;
    lanes_meet();
    places[wave][0][lane % kTile] = k_at;
    places[wave][1][lane % kTile] = v_at;
    lanes_meet();
    live = static_cast<uint32_t>(__ballot(ok));
  };
  u32x4 kr[2][KN], vr[VC][8];
  auto load_k = [&]() {
    uint32_t at[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) at[t] = places[wave][0][t * 16 + l16];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint8_t* p = kb + static_cast<uint64_t>(at[t]) * 16;
#pragma unroll
      for (int s = 0; s < KN; ++s)
        kr[t][s] = *reinterpret_cast<const u32x4*>(p + decode_k_dim<DP, FULL>(s, lg, EB, a.dim) * EB);
    }
  };
  auto load_v = [&]() {
    u32x4 at[2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
      at[t] = *reinterpret_cast<const u32x4*>(&places[wave][1][t * 16 + lg * 4]);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const uint8_t* p = vb + static_cast<uint64_t>(at[t / 4][t % 4]) * 16;
#pragma unroll
      for (int c = 0; c < VC; ++c)  // (what stands for dims past the end nothing uses)
        vr[c][t] = load_words<VE * EB>(p + decode_v_dim<DP, FULL>(c, l16, a.dim) * EB);
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
  int page;  // of the lane's token in the next tile
  // q as the B operand: head l16, dims of step s. An f16 operand is scaled by
  // a power of two that brings the head's largest |q| to 2^14..2^15, so that
  // no piece of an f32 or bf16 q leaves f16's range.
  u32x4 qf[QS][NQ];
  float qs = a.c;
  {
    float x[QS][8];
    float top = 0.f;
    const uint8_t* qr = a.q + row_at(min(l16, heads - 1), a.q_row, a.q_head);
    auto q_dim = [&](int s) {
      return KL == 1 ? s * 32 + lg * 8 : (s / 2) * 64 + lg * 16 + (s % 2) * 8;
    };
    u32x4 raw[QS][IB / 2];
#pragma unroll
    for (int s = 0; s < QS; ++s) {
      const bool in = l16 < heads && (FULL || q_dim(s) < a.dim);
#pragma unroll
      for (int i = 0; i < IB / 2; ++i) {
        raw[s][i] = load_words<16>(in ? qr + q_dim(s) * IB + i * 16 : a.q);
        if (!in) raw[s][i] = u32x4{0, 0, 0, 0};
      }
    }
    // The first tile's loads go out behind q's, before q is waited for.
    if (u0 < end) {
      page = page_of(u0);
      const int next = page_of(u0 + kStep);
      place(u0, page);
      page = next;
      load_k();
      load_v();
    }
#pragma unroll
    for (int s = 0; s < QS; ++s)
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        f32x2 y;
        if constexpr (IO == kF32) {
          const uint32_t y0 = raw[s][e / 4][e % 4], y1 = raw[s][e / 4][e % 4 + 1];
          y = f32x2{__builtin_bit_cast(float, y0), __builtin_bit_cast(float, y1)};
        } else {
          y = unpack2<IO>(raw[s][0][e / 2]);
        }
        x[s][e] = y.x;
        x[s][e + 1] = y.y;
        top = fmaxf(top, fmaxf(fabsf(y.x), fabsf(y.y)));
      }
    float mul = 1.f;
    if constexpr (MT == kF16) {
      top = heads_max(top);
      if (top > 0.f && top < INFINITY) {
        const int e = min(__builtin_amdgcn_frexp_expf(top), 126) - 15;
        mul = ldexpf(1.f, min(127, -e));
        qs = a.c * ldexpf(1.f, max(-127, e));
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

  // The loads of the next tile are not conditional (past the last, its tokens
  // are not there and read what was read before): the compiler then knows how
  // many are under way and waits for no more than it needs.
  while (u0 < end) {  // wave-uniform
    const uint32_t here = live;
    f32x4 st[2] = {zero4, zero4};
#pragma unroll
    for (int s = 0; s < QS; ++s)
#pragma unroll
      for (int p = 0; p < NQ; ++p)
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
          if constexpr (!FULL) {
            // q is 0 past the end, but 0 * infinity is not.
            const int d0 = KL == 1 ? s * 32 + lg * 8 : (s / 2) * 64 + lg * 16 + (s % 2) * 8;
            if (d0 >= a.dim) kf = u32x4{0, 0, 0, 0};
          }
          st[t] = mfma16<MT>(kf, qf[s][p], st[t]);
        }
    place(u0 + kStep, page);
    page = page_of(u0 + 2 * kStep);
    load_k();

    // Which of the tile's tokens this lane's row sees.
    uint32_t sees = here;
    bool same = true;  // for all rows
    if constexpr (CHUNK) {
      const int u = u0;
      const int j0 = token_of(u), j31 = token_of(u + kTile - 1);
      same = j31 <= pmin && (!a.window || j0 > pmax - a.window || j31 < sinks);
      if (!same) {
        // Bit k is token u + k where that is a sink, else token j + k.
        const int j = lo + u - ns;
        const uint32_t sink = below(ns - u) & below(pos + 1 - u);
        const uint32_t rest = ~below(ns - u) & below(pos + 1 - j) &
                              (a.window ? ~below(pos - a.window + 1 - j) | below(sinks - j) : ~0u);
        sees = sink | rest;
        sees &= here;
      }
    }
    float s[8];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[i] = st[i / 4][i % 4] * qs;
      if (!((sees >> ((i / 4) * 16 + lg * 4 + i % 4)) & 1)) s[i] = -INFINITY;
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
    // Whether the tile's V has an infinity or NaN: an exponent of all ones (of
    // 8 bits, all ones but the sign) carries into the sign's place. (An 8-bit V
    // has no infinity, and a NaN that every row sees needs no care.)
    bool odd = false;
    if (CT != kE4M3 || !same) {
      uint32_t carry = 0;
#pragma unroll
      for (int c = 0; c < VC; ++c)
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int i = 0; i < VE * EB / 4; ++i) carry |= (vr[c][t][i] & ~kSigns) + kOne;
      odd = __ballot(carry & kSigns) != 0;
    }
    if (CHUNK && odd && !same) {
      // Some rows do not see it, and 0 * NaN must not reach them: such values
      // are left out of the product and added to the rows that do.
#pragma unroll
      for (int c = 0; c < VC; ++c)
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int i = 0; i < VE * EB / 4; ++i) {
            const uint32_t w = vr[c][t][i];
            const uint32_t ones = (((w & ~kSigns) + kOne) & kSigns) >> (8 * EB - 1);
            vr[c][t][i] = w & ~(ones * (EB == 1 ? 0xffu : 0xffffu));
          }
      odd = false;
#pragma unroll 1
      for (int k = 0; k < kTile; ++k) {
        const uint32_t page0 = table[div_by(token_of(min(u0 + k, end - 1)), a.kv.page)];
        if (!((here >> k) & 1)) continue;
        const uint32_t j = token_of(u0 + k), slot = j - div_by(j, a.kv.page) * a.kv.page.d;
        const uint8_t* row = vb + page0 * a.kv.v_page + slot * a.kv.v_tok;
        const bool in = (sees >> k) & 1;
#pragma unroll
        for (int c = 0; c < VC; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            u32x4 w = load_words<VE * EB>(row + decode_v_dim<DP, FULL>(c, lg * 4 + i, a.dim) * EB);
            if constexpr (EB == 1) {
              const u32x2 x = widen4<MT>(w.x), y = widen4<MT>(w.y);
              w = u32x4{x.x, x.y, y.x, y.y};
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) {
              const f32x2 pair = unpack2<MT>(w[e / 2]);
              const float x = e % 2 ? pair.y : pair.x;
              o[c][e][i] += in && !(fabsf(x) < INFINITY) ? x : 0.f;
            }
            __builtin_amdgcn_sched_barrier(0);
          }
      }
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
            o[c][j][i] += fabsf(x[i]) < INFINITY ? x[i] : 0.f;
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    load_v();
    u0 += kStep;
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
  constexpr int PR = DP + 4;  // floats of a partial result per head: o, m, l, two of padding
  const bool whole = begin_step == 0 && end_step == steps;
  // A workgroup has at most two parts of sequences that it shares: its first
  // and its last.
  const int64_t part_size = static_cast<int64_t>(min(kHeadTile, a.group)) * PR;
  float* mine = a.part + (2 * blockIdx.x + (first ? 0 : 1)) * part_size;
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
        store_from_f32(a.out + row_at(r, a.out_row, a.out_head), IO, d,
                       sum == 0.f ? 0.f : x / sum * a.v_scale);
    } else {
      __hip_atomic_store(mine + i, x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (d == 0) {
        __hip_atomic_store(mine + heads * DP + r, top, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(mine + heads * DP + heads + r, sum, __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
      }
    }
  }

  if (!whole) {  // workgroup-uniform
    // The ranges that hold the sequence's first and last step; the first one's
    // counter counts, and its part is its second if it began with another one.
    const int r0 = static_cast<uint32_t>(seq0) / static_cast<uint32_t>(each);
    const int parts = static_cast<uint32_t>(seq0 + steps - 1) / static_cast<uint32_t>(each) - r0 + 1;
    const int second = r0 * each < seq0;
    const int g0 = r0 * per_seq + unit;
    // The last part to arrive joins them all. The partials and the counter are
    // agent-scope atomics, which bypass the per-XCD L2's non-coherent state;
    // each wave waits for its stores' acknowledgement before the barrier, so
    // whoever sees the last count sees every partial. It drops what its caches
    // hold (the acquire fence) and reads them with plain 16-byte loads, several
    // under way at once: read as atomics, 4 bytes at a time, 32 parts of 4
    // heads took 18 us longer than 16.
    __shared__ int last;
    __builtin_amdgcn_s_waitcnt(kWaitVm0);
    __syncthreads();
    if (tid == 0)
      last = __hip_atomic_fetch_add(a.count + g0 * kCounterStride, 1, __ATOMIC_RELAXED,
                                    __HIP_MEMORY_SCOPE_AGENT) == parts - 1;
    __syncthreads();
    if (last) {  // workgroup-uniform
      if (tid == 0)
        __hip_atomic_store(a.count + g0 * kCounterStride, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
      const float* p_first = a.part + (2 * g0 + second) * part_size;
      const float* p_rest = a.part + 2 * g0 * part_size;  // part i > 0 is p_step * i on
      const int64_t p_step = 2 * per_seq * part_size;
      auto part = [&](int i) { return i ? p_rest + i * p_step : p_first; };
      // A thread adds up four outputs over every `teams`th part, then the teams
      // are added up. The first of its loads go out ahead of those that the
      // factors wait for.
      constexpr int kAhead = 8;
      const int quads = heads * DP / 4, teams = join_teams(kThreads, quads);
      const int team = tid % teams;
      f32x4 ahead[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        ahead[k] = reinterpret_cast<const f32x4*>(part(min(team + k * teams, parts - 1)))[min(tid / teams, quads - 1)];
      // The parts' factors exp(m - max m) / sum, [head][part], in LDS.
      for (int r = wave; r < heads; r += kWaves) {
        const float* ml = part(min(lane, parts - 1)) + heads * DP + r;
        const float m0 = lane < parts ? ml[0] : -INFINITY, l0 = ml[heads];
        float top = m0;
        for (int i = lane + kWave; i < parts; i += kWave) top = fmaxf(top, part(i)[heads * DP + r]);
        top = wave_max(top);
        const float base = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
        for (int i = lane; i < parts; i += kWave) {
          const float* p = part(i) + heads * DP + r;
          const float f = exp2_fast((i < kWave ? m0 : p[0]) - base);
          lds[r * parts + i] = f;
          sum += f * (i < kWave ? l0 : p[heads]);
        }
        sum = wave_sum(sum);
        const float inv = sum == 0.f ? 0.f : a.v_scale / sum;
        for (int i = lane; i < parts; i += kWave) lds[r * parts + i] *= inv;
      }
      __syncthreads();
      f32x4* sums = reinterpret_cast<f32x4*>(lds + (heads * parts + 3) / 4 * 4);
      for (int q0 = 0; q0 < quads; q0 += kThreads / teams) {
        const int q = q0 + tid / teams, r = q * 4 / DP, d = q * 4 % DP;
        f32x4 x = zero4;
        if (q < quads) {
          int i = team;
          if (q0 == 0) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k, i += teams)
              if (i < parts) x += lds[r * parts + i] * ahead[k];
          }
#pragma unroll 8
          for (; i < parts; i += teams)
            x += lds[r * parts + i] * reinterpret_cast<const f32x4*>(part(i))[q];
        }
        if (teams > 1) {
          sums[tid] = x;
          __syncthreads();
          if (join_adds(tid, teams, quads - q0))
            for (int i = 1; i < teams; ++i) x += sums[tid + i];
          __syncthreads();
        }
        if (join_adds(tid, teams, quads - q0) && d < a.dim) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            store_from_f32(a.out + row_at(r, a.out_row, a.out_head), IO, d + i, x[i]);
        }
      }
    }
  }

  // On to the next sequence.
  at = seq0 = seq0 + steps;
  if (at >= stop) break;
  ++seq;
  n = length_of(a.lens[seq]);
  steps = steps_of(n);
  __syncthreads();  // LDS is free again
  }
}

// Units of a sequence: a kv head and 16 of its heads each.
int64_t units_of(int64_t heads, const xq_kv& kv) {
  return kv.kv_heads * ((heads / kv.kv_heads + kHeadTile - 1) / kHeadTile);
}

struct Plan {
  int64_t per_seq, ranges;  // units of a sequence; parts of all sequences' steps
  bool shared;
};
// As many workgroups as fill the card share the work evenly, to a step:
// sequences of any lengths keep all of it busy to the end, at the price of a
// join (3.6 us) for each sequence that crosses from one range to the next. Up
// to three steps (384 tokens) one workgroup is faster than a join: 300 tokens
// take 10.4 against 11.2 us, 517 tokens 13 against 11.2. With three and more
// units for each such workgroup, one unit each is even enough where the lengths
// are alike (32 heads on 8 kv heads of 128 dims, bf16: 128 sequences of 2000 178
// us, 5.9 TB/s, as 95 of them that share; 256 of 500 to 4000 380 us, 6.1 TB/s)
// and far from it where one is much longer: 96 sequences, one of 131072 and 95
// of 1000, take 1.38 ms, with 94 of 1000, shared, 161 us.
Plan plan(int64_t seqs, int64_t heads, const xq_kv& kv, int64_t max_len, int64_t window,
          int64_t sinks) {
  Plan p;
  p.per_seq = units_of(heads, kv);
  const int64_t most = window && window + sinks < max_len ? window + sinks : max_len;
  const int64_t steps = (most + kStep - 1) / kStep;
  const int dp = decode_dim_pad(static_cast<int>(kv.dim));
  const bool apart = dp == 128 && kv.k_stride[3] != kv.dim && kv.page > 1;
  const int64_t room = 256 * (apart ? 1 : groups_per_cu(kv.dtype, dp));
  p.shared = steps > 3 && seqs * p.per_seq < 3 * room && p.per_seq <= room && seqs * steps < (1 << 30);
  p.ranges = p.shared ? std::min(room / p.per_seq, seqs * steps) : seqs;
  return p;
}

constexpr size_t kCounterBytes = static_cast<size_t>(kMaxGroups) * kCounterStride * 4;

template <int CT, int IO, int DP, bool FULL, bool CHUNK>
hipError_t launch(const DecodeArgs& a, const Plan& p, hipStream_t stream) {
  const int heads = CHUNK ? kHeadTile : std::min(kHeadTile, a.group);
  size_t lds = static_cast<size_t>(kWaves) * heads * (DP + 4 + 2) * 4;
  if (!CHUNK) lds = std::max(lds, (static_cast<size_t>(heads) * (p.ranges + 1) + kThreads * 4 + 4) * 4);
  auto kernel = attn_decode_kernel<CT, IO, DP, FULL, CHUNK>;
  if (lds > 48 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(lds));
    if (e != hipSuccess) return e;
  }
  kernel<<<dim3(static_cast<uint32_t>(p.per_seq * p.ranges)), dim3(kThreads), lds, stream>>>(a);
  return hipGetLastError();
}

template <int CT, int IO, bool CHUNK>
hipError_t launch_dim(const DecodeArgs& a, const Plan& p, hipStream_t stream) {
  switch (a.dim) {
    case 64: return launch<CT, IO, 64, true, CHUNK>(a, p, stream);
    case 128: return launch<CT, IO, 128, true, CHUNK>(a, p, stream);
    case 192: return launch<CT, IO, 192, true, CHUNK>(a, p, stream);
    case 256: return launch<CT, IO, 256, true, CHUNK>(a, p, stream);
  }
  switch (decode_dim_pad(a.dim)) {
    case 64: return launch<CT, IO, 64, false, CHUNK>(a, p, stream);
    case 128: return launch<CT, IO, 128, false, CHUNK>(a, p, stream);
    case 192: return launch<CT, IO, 192, false, CHUNK>(a, p, stream);
    default: return launch<CT, IO, 256, false, CHUNK>(a, p, stream);
  }
}

template <int CT>
hipError_t launch_io(int io, const DecodeArgs& a, const Plan& p, hipStream_t stream) {
  switch (io) {
    case kF32: return launch_dim<CT, kF32, false>(a, p, stream);
    case kBF16: return launch_dim<CT, kBF16, false>(a, p, stream);
    default: return launch_dim<CT, kF16, false>(a, p, stream);
  }
}

}  // namespace

int64_t attn_decode_units(int64_t seqs, int64_t heads, const xq_kv& kv) { return seqs * units_of(heads, kv); }

size_t attn_decode_workspace_bytes(int64_t seqs, int64_t heads, const xq_kv& kv, int64_t max_len,
                                   int64_t window, int64_t sinks) {
  const Plan p = plan(seqs, heads, kv, max_len, window, sinks);
  if (!p.shared) return 0;
  return kCounterBytes + static_cast<size_t>(p.per_seq * p.ranges) * 2 * std::min<int64_t>(kHeadTile, heads / kv.kv_heads) *
                             (decode_dim_pad(static_cast<int>(kv.dim)) + 4) * 4;
}

namespace {

DecodeArgs fill(const RowsView& out, const RowsView& q, int64_t heads, const xq_kv& kv,
                const TableView& tables, const int32_t* lens, float scale, int64_t window,
                int64_t sinks) {
  const int eb = elem_bytes(kv.dtype), ib = elem_bytes(q.type);
  DecodeArgs a = {};
  a.kv = KvView{static_cast<uint8_t*>(kv.k), static_cast<uint8_t*>(kv.v),
                kv.k_stride[1] * eb, kv.k_stride[2] * eb, kv.k_stride[3] * eb,
                kv.v_stride[1] * eb, kv.v_stride[2] * eb, kv.v_stride[3] * eb,
                fast_div(static_cast<uint32_t>(kv.page)), static_cast<int>(kv.pages)};
  a.q = static_cast<const uint8_t*>(q.data);
  a.out = static_cast<uint8_t*>(out.data);
  a.tables = tables.data;
  a.lens = lens;
  a.q_row = q.row * ib;
  a.q_head = q.head * ib;
  a.out_row = out.row * ib;
  a.out_head = out.head * ib;
  a.table_stride = tables.stride;
  a.table_tokens = tables.width * kv.page;
  a.kv_heads = static_cast<int>(kv.kv_heads);
  a.group = static_cast<int>(heads / kv.kv_heads);
  a.dim = static_cast<int>(kv.dim);
  a.k_page16 = static_cast<uint32_t>(a.kv.k_page / 16);
  a.k_tok16 = static_cast<uint32_t>(a.kv.k_tok / 16);
  a.v_page16 = static_cast<uint32_t>(a.kv.v_page / 16);
  a.v_tok16 = static_cast<uint32_t>(a.kv.v_tok / 16);
  a.max_len = 1 << 30;
  a.window = static_cast<int>(window);
  a.sinks = static_cast<int>(sinks);
  a.c = scale * kv.k_scale * kLog2e;
  a.v_scale = kv.v_scale;
  return a;
}

// Row tiles of a sequence's kv heads.
int64_t chunk_units(int64_t heads, const xq_kv& kv, int64_t max_chunk) {
  return kv.kv_heads * ((max_chunk * (heads / kv.kv_heads) + kHeadTile - 1) / kHeadTile);
}

}  // namespace

hipError_t launch_attn_decode(const RowsView& out, const RowsView& q, int64_t seqs, int64_t heads,
                              const xq_kv& kv, const TableView& tables, const int32_t* lens,
                              float scale, int64_t window, int64_t sinks, int64_t max_len, void* ws,
                              hipStream_t stream) {
  const Plan p = plan(seqs, heads, kv, max_len, window, sinks);
  DecodeArgs a = fill(out, q, heads, kv, tables, lens, scale, window, sinks);
  a.count = static_cast<int32_t*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kCounterBytes);
  a.max_len = static_cast<int>(max_len);
  a.seqs = static_cast<int>(seqs);
  a.shared = p.shared;
  a.ranges = fast_div(static_cast<uint32_t>(p.ranges));
  a.head_tiles = static_cast<int>(p.per_seq / kv.kv_heads);
  switch (kv.dtype) {
    case kBF16: return launch_io<kBF16>(q.type, a, p, stream);
    case kF16: return launch_io<kF16>(q.type, a, p, stream);
    default: return launch_io<kE4M3>(q.type, a, p, stream);
  }
}

// Tiles of 16 rows, each walked by a workgroup's four waves in steps of 128
// tokens, against tiles of 128 rows in steps of 64: as long as all of the
// former are on the card at once (two a CU) they are the shorter walk, whatever
// its length. bf16, 32 heads on 8 kv heads of 128 dims: 11 new tokens on 1530 26
// against 47 us, 8 on 131072 1.33 against 3.53 ms, 256 on 131072 (512 tiles)
// 2.69 against 3.54; 512 on 131072 5.31 against 3.56. 8 heads on 2: 364 on 624
// 17.5 against 25 us, 90 on 1976 of 192 dims 47 against 89. A walk of a single
// step is the exception, 8 on 92 of 192 dims 15.5 against 12. Neither kernel
// shares one tile's tokens between workgroups: 8 on 131072 are 16 workgroups
// that read 0.4 TB/s, where single tokens on the whole card read 6.
bool chunk_in_rows(int64_t seqs, int64_t heads, const xq_kv& kv, int64_t max_chunk) {
  return seqs * chunk_units(heads, kv, max_chunk) <= 512;
}

hipError_t launch_attn_chunk(const RowsView& out, const RowsView& q, int64_t rows, int64_t seqs,
                             int64_t heads, const xq_kv& kv, const TableView& tables,
                             const int32_t* lens, const int32_t* starts, int64_t max_chunk,
                             float scale, int64_t window, int64_t sinks, hipStream_t stream) {
  DecodeArgs a = fill(out, q, heads, kv, tables, lens, scale, window, sinks);
  Plan p;
  p.per_seq = chunk_units(heads, kv, max_chunk);
  p.ranges = seqs;
  p.shared = false;
  a.head_tiles = static_cast<int>(p.per_seq / kv.kv_heads);
  a.starts = starts;
  a.rows = static_cast<int>(rows);
  a.max_chunk = static_cast<int>(max_chunk);
  a.group_div = fast_div(static_cast<uint32_t>(a.group));
  if (kv.dtype == kBF16) return launch_dim<kBF16, kBF16, true>(a, p, stream);
  if (kv.dtype == kF16) return launch_dim<kF16, kF16, true>(a, p, stream);
  return q.type == kBF16 ? launch_dim<kE4M3, kBF16, true>(a, p, stream)
                         : launch_dim<kE4M3, kF16, true>(a, p, stream);
}

}  // namespace xq
