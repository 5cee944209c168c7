// rope.hip — rotary positions, alone and fused with the append to the cache.
//
//   angle = pos[axis][t] * freq[i];  (a, b) -> (a cos - b sin, a sin + b cos)
//
// What bounds it: bytes, each element read once and written once. A workgroup
// takes a few tokens and some of their heads: its threads first form the
// tokens' sines and cosines, one pair each, into LDS, then walk over (head,
// piece of 8 elements) items: a piece holds four pairs (two loads of four
// elements, at i and i + rot/2 or side by side), or elements to copy.
//
// Measured: the append of 8192 tokens (32 + 2 x 8 heads of 128, f32 to bf16, three
// axes) 60 us, 5.0 TB/s read and written, a large copy's rate (4.93). Four items
// ahead per thread were slower for their registers (85 against 77 us).
//
// Precision: a position of 2^18 times a frequency of 1 needs 18 bits before
// the point, so the angle is formed and reduced to [-pi/4, pi/4] in f64 (this
// card's f64 multiplies are as fast as its f32 ones); the sine and cosine of
// the rest are Taylor sums in f32 whose first left-out terms are below 2^-28.
#include <algorithm>

#include "kv_device.h"
#include "kv_launch.h"
#include "kv_view.h"

namespace xq {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 4;  // of a workgroup

struct RopeArgs {
  const uint8_t* src[3];             // q, k, v
  int64_t row[3], head[3];           // bytes
  uint8_t* out;
  int64_t out_row, out_head;
  KvView kv;
  const int32_t* pos;
  const double* freq;
  const int64_t* slots;
  int64_t pos_stride, cache_slots;
  int tokens, heads, kv_heads, dim, half, x_type, out_type, cache_type, adjacent, inverse;
  int per_block, head_blocks;        // tokens of a workgroup; workgroups that share a token's heads
  int bound[3];                      // first pair of axes 1, 2 and 3
  FastDiv items;                     // dim / 8, pieces of a head
  float k_scale, v_scale;
  ExpView exps;
  FastDiv quarters;                  // dim / 4
  double k_inv, v_inv;               // 1 / k_scale, 1 / v_scale
  int q_blocks, kv_block, kv_parts;  // workgroups of q; tokens of one of k and v, and those that share them
};

__device__ __forceinline__ void sin_cos(double angle, float* s, float* c) {
  // angle = n * pi/2 + r; pi/2 in two parts, so that r is good to f64's own
  // rounding of the angle.
  const double n = rint(angle * 0.63661977236758134308);
  double r = fma(n, -1.57079632679489655800, angle);
  r = fma(n, -6.12323399573676603587e-17, r);
  const float x = static_cast<float>(r), y = x * x;
  float sn = 2.75573192e-6f;
  sn = fmaf(sn, y, -1.98412698e-4f);
  sn = fmaf(sn, y, 8.33333333e-3f);
  sn = fmaf(sn, y, -1.66666667e-1f);
  sn = fmaf(sn * y, x, x);
  float cs = -2.75573192e-7f;
  cs = fmaf(cs, y, 2.48015873e-5f);
  cs = fmaf(cs, y, -1.38888889e-3f);
  cs = fmaf(cs, y, 4.16666667e-2f);
  cs = fmaf(cs, y, -0.5f);
  cs = fmaf(cs, y, 1.f);
  // The quadrant n mod 4, from the f64's last whole bits.
  const int q = static_cast<int>(n - 4.0 * floor(n * 0.25));
  const float u = q & 1 ? cs : sn, w = q & 1 ? sn : cs;
  *s = q & 2 ? -u : u;
  *c = (q + 1) & 2 ? -w : w;
}

// Four elements from p, p 4-element aligned when VEC.
template <bool VEC>
__device__ __forceinline__ f32x4 load4(const uint8_t* p, int type, int at) {
  if constexpr (VEC) {
    if (type == kF32) return *reinterpret_cast<const f32x4*>(p + at * 4);
    const u32x2 w = *reinterpret_cast<const u32x2*>(p + at * 2);
    const f32x2 a = type == kBF16 ? unpack2<kBF16>(w.x) : unpack2<kF16>(w.x);
    const f32x2 b = type == kBF16 ? unpack2<kBF16>(w.y) : unpack2<kF16>(w.y);
    return f32x4{a.x, a.y, b.x, b.y};
  } else {
    return f32x4{load_as_f32(p, type, at), load_as_f32(p, type, at + 1),
                 load_as_f32(p, type, at + 2), load_as_f32(p, type, at + 3)};
  }
}

__device__ __forceinline__ float clamp8(float x) {
  // NaN passes (fminf and fmaxf would drop it).
  return x > 448.f ? 448.f : x < -448.f ? -448.f : x;
}
__device__ __forceinline__ uint32_t pack4_e4m3(f32x4 x) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(clamp8(x.x), clamp8(x.y), 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(clamp8(x.z), clamp8(x.w), w, true));
}

template <bool VEC>
__device__ __forceinline__ void store4(uint8_t* p, int type, int at, f32x4 x) {
  if constexpr (VEC) {
    if (type == kF32) {
      *reinterpret_cast<f32x4*>(p + at * 4) = x;
    } else if (type == kE4M3) {
      *reinterpret_cast<uint32_t*>(p + at) = pack4_e4m3(x);
    } else {
      *reinterpret_cast<u32x2*>(p + at * 2) =
          type == kBF16 ? u32x2{pack2<kBF16>(x.x, x.y), pack2<kBF16>(x.z, x.w)}
                        : u32x2{pack2<kF16>(x.x, x.y), pack2<kF16>(x.z, x.w)};
    }
  } else if (type == kE4M3) {
    const uint32_t w = pack4_e4m3(x);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[at + i] = static_cast<uint8_t>(w >> (8 * i));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) store_from_f32(p, type, at + i, x[i]);
  }
}

template <bool VEC>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a) {
  extern __shared__ float trig[];  // [token][half] cosines, then sines
  const int tid = threadIdx.x;
  const int t0 = (blockIdx.x / a.head_blocks) * a.per_block, hb = blockIdx.x % a.head_blocks;
  const int tokens = min(a.per_block, a.tokens - t0);
  float* sines = trig + a.per_block * a.half;
  for (int i = tid; i < tokens * a.half; i += kThreads) {
    const int t = i / a.half, pair = i - t * a.half;
    const int axis = (pair >= a.bound[0]) + (pair >= a.bound[1]) + (pair >= a.bound[2]);
    float s, c;
    sin_cos(a.pos[axis * a.pos_stride + t0 + t] * a.freq[pair], &s, &c);
    trig[i] = c;
    sines[i] = a.inverse ? -s : s;
  }
  __syncthreads();

  const int all = a.heads + 2 * a.kv_heads;
  // This workgroup's heads of the q, k, v row.
  const int h0 = static_cast<int>(static_cast<int64_t>(all) * hb / a.head_blocks);
  const int h1 = static_cast<int>(static_cast<int64_t>(all) * (hb + 1) / a.head_blocks);
  const int per_token = (h1 - h0) * static_cast<int>(a.items.d);
  for (int i = tid; i < tokens * per_token; i += kThreads) {
    const int t = i / per_token, j = i - t * per_token;
    const int hi = div_by(j, a.items);
    const int piece = j - hi * a.items.d;
    const int h = h0 + hi;
    const int which = h < a.heads ? 0 : h < a.heads + a.kv_heads ? 1 : 2;
    const int hd = which == 0 ? h : which == 1 ? h - a.heads : h - a.heads - a.kv_heads;
    const int64_t token = t0 + t;
    const uint8_t* src = a.src[which] + token * a.row[which] + hd * a.head[which];
    uint8_t* dst;
    int type;
    float scale = 1.f;
    if (which == 0) {
      dst = a.out + token * a.out_row + hd * a.out_head;
      type = a.out_type;
    } else {
      const int64_t slot = a.slots[token];
      if (slot < 0 || slot >= a.cache_slots) continue;
      const uint32_t page = div_by(static_cast<uint32_t>(slot), a.kv.page);
      const int64_t at = slot - static_cast<int64_t>(page) * a.kv.page.d;
      dst = which == 1 ? a.kv.k + page * a.kv.k_page + hd * a.kv.k_head + at * a.kv.k_tok
                       : a.kv.v + page * a.kv.v_page + hd * a.kv.v_head + at * a.kv.v_tok;
      type = a.cache_type;
      scale = which == 1 ? a.k_scale : a.v_scale;
    }
    // Pieces below half / 4 hold four pairs each; the rest is copied.
    const bool turns = which != 2 && piece * 4 < a.half;
    const bool split = turns && !a.adjacent;
    const int at0 = split ? piece * 4 : piece * 8, at1 = split ? a.half + piece * 4 : piece * 8 + 4;
    f32x4 x = load4<VEC>(src, a.x_type, at0), y = load4<VEC>(src, a.x_type, at1);
    if (turns) {
      const float* c = trig + t * a.half + piece * 4;
      const float* s = sines + t * a.half + piece * 4;
      if (split) {
        const f32x4 u = x, w = y;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = u[e] * c[e] - w[e] * s[e];
          y[e] = u[e] * s[e] + w[e] * c[e];
        }
      } else {
        const f32x4 u = x, w = y;
        x = f32x4{u.x * c[0] - u.y * s[0], u.x * s[0] + u.y * c[0],
                  u.z * c[1] - u.w * s[1], u.z * s[1] + u.w * c[1]};
        y = f32x4{w.x * c[2] - w.y * s[2], w.x * s[2] + w.y * c[2],
                  w.z * c[3] - w.w * s[3], w.z * s[3] + w.w * c[3]};
      }
    }
    if (scale != 1.f) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] /= scale;
        y[e] /= scale;
      }
    }
    store4<VEC>(dst, type, at0, x);
    store4<VEC>(dst, type, at1, y);
  }
}

// Sine and cosine in f64: the same reduction (2^-105 of pi/2 is left out), then
// Taylor sums whose first left-out terms are below 2^-60.
__device__ __forceinline__ void sin_cos(double angle, double* s, double* c) {
  const double n = rint(angle * 0.63661977236758134308);
  double x = fma(n, -1.57079632679489655800, angle);
  x = fma(n, -6.12323399573676603587e-17, x);
  const double y = x * x;
  double sn = 1.0 / 355687428096000.0;
  sn = fma(sn, y, -1.0 / 1307674368000.0);
  sn = fma(sn, y, 1.0 / 6227020800.0);
  sn = fma(sn, y, -1.0 / 39916800.0);
  sn = fma(sn, y, 1.0 / 362880.0);
  sn = fma(sn, y, -1.0 / 5040.0);
  sn = fma(sn, y, 1.0 / 120.0);
  sn = fma(sn, y, -1.0 / 6.0);
  sn = fma(sn * y, x, x);
  double cs = -1.0 / 6402373705728000.0;
  cs = fma(cs, y, 1.0 / 20922789888000.0);
  cs = fma(cs, y, -1.0 / 87178291200.0);
  cs = fma(cs, y, 1.0 / 479001600.0);
  cs = fma(cs, y, -1.0 / 3628800.0);
  cs = fma(cs, y, 1.0 / 40320.0);
  cs = fma(cs, y, -1.0 / 720.0);
  cs = fma(cs, y, 1.0 / 24.0);
  cs = fma(cs, y, -0.5);
  cs = fma(cs, y, 1.0);
  const int q = static_cast<int>(n - 4.0 * floor(n * 0.25));
  const double u = q & 1 ? cs : sn, w = q & 1 ? sn : cs;
  *s = q & 2 ? -u : u;
  *c = (q + 1) & 2 ? -w : w;
}

// The largest over each aligned group of 8 lanes.
__device__ __forceinline__ int lane8_max(int v) {
  v = max(v, dpp<kDppQuadSwap1>(v));
  v = max(v, dpp<kDppQuadSwap2>(v));
  return max(v, dpp<kDppRowHalfMirror>(v));
}

// |x| as f32, cut off with its last bit set where that loses anything: on the
// same side of every border between two codes, and never on one that x is not
// on. Below f32's normal numbers 0, above them the largest.
__device__ __forceinline__ float cut_to_f32(double x) {
  const uint32_t hi = static_cast<uint32_t>(__double2hiint(x)) & 0x7fffffffu, lo = static_cast<uint32_t>(__double2loint(x));
  const uint32_t bits = __builtin_amdgcn_alignbit(hi, lo, 29) - (896u << 23) | min(lo & 0x1fffffffu, 1u);
  const uint32_t small = hi < 0x38100000u ? 0u : bits;
  return __builtin_bit_cast(float, hi >= 0x47f00000u ? 0x7f7fffffu : small);
}

// Four elements to their codes (16 bits) and, in `power`, the exponent of the
// block that 8 threads next to each other have, or NaN's. A code depends on the
// side of a border that its value lies on, so the quotient by the scale is f64's:
// with one correction it is the number itself where that is one of f64, a border
// between two codes say.
__device__ __forceinline__ uint32_t codes_of(const double (&x)[4], float scale, double inverse, int* power) {
  double y[4] = {x[0], x[1], x[2], x[3]};
  auto largest = [&]() {
    int top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) top = max(top, static_cast<int>(__double2hiint(y[e]) & 0x7fffffff));
    return lane8_max(top);
  };
  int top;
  if (scale != 1.f) {
    const double d = scale;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const double q = x[e] * inverse;
      y[e] = fma(fma(-q, d, x[e]), inverse, q);
    }
    top = largest();
    if (__ballot(top >= 0x7ff00000)) {
      // (An infinity's correction is NaN.)
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = fabs(x[e]) < INFINITY ? y[e] : x[e];
      top = largest();
    }
  } else {
    top = largest();
  }
  // The largest |y| by its upper word: m * 2^E is below 7 * 2^e from e = E - 2 on
  // where m < 1.75, else from E - 1 on.
  const int e = min(max((top >> 20) - 1023 - 2 + ((top >> 18 & 3) == 3), -23), 13) + 127;
  *power = top > 0x7ff00000 ? 255 : e;
  float u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = copysignf(cut_to_f32(y[i]), __builtin_bit_cast(float, __double2hiint(x[i])));
  const uint32_t low = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, u[0], u[1], block_power(e), 0);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(low, u[2], u[3], block_power(e), 1);
}

// Eight elements: as they lie in memory, and as f32.
struct Raw8 {
  u32x4 a, b;  // b: of f32
};
__device__ __forceinline__ Raw8 load8(const uint8_t* p, int type, int at) {
  Raw8 r;
  r.a = *reinterpret_cast<const u32x4*>(p + at * (type == kF32 ? 4 : 2));
  r.b = u32x4{0, 0, 0, 0};
  if (type == kF32) r.b = *reinterpret_cast<const u32x4*>(p + at * 4 + 16);
  return r;
}
__device__ __forceinline__ void unpack8(const Raw8& r, int type, float (&x)[8]) {
  if (type == kF32) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t u = r.a[e], w = r.b[e];
      x[e] = __builtin_bit_cast(float, u);
      x[4 + e] = __builtin_bit_cast(float, w);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const f32x2 y = type == kBF16 ? unpack2<kBF16>(r.a[e]) : unpack2<kF16>(r.a[e]);
      x[2 * e] = y.x;
      x[2 * e + 1] = y.y;
    }
  }
}
__device__ __forceinline__ void store8(uint8_t* p, int type, int at, const float (&x)[8]) {
  if (type == kF32) {
    *reinterpret_cast<f32x4*>(p + at * 4) = f32x4{x[0], x[1], x[2], x[3]};
    *reinterpret_cast<f32x4*>(p + at * 4 + 16) = f32x4{x[4], x[5], x[6], x[7]};
  } else if (type == kBF16) {
    *reinterpret_cast<u32x4*>(p + at * 2) = u32x4{pack2<kBF16>(x[0], x[1]), pack2<kBF16>(x[2], x[3]),
                                                  pack2<kBF16>(x[4], x[5]), pack2<kBF16>(x[6], x[7])};
  } else {
    *reinterpret_cast<u32x4*>(p + at * 2) = u32x4{pack2<kF16>(x[0], x[1]), pack2<kF16>(x[2], x[3]),
                                                  pack2<kF16>(x[4], x[5]), pack2<kF16>(x[6], x[7])};
  }
}

// The append to a cache of 4 bits. The first workgroups turn q, as rope_kernel
// does (WIDE: 16 elements a thread, in 16-byte words). The others have some tokens'
// k and v each: a thread takes four elements, 8 threads next to each other a block
// of 32, whose power of two they agree on. k is turned in f64: the codes are those
// of the exact turn by f64's product pos * freq, but for values within a few 2^-53
// of |a| + |b|, the pair's elements, of a border between two codes. (That product
// is off by up to 2^-53 of the angle itself, 2^-36 where that is 2^17, as in every
// call here.) A partner element is loaded by both threads that need it; the second
// load is a cache hit.
//
// Measured: 8192 tokens (32 + 2 x 8 heads of 128, bf16, three axes, both scales not
// 1) 63 us, 2.8 TB/s, as the append to a bf16 cache; without k and v 44. What it
// waits for is the chain from positions to angles to stores. (Codes by seven f64
// comparisons each, a reciprocal in each thread and 8-byte words took 79.)
template <bool VEC, bool WIDE>
__global__ __launch_bounds__(kThreads) void rope_append4_kernel(RopeArgs a) {
  extern __shared__ double trig64[];
  const int tid = threadIdx.x;
  auto axis_of = [&](int pair) { return (pair >= a.bound[0]) + (pair >= a.bound[1]) + (pair >= a.bound[2]); };
  if (static_cast<int>(blockIdx.x) < a.q_blocks) {
    float* trig = reinterpret_cast<float*>(trig64);  // [token][half] cosines, then sines
    const int t0 = (blockIdx.x / a.head_blocks) * a.per_block, hb = blockIdx.x % a.head_blocks;
    const int tokens = min(a.per_block, a.tokens - t0);
    float* sines = trig + a.per_block * a.half;
    const int h0 = static_cast<int>(static_cast<int64_t>(a.heads) * hb / a.head_blocks);
    const int h1 = static_cast<int>(static_cast<int64_t>(a.heads) * (hb + 1) / a.head_blocks);
    const uint8_t* q = a.src[0] + t0 * a.row[0] + h0 * a.head[0];
    uint8_t* out = a.out + t0 * a.out_row + h0 * a.out_head;
    const int per_token = (h1 - h0) * static_cast<int>(a.items.d), items = tokens * per_token;
    // An item: 4 or 8 pairs of a head, or as many elements that are copied.
    constexpr int PAIRS = WIDE ? 8 : 4;
    struct Item {
      int t, piece, at0, at1;
      int64_t src, dst;
      bool turns, split;
    };
    auto item = [&](int i) {
      Item m;
      m.t = a.per_block == 1 ? 0 : i / per_token;
      const int j = i - m.t * per_token, hi = div_by(j, a.items);
      m.piece = j - hi * a.items.d;
      m.turns = m.piece * PAIRS < a.half;
      m.split = m.turns && !a.adjacent;
      m.at0 = m.piece * (m.split ? PAIRS : 2 * PAIRS);
      m.at1 = m.split ? a.half + m.at0 : m.at0 + PAIRS;
      m.src = m.t * a.row[0] + hi * a.head[0];
      m.dst = m.t * a.out_row + hi * a.out_head;
      return m;
    };
    Raw8 x0, x1;
    if constexpr (WIDE) {
      // The first item's loads are under way while the angles are worked out.
      const Item m = item(min(tid, items - 1));
      x0 = load8(q + m.src, a.x_type, m.at0);
      x1 = load8(q + m.src, a.x_type, m.at1);
    }
    for (int i = tid; i < tokens * a.half; i += kThreads) {
      const int t = i / a.half, pair = i - t * a.half;
      sin_cos(a.pos[axis_of(pair) * a.pos_stride + t0 + t] * a.freq[pair], &sines[i], &trig[i]);
    }
    __syncthreads();
    for (int i = tid; i < items; i += kThreads) {
      const Item m = item(i);
      float u[PAIRS], w[PAIRS];
      if constexpr (WIDE) {
        if (i != tid) {
          x0 = load8(q + m.src, a.x_type, m.at0);
          x1 = load8(q + m.src, a.x_type, m.at1);
        }
        unpack8(x0, a.x_type, u);
        unpack8(x1, a.x_type, w);
      } else {
        const f32x4 y = load4<VEC>(q + m.src, a.x_type, m.at0), z = load4<VEC>(q + m.src, a.x_type, m.at1);
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = y[e], w[e] = z[e];
      }
      if (m.turns) {
        const float* c = trig + m.t * a.half + m.piece * PAIRS;
        const float* s = sines + m.t * a.half + m.piece * PAIRS;
        if (m.split) {
#pragma unroll
          for (int e = 0; e < PAIRS; ++e) {
            const float x = u[e], y = w[e];
            u[e] = x * c[e] - y * s[e];
            w[e] = x * s[e] + y * c[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < PAIRS; e += 2) {
            const float x = u[e], y = u[e + 1], z = w[e], v = w[e + 1];
            const int p = e / 2, r = PAIRS / 2 + e / 2;
            u[e] = x * c[p] - y * s[p];
            u[e + 1] = x * s[p] + y * c[p];
            w[e] = z * c[r] - v * s[r];
            w[e + 1] = z * s[r] + v * c[r];
          }
        }
      }
      if constexpr (WIDE) {
        store8(out + m.dst, a.out_type, m.at0, u);
        store8(out + m.dst, a.out_type, m.at1, w);
      } else {
        store4<VEC>(out + m.dst, a.out_type, m.at0, f32x4{u[0], u[1], u[2], u[3]});
        store4<VEC>(out + m.dst, a.out_type, m.at1, f32x4{w[0], w[1], w[2], w[3]});
      }
    }
    return;
  }

  const int block = blockIdx.x - a.q_blocks;
  const int t0 = block / a.kv_parts * a.kv_block, part = block % a.kv_parts;
  const int tokens = min(a.kv_block, a.tokens - t0);
  double* sines = trig64 + a.kv_block * a.half;
  for (int i = tid; i < tokens * a.half; i += kThreads) {
    const int t = i / a.half, pair = i - t * a.half;
    sin_cos(a.pos[axis_of(pair) * a.pos_stride + t0 + t] * a.freq[pair], &sines[i], &trig64[i]);
  }
  __syncthreads();
  const int h0 = static_cast<int>(static_cast<int64_t>(a.kv_heads) * part / a.kv_parts);
  const int h1 = static_cast<int>(static_cast<int64_t>(a.kv_heads) * (part + 1) / a.kv_parts);
  // 8 | dim / 4: the 8 threads of a block are in one wave's row and take every
  // turn of a loop together.
  const int quarters = a.quarters.d, items = (h1 - h0) * quarters;
  // A thread's four elements of k, those that k's turn needs besides, and of v.
  struct Own {
    f32x4 k, other, v;
  };
  auto load = [&](int t, int i) {
    const int64_t token = t0 + t;
    const int head = div_by(i, a.quarters), at = (i - head * quarters) * 4;
    const uint8_t* k = a.src[1] + token * a.row[1] + (h0 + head) * a.head[1];
    Own o;
    o.k = load4<VEC>(k, a.x_type, at);
    o.v = load4<VEC>(a.src[2] + token * a.row[2] + (h0 + head) * a.head[2], a.x_type, at);
    o.other = o.k;
    if (!a.adjacent && at < 2 * a.half) o.other = load4<VEC>(k, a.x_type, at >= a.half ? at - a.half : at + a.half);
    return o;
  };
  // The next token's elements load while one's are worked on.
  Own next = load(0, min(tid, items - 1));
  for (int t = 0; t < tokens; ++t) {
    Own now = next;
    next = load(min(t + 1, tokens - 1), min(tid, items - 1));
    const int64_t slot = a.slots[t0 + t];
    if (slot < 0 || slot >= a.cache_slots) continue;  // workgroup-uniform
    const uint32_t page = div_by(static_cast<uint32_t>(slot), a.kv.page);
    const int64_t in = slot - static_cast<int64_t>(page) * a.kv.page.d;
    uint8_t* k_at = a.kv.k + page * a.kv.k_page + in * a.kv.k_tok + h0 * a.kv.k_head;
    uint8_t* v_at = a.kv.v + page * a.kv.v_page + in * a.kv.v_tok + h0 * a.kv.v_head;
    uint8_t* ke_at = a.exps.k + page * a.exps.k_page + in * a.exps.k_tok + h0 * a.exps.k_head;
    uint8_t* ve_at = a.exps.v + page * a.exps.v_page + in * a.exps.v_tok + h0 * a.exps.v_head;
    const double* c = trig64 + t * a.half;
    const double* s = sines + t * a.half;
    for (int i = tid; i < items; i += kThreads) {
      if (i != tid) now = load(t, i);
      const int head = div_by(i, a.quarters), at = (i - head * quarters) * 4;
      const f32x4 own = now.k, other = now.other, v = now.v;
      double x[4] = {own.x, own.y, own.z, own.w};
      if (at < 2 * a.half) {
        if (a.adjacent) {
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const int pair = (at + e) / 2;
            const double u = x[e], w = x[e + 1];
            x[e] = u * c[pair] - w * s[pair];
            x[e + 1] = u * s[pair] + w * c[pair];
          }
        } else {
          // The second half's elements turn by the sine as they are, the first
          // half's by its negative.
          const bool second = at >= a.half;
          const int first = second ? at - a.half : at;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const double turn = s[first + e] * static_cast<double>(other[e]);
            x[e] = x[e] * c[first + e] + (second ? turn : -turn);
          }
        }
      }
      int power;
      const uint32_t codes = codes_of(x, a.k_scale, a.k_inv, &power);
      *reinterpret_cast<uint16_t*>(k_at + head * a.kv.k_head + at / 2) = static_cast<uint16_t>(codes);
      if (at % 32 == 0) ke_at[head * a.exps.k_head + at / 32] = static_cast<uint8_t>(power);
      const double w[4] = {v.x, v.y, v.z, v.w};
      const uint32_t v_codes = codes_of(w, a.v_scale, a.v_inv, &power);
      *reinterpret_cast<uint16_t*>(v_at + head * a.kv.v_head + at / 2) = static_cast<uint16_t>(v_codes);
      if (at % 32 == 0) ve_at[head * a.exps.v_head + at / 32] = static_cast<uint8_t>(power);
    }
  }
}

// Whether four elements at a multiple of four into any row are one aligned
// word.
bool rows_aligned(const RowsView& r) {
  const uintptr_t w = static_cast<uintptr_t>(4 * elem_bytes(r.type));
  return reinterpret_cast<uintptr_t>(r.data) % w == 0 && r.row % 4 == 0 && r.head % 4 == 0;
}

// Launches of whole tokens whose threads 32 bits count.
hipError_t launch_append4(RopeArgs a, bool vec, bool wide, int64_t tokens, int64_t heads, hipStream_t stream) {
  const int64_t most = int64_t{1} << 21;
  if (wide) a.items = fast_div(static_cast<uint32_t>(a.dim / 16));
  const int64_t q_items = heads * a.items.d, kv_items = static_cast<int64_t>(a.kv_heads) * a.quarters.d;
  for (int64_t left = tokens; left > 0; left -= most) {
    const int64_t now = std::min(left, most);
    a.tokens = static_cast<int>(now);
    const bool several = now >= 1024 && q_items < kThreads;
    a.per_block = several ? static_cast<int>(std::min<int64_t>(kMaxTokens, kThreads / q_items)) : 1;
    const int64_t q_groups = (now + a.per_block - 1) / a.per_block;
    // (As many workgroups of a token as its items fill, fewer where tokens do.)
    auto shared_by = [](int64_t groups, int64_t of_heads, int64_t items) {
      return static_cast<int>(
          std::clamp<int64_t>(1024 / groups, 1, std::min<int64_t>(of_heads, (items + kThreads - 1) / kThreads)));
    };
    a.head_blocks = shared_by(q_groups, heads, q_items);
    // Four tokens' sines and cosines keep all threads busy; few tokens are
    // shared by workgroups instead.
    a.kv_block = now >= 4096 ? kMaxTokens : 1;
    const int64_t kv_groups = (now + a.kv_block - 1) / a.kv_block;
    a.kv_parts = shared_by(kv_groups, a.kv_heads, kv_items);
    a.q_blocks = static_cast<int>(q_groups * a.head_blocks);
    const size_t lds = std::max<size_t>(a.per_block * sizeof(float), a.kv_block * sizeof(double)) * a.half * 2;
    const dim3 grid(static_cast<uint32_t>(a.q_blocks + kv_groups * a.kv_parts));
    if (wide)
      rope_append4_kernel<true, true><<<grid, dim3(kThreads), lds, stream>>>(a);
    else if (vec)
      rope_append4_kernel<true, false><<<grid, dim3(kThreads), lds, stream>>>(a);
    else
      rope_append4_kernel<false, false><<<grid, dim3(kThreads), lds, stream>>>(a);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    for (int i = 0; i < 3; ++i) a.src[i] += now * a.row[i];
    a.out += now * a.out_row;
    a.pos += now;
    a.slots += now;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_rope(const RowsView& out, const RowsView& q, const RowsView* k, const RowsView* v,
                       int64_t tokens, int64_t heads, int64_t dim, const xq_kv* kv,
                       const int32_t* pos, int64_t pos_stride, const xq_rope_freqs& rope,
                       bool inverse, const int64_t* slots, hipStream_t stream) {
  RopeArgs a = {};
  const int xb = elem_bytes(q.type);
  a.src[0] = static_cast<const uint8_t*>(q.data);
  a.row[0] = q.row * xb;
  a.head[0] = q.head * xb;
  a.out = static_cast<uint8_t*>(out.data);
  a.out_row = out.row * elem_bytes(out.type);
  a.out_head = out.head * elem_bytes(out.type);
  a.out_type = out.type;
  a.x_type = q.type;
  bool vec = rope.rot % 8 == 0 && rows_aligned(q) && rows_aligned(out);
  if (kv) {
    const RowsView* kvs[2] = {k, v};
    for (int i = 0; i < 2; ++i) {
      a.src[1 + i] = static_cast<const uint8_t*>(kvs[i]->data);
      a.row[1 + i] = kvs[i]->row * xb;
      a.head[1 + i] = kvs[i]->head * xb;
      vec = vec && rows_aligned(*kvs[i]);
    }
    a.kv = kv_view(*kv);
    a.exps = exp_view(*kv);
    a.kv_heads = static_cast<int>(kv->kv_heads);
    a.cache_type = kv->dtype;
    a.cache_slots = kv->pages * kv->page;
    a.k_scale = kv->k_scale;
    a.v_scale = kv->v_scale;
    a.k_inv = 1.0 / kv->k_scale;
    a.v_inv = 1.0 / kv->v_scale;
    a.slots = slots;
  }
  a.pos = pos;
  a.pos_stride = pos_stride;
  a.freq = rope.freq;
  a.tokens = static_cast<int>(tokens);
  a.heads = static_cast<int>(heads);
  a.dim = static_cast<int>(dim);
  a.half = static_cast<int>(rope.rot / 2);
  a.adjacent = static_cast<int>(rope.adjacent);
  a.inverse = inverse;
  int first = 0;
  for (int i = 0; i < 3; ++i) {
    first += static_cast<int>(rope.sections[i]);
    a.bound[i] = i + 1 < rope.axes ? first : a.half;
  }
  a.items = fast_div(static_cast<uint32_t>(dim / 8));
  a.quarters = fast_div(static_cast<uint32_t>(dim / 4));
  const bool four = kv && kv->dtype == kE2M1;
  // One token a workgroup, its heads shared between several where tokens are
  // few. More tokens only where a token's items leave more than a quarter of
  // the threads without work and there are tokens enough: 8192 tokens of 64
  // heads of 128 take 63 us with one token, 69 and 78 with two and four; 4500
  // tokens of 24 heads of 96 (288 items) 16.1 with one, 14.8 with two.
  const int64_t items = (heads + 2 * a.kv_heads) * (dim / 8);
  a.per_block = 1;
  auto busy = [&](int64_t n) { return 4 * n * items >= 3 * ((n * items + kThreads - 1) / kThreads) * kThreads; };
  while (a.per_block < kMaxTokens && !busy(a.per_block) && tokens >= 1024 * (a.per_block + 1) &&
         (a.per_block + 1) * a.half <= 2048)
    ++a.per_block;
  const int64_t blocks = (tokens + a.per_block - 1) / a.per_block;
  a.head_blocks = static_cast<int>(std::clamp<int64_t>(1024 / blocks, 1, (items + kThreads - 1) / kThreads));
  if (four) {
    // q and its output in 16-byte words of eight 16-bit elements: their rows lie
    // so, and a half of the pairs is a multiple of eight.
    auto words = [](const RowsView& r) {
      return reinterpret_cast<uintptr_t>(r.data) % 16 == 0 && r.row % 8 == 0 && r.head % 8 == 0;
    };
    return launch_append4(a, vec, vec && a.half % 8 == 0 && words(q) && words(out), tokens, heads, stream);
  }
  const size_t lds = static_cast<size_t>(a.per_block) * a.half * 2 * sizeof(float);
  // A launch's threads are counted in 32 bits, and more wrap round without an
  // error: so many workgroups (of 2^24 - 1) take the tokens in several launches.
  const int64_t most = int64_t{1} << 23;
  for (int64_t left = blocks; left > 0; left -= most) {
    const int64_t now = std::min(left, most), done = now * a.per_block;
    a.tokens = static_cast<int>(std::min(done, tokens));
    const dim3 grid(static_cast<uint32_t>(now * a.head_blocks));
    if (vec)
      rope_kernel<true><<<grid, dim3(kThreads), lds, stream>>>(a);
    else
      rope_kernel<false><<<grid, dim3(kThreads), lds, stream>>>(a);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    tokens -= done;
    for (int i = 0; i < 3; ++i)
      if (a.src[i]) a.src[i] += done * a.row[i];
    a.out += done * a.out_row;
    a.pos += done;
    if (a.slots) a.slots += done;
  }
  return hipSuccess;
}

}  // namespace xq
