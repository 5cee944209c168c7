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

// Whether four elements at a multiple of four into any row are one aligned
// word.
bool rows_aligned(const RowsView& r) {
  const uintptr_t w = static_cast<uintptr_t>(4 * elem_bytes(r.type));
  return reinterpret_cast<uintptr_t>(r.data) % w == 0 && r.row % 4 == 0 && r.head % 4 == 0;
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
    const int eb = elem_bytes(kv->dtype);
    a.kv = KvView{static_cast<uint8_t*>(kv->k), static_cast<uint8_t*>(kv->v),
                  kv->k_stride[1] * eb, kv->k_stride[2] * eb, kv->k_stride[3] * eb,
                  kv->v_stride[1] * eb, kv->v_stride[2] * eb, kv->v_stride[3] * eb,
                  fast_div(static_cast<uint32_t>(kv->page)), static_cast<int>(kv->pages)};
    a.kv_heads = static_cast<int>(kv->kv_heads);
    a.cache_type = kv->dtype;
    a.cache_slots = kv->pages * kv->page;
    a.k_scale = kv->k_scale;
    a.v_scale = kv->v_scale;
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
