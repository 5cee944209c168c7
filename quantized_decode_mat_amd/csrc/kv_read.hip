// kv_read.hip — tokens of a paged cache as values.
//
//   k_out[t][h] = k[slots[t]][h] * k_scale, v the same.
//
// What bounds it: bytes, mostly those written, and for few tokens the launch. A
// thread takes eight dims of a row of k or v: four bytes of a 4-bit cache (its
// values are exact in bf16, and so in f32), one or two 16-byte stores.
//
// Measured: 8192 tokens of 2 x 8 heads of 128 dims, 4 bits to bf16: 13.7 us, 43 MB
// read and written; 8 tokens 3.2 us.
#include "kv_device.h"
#include "kv_launch.h"
#include "kv_view.h"

namespace xq {
namespace {

constexpr int kThreads = 256;

struct ReadArgs {
  KvView kv;
  ExpView exps;
  uint8_t* out[2];
  int64_t row[2], head[2];  // bytes
  const int64_t* slots;
  int64_t cache_slots, items;
  FastDiv pieces, kv_heads;  // dim / 8
  int type, out_type, wide;  // wide: outputs take 16-byte stores
  float scale[2];
};

__device__ __forceinline__ f32x2 pair_of(u32x4 w, int i, bool bf16) {
  return bf16 ? unpack2<kBF16>(w[i]) : unpack2<kF16>(w[i]);
}

__global__ __launch_bounds__(kThreads) void read_kernel(ReadArgs a) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= a.items) return;
  // (token, k or v, head, piece), the last fastest; a token's fit 32 bits.
  const uint32_t per = 2 * a.kv_heads.d * a.pieces.d;
  const int64_t token = i / per;
  const uint32_t rest = static_cast<uint32_t>(i - token * per), row_of = div_by(rest, a.pieces);
  const int d0 = static_cast<int>(rest - row_of * a.pieces.d) * 8;
  const int which = row_of >= a.kv_heads.d, head = static_cast<int>(row_of - (which ? a.kv_heads.d : 0));
  const int64_t slot = a.slots[token];
  float x[8] = {};
  if (slot >= 0 && slot < a.cache_slots) {
    const uint32_t page = div_by(static_cast<uint32_t>(slot), a.kv.page);
    const int64_t in = slot - static_cast<int64_t>(page) * a.kv.page.d;
    const uint8_t* row = which ? a.kv.v + page * a.kv.v_page + head * a.kv.v_head + in * a.kv.v_tok
                               : a.kv.k + page * a.kv.k_page + head * a.kv.k_head + in * a.kv.k_tok;
    u32x4 w = {};
    bool bf16 = a.type == kBF16;
    if (a.type == kE2M1) {
      const uint8_t* exps = which ? a.exps.v + page * a.exps.v_page + head * a.exps.v_head + in * a.exps.v_tok
                                  : a.exps.k + page * a.exps.k_page + head * a.exps.k_head + in * a.exps.k_tok;
      w = widen8<kBF16>(*reinterpret_cast<const uint32_t*>(row + d0 / 2), block_power(exps[d0 / 32]));
      bf16 = true;
    } else if (a.type == kE4M3) {
      const u32x2 r = *reinterpret_cast<const u32x2*>(row + d0);
      const u32x2 u = widen4<kBF16>(r.x), v = widen4<kBF16>(r.y);
      w = u32x4{u.x, u.y, v.x, v.y};
      bf16 = true;
    } else {
      w = *reinterpret_cast<const u32x4*>(row + d0 * 2);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const f32x2 p = pair_of(w, e, bf16);
      x[2 * e] = p.x * a.scale[which];
      x[2 * e + 1] = p.y * a.scale[which];
    }
  }
  uint8_t* out = (which ? a.out[1] : a.out[0]) + token * a.row[which] + head * a.head[which];
  if (!a.wide) {
#pragma unroll
    for (int e = 0; e < 8; ++e) store_from_f32(out, a.out_type, d0 + e, x[e]);
  } else if (a.out_type == kF32) {
    *reinterpret_cast<f32x4*>(out + d0 * 4) = f32x4{x[0], x[1], x[2], x[3]};
    *reinterpret_cast<f32x4*>(out + d0 * 4 + 16) = f32x4{x[4], x[5], x[6], x[7]};
  } else if (a.out_type == kBF16) {
    *reinterpret_cast<u32x4*>(out + d0 * 2) = u32x4{pack2<kBF16>(x[0], x[1]), pack2<kBF16>(x[2], x[3]),
                                                    pack2<kBF16>(x[4], x[5]), pack2<kBF16>(x[6], x[7])};
  } else {
    *reinterpret_cast<u32x4*>(out + d0 * 2) = u32x4{pack2<kF16>(x[0], x[1]), pack2<kF16>(x[2], x[3]),
                                                    pack2<kF16>(x[4], x[5]), pack2<kF16>(x[6], x[7])};
  }
}

}  // namespace

hipError_t launch_cache_read(const RowsView& k_out, const RowsView& v_out, const xq_kv& kv,
                             const int64_t* slots, int64_t tokens, hipStream_t stream) {
  ReadArgs a = {};
  a.kv = kv_view(kv);
  a.exps = exp_view(kv);
  const RowsView* outs[2] = {&k_out, &v_out};
  a.wide = 1;
  for (int i = 0; i < 2; ++i) {
    const int ob = elem_bytes(outs[i]->type);
    a.out[i] = static_cast<uint8_t*>(outs[i]->data);
    a.row[i] = outs[i]->row * ob;
    a.head[i] = outs[i]->head * ob;
    if (reinterpret_cast<uintptr_t>(a.out[i]) % 16 || a.row[i] % 16 || a.head[i] % 16) a.wide = 0;
  }
  a.slots = slots;
  a.cache_slots = kv.pages * kv.page;
  a.pieces = fast_div(static_cast<uint32_t>(kv.dim / 8));
  a.kv_heads = fast_div(static_cast<uint32_t>(kv.kv_heads));
  a.type = kv.dtype;
  a.out_type = k_out.type;
  a.scale[0] = kv.k_scale;
  a.scale[1] = kv.v_scale;
  // A launch's threads are counted in 32 bits: more take several launches, of
  // whole tokens.
  const int64_t per = 2 * kv.kv_heads * (kv.dim / 8), most = ((int64_t{1} << 31) - kThreads) / per;
  for (int64_t left = tokens; left > 0; left -= most) {
    const int64_t now = left < most ? left : most;
    a.items = now * per;
    read_kernel<<<dim3(static_cast<uint32_t>((a.items + kThreads - 1) / kThreads)), dim3(kThreads), 0, stream>>>(a);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    for (int i = 0; i < 2; ++i) a.out[i] += now * a.row[i];
    a.slots += now;
  }
  return hipSuccess;
}

}  // namespace xq
