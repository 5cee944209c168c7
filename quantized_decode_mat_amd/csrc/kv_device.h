// kv_device.h — device helpers shared by the kernels of the paged cache:
// 16-bit vectors and their matrix instructions, conversions, the cache's
// addressing.
#pragma once

#include "xq_device.h"

namespace xq {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// The element types of the C ABI (XQ_F32, ...).
enum ElemType : int { kF32 = 0, kBF16 = 1, kF16 = 2, kE4M3 = 3 };

__host__ __device__ constexpr int elem_bytes(int t) { return t == kF32 ? 4 : t == kE4M3 ? 1 : 2; }

// x / d for 0 <= x < 2^31: multiplier floor(2^(31+s)/d) + 1 with
// s = ceil(log2 d). Its excess over 2^(31+s)/d is at most 1, so the quotient's
// is below x / 2^(31+s) < 1/d: never enough to pass the next whole number.
struct FastDiv {
  uint32_t d, m, s;
};
inline FastDiv fast_div(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  return FastDiv{d, d == 1 ? 0x80000001u : static_cast<uint32_t>(((1ull << (31 + s)) / d) + 1), s};
}
__device__ __forceinline__ uint32_t div_by(uint32_t x, const FastDiv& f) {
  return static_cast<uint32_t>((static_cast<uint64_t>(x) * f.m) >> (31 + f.s));
}

// Two f32 rounded to the nearest 16-bit value, the first in the low half.
template <int T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const f32x2 v = {a, b};
  if constexpr (T == kBF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
  else return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}
template <int T>
__device__ __forceinline__ f32x2 unpack2(uint32_t w) {
  if constexpr (T == kBF16)
    return f32x2{__builtin_bit_cast(float, w << 16), __builtin_bit_cast(float, w & 0xffff0000u)};
  else
    return __builtin_convertvector(__builtin_bit_cast(f16x2, w), f32x2);
}

// Four 8-bit values (one dword) as four 16-bit ones: exact in either type.
template <int T>
__device__ __forceinline__ u32x2 widen4(uint32_t w) {
  if constexpr (T == kBF16)
    return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true))};
  else
    return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true))};
}

// 16x16x32: A row / B column l % 16, 8 of the 32 from 8 * (l / 16); D column
// l % 16, rows 4 * (l / 16) + i.
template <int T>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (T == kBF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
// 32x32x16: A row / B column l % 32, 8 of the 16 from 8 * (l / 32); D column
// l % 32, rows 8 * (i / 4) + 4 * (l / 32) + i % 4.
template <int T>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (T == kBF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Element i of a row of type t as f32, and back (one rounding).
__device__ __forceinline__ float load_as_f32(const uint8_t* p, int t, int64_t i) {
  if (t == kF32) return reinterpret_cast<const float*>(p)[i];
  const uint32_t w = reinterpret_cast<const uint16_t*>(p)[i];
  return t == kBF16 ? unpack2<kBF16>(w).x : unpack2<kF16>(w).x;
}
__device__ __forceinline__ void store_from_f32(uint8_t* p, int t, int64_t i, float v) {
  if (t == kF32) {
    reinterpret_cast<float*>(p)[i] = v;
  } else {
    reinterpret_cast<uint16_t*>(p)[i] =
        static_cast<uint16_t>(t == kBF16 ? pack2<kBF16>(v, 0.f) : pack2<kF16>(v, 0.f));
  }
}

// One layer of a paged cache as a kernel sees it; strides in bytes.
struct KvView {
  uint8_t* k;
  uint8_t* v;
  int64_t k_page, k_head, k_tok, v_page, v_head, v_tok;
  FastDiv page;
  int pages;
};

}  // namespace xq
