// kv_view.h — a layer of the C ABI's cache as the kernels see it.
#pragma once

#include "kv_device.h"
#include "kv_launch.h"

namespace xq {

inline KvView kv_view(const xq_kv& kv) {
  auto at = [&](const int64_t* stride, int i) { return cache_bytes(stride[i], kv.dtype); };
  return KvView{static_cast<uint8_t*>(kv.k), static_cast<uint8_t*>(kv.v),
                at(kv.k_stride, 1), at(kv.k_stride, 2), at(kv.k_stride, 3),
                at(kv.v_stride, 1), at(kv.v_stride, 2), at(kv.v_stride, 3),
                fast_div(static_cast<uint32_t>(kv.page)), static_cast<int>(kv.pages)};
}

inline ExpView exp_view(const xq_kv& kv) {
  if (kv.dtype != XQ_E2M1) return ExpView{};
  return ExpView{static_cast<uint8_t*>(kv.k_exp), static_cast<uint8_t*>(kv.v_exp),
                 kv.k_exp_stride[1], kv.k_exp_stride[2], kv.k_exp_stride[3],
                 kv.v_exp_stride[1], kv.v_exp_stride[2], kv.v_exp_stride[3]};
}

}  // namespace xq
