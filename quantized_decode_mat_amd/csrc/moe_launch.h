// moe_launch.h — internal launchers of the mixture-of-experts kernels, called
// by the C ABI (moe_api.cpp) after it has validated every argument.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace xq {

// Strides of x and y in elements.
size_t moe_route_workspace_bytes(int64_t tokens, int64_t experts);
hipError_t launch_moe_route(int32_t* ids, float* weights, const void* x, int x_type, int64_t x_row,
                            const void* router, int router_type, const float* bias, int64_t tokens,
                            int64_t experts, int64_t used, int64_t k, bool sigmoid, bool normalize,
                            float scale, void* ws, hipStream_t stream);
size_t moe_q4k_workspace_bytes(int64_t tokens, int64_t used, int64_t hidden, int64_t ffn);
hipError_t launch_moe_q4k(void* y, int64_t y_row, const void* x, int64_t x_row, int io, const void* gate,
                          const void* up, const void* down, const int32_t* ids, const float* weights,
                          int64_t tokens, int64_t used, int64_t experts, int64_t hidden, int64_t ffn, void* ws,
                          hipStream_t stream);

}  // namespace xq
