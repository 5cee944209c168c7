// moe_api.cpp — the C ABI of the mixture-of-experts layer (include/xq.h). Gates
// in the order of xq_api.cpp: null pointers, shapes, alignment, then the
// device; nothing is launched after a refusal.
#include <cmath>

#include "moe_launch.h"
#include "xq_host.h"

using namespace xq::host;

namespace {

constexpr int64_t kMaxPairs = 512;
constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxWidth = 32768;

int type_bytes(int32_t t) { return t == XQ_F32 ? 4 : 2; }
bool row_type(int32_t t) { return t == XQ_F32 || t == XQ_BF16 || t == XQ_F16; }

xq_status check_route(int64_t tokens, int64_t experts) {
  if (tokens < 1 || tokens > kMaxPairs)
    return fail(XQ_E_SHAPE, "tokens=%lld outside 1..512", (long long)tokens);
  if (experts < 1 || experts > kMaxExperts)
    return fail(XQ_E_SHAPE, "experts=%lld outside 1..1024", (long long)experts);
  return XQ_OK;
}

xq_status check_layer(int64_t tokens, int64_t used, int64_t hidden, int64_t ffn) {
  if (tokens < 1 || used < 1 || tokens > kMaxPairs || used > kMaxPairs / tokens)
    return fail(XQ_E_SHAPE, "tokens*used = %lld*%lld outside 1..512", (long long)tokens, (long long)used);
  if (hidden < 256 || hidden > kMaxWidth || hidden % 256)
    return fail(XQ_E_SHAPE, "hidden=%lld not a multiple of 256 in 256..32768", (long long)hidden);
  if (ffn < 256 || ffn > kMaxWidth || ffn % 256)
    return fail(XQ_E_SHAPE, "ffn=%lld not a multiple of 256 in 256..32768", (long long)ffn);
  return XQ_OK;
}

// Strides of rows: 0 where there is one row, else not below the row.
xq_status check_row(int64_t row, int64_t rows, int64_t width, const char* what) {
  if (row < (rows > 1 ? width : 0) || row > (1LL << 40))
    return fail(XQ_E_SHAPE, "%s row stride=%lld below its width=%lld", what, (long long)row, (long long)width);
  return XQ_OK;
}

}  // namespace

extern "C" {

size_t xq_moe_route_workspace_bytes(int64_t tokens, int64_t experts) {
  return check_route(tokens, experts) == XQ_OK ? xq::moe_route_workspace_bytes(tokens, experts) : 0;
}

xq_status xq_moe_route(int32_t *ids, float *weights, const void *x, int32_t x_type, int64_t x_row,
                       const void *router, int32_t router_type, const float *bias, int64_t tokens,
                       int64_t experts, int64_t used, int64_t K, int32_t score, int32_t normalize,
                       float scale, void *workspace, size_t workspace_bytes, void *stream) {
  if (!ids) return fail(XQ_E_NULL, "ids is NULL");
  if (!weights) return fail(XQ_E_NULL, "weights is NULL");
  if (!x) return fail(XQ_E_NULL, "x is NULL");
  if (!router) return fail(XQ_E_NULL, "router is NULL");
  if (!row_type(x_type)) return fail(XQ_E_SHAPE, "x_type=%d is none of XQ_F32, XQ_BF16, XQ_F16", x_type);
  if (!row_type(router_type))
    return fail(XQ_E_SHAPE, "router_type=%d is none of XQ_F32, XQ_BF16, XQ_F16", router_type);
  if (xq_status s = check_route(tokens, experts)) return s;
  if (used < 1 || used > 64 || used > experts)
    return fail(XQ_E_SHAPE, "used=%lld outside 1..64 or above experts=%lld", (long long)used, (long long)experts);
  if (K < 8 || K > XQ_MAX_K || K % 8)
    return fail(XQ_E_SHAPE, "K=%lld not a multiple of 8 in 8..%d", (long long)K, XQ_MAX_K);
  if (score != XQ_SOFTMAX && score != XQ_SIGMOID)
    return fail(XQ_E_SHAPE, "score=%d is neither XQ_SOFTMAX nor XQ_SIGMOID", score);
  if (normalize != 0 && normalize != 1) return fail(XQ_E_SHAPE, "normalize=%d is neither 0 nor 1", normalize);
  if (!std::isfinite(scale)) return fail(XQ_E_SHAPE, "scale=%g not finite", scale);
  if (xq_status s = check_row(x_row, tokens, K, "x")) return s;
  const size_t need = xq::moe_route_workspace_bytes(tokens, experts);
  if (xq_status s = check_workspace(workspace, workspace_bytes, need, "xq_moe_route_workspace_bytes")) return s;
  if (!aligned(ids, 4)) return fail(XQ_E_ALIGN, "ids not 4-byte aligned");
  if (!aligned(weights, 4)) return fail(XQ_E_ALIGN, "weights not 4-byte aligned");
  if (!aligned(x, 16) || x_row * type_bytes(x_type) % 16) return fail(XQ_E_ALIGN, "x or its rows not 16-byte aligned");
  if (!aligned(router, 16)) return fail(XQ_E_ALIGN, "router not 16-byte aligned");
  if (bias && !aligned(bias, 4)) return fail(XQ_E_ALIGN, "bias not 4-byte aligned");
  if (xq_status s = check_workspace_align(workspace, need)) return s;
  if (xq_status s = check_device()) return s;
  return launched(xq::launch_moe_route(ids, weights, x, x_type, x_row, router, router_type, bias, tokens, experts,
                                       used, K, score == XQ_SIGMOID, normalize == 1, scale, workspace,
                                       static_cast<hipStream_t>(stream)),
                  "xq_moe_route");
}

size_t xq_moe_q4k_workspace_bytes(int64_t tokens, int64_t used, int64_t hidden, int64_t ffn) {
  return check_layer(tokens, used, hidden, ffn) == XQ_OK ? xq::moe_q4k_workspace_bytes(tokens, used, hidden, ffn) : 0;
}

xq_status xq_moe_q4k(void *y, int64_t y_row, const void *x, int64_t x_row, int32_t io,
                     const void *gate, const void *up, const void *down, const int32_t *ids,
                     const float *weights, int64_t tokens, int64_t used, int64_t experts,
                     int64_t hidden, int64_t ffn, void *workspace, size_t workspace_bytes,
                     void *stream) {
  if (!y) return fail(XQ_E_NULL, "y is NULL");
  if (!x) return fail(XQ_E_NULL, "x is NULL");
  if (!gate) return fail(XQ_E_NULL, "gate is NULL");
  if (!up) return fail(XQ_E_NULL, "up is NULL");
  if (!down) return fail(XQ_E_NULL, "down is NULL");
  if (!ids) return fail(XQ_E_NULL, "ids is NULL");
  if (!weights) return fail(XQ_E_NULL, "weights is NULL");
  if (!row_type(io)) return fail(XQ_E_SHAPE, "io=%d is none of XQ_F32, XQ_BF16, XQ_F16", io);
  if (xq_status s = check_layer(tokens, used, hidden, ffn)) return s;
  if (experts < 1 || experts > kMaxExperts)
    return fail(XQ_E_SHAPE, "experts=%lld outside 1..1024", (long long)experts);
  if (xq_status s = check_row(y_row, tokens, hidden, "y")) return s;
  if (xq_status s = check_row(x_row, tokens, hidden, "x")) return s;
  const size_t need = xq::moe_q4k_workspace_bytes(tokens, used, hidden, ffn);
  if (xq_status s = check_workspace(workspace, workspace_bytes, need, "xq_moe_q4k_workspace_bytes")) return s;
  if (!aligned(y, type_bytes(io))) return fail(XQ_E_ALIGN, "y not aligned to its elements");
  if (!aligned(x, 16) || x_row * type_bytes(io) % 16) return fail(XQ_E_ALIGN, "x or its rows not 16-byte aligned");
  if (!aligned(gate, 16)) return fail(XQ_E_ALIGN, "gate not 16-byte aligned");
  if (!aligned(up, 16)) return fail(XQ_E_ALIGN, "up not 16-byte aligned");
  if (!aligned(down, 16)) return fail(XQ_E_ALIGN, "down not 16-byte aligned");
  if (!aligned(ids, 4)) return fail(XQ_E_ALIGN, "ids not 4-byte aligned");
  if (!aligned(weights, 4)) return fail(XQ_E_ALIGN, "weights not 4-byte aligned");
  if (xq_status s = check_workspace_align(workspace, need)) return s;
  if (xq_status s = check_device()) return s;
  return launched(xq::launch_moe_q4k(y, y_row, x, x_row, io, gate, up, down, ids, weights, tokens, used, experts,
                                     hidden, ffn, workspace, static_cast<hipStream_t>(stream)),
                  "xq_moe_q4k");
}

}  // extern "C"
