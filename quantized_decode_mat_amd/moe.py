"""Python binding of the mixture-of-experts layer's calls (include/xq.h): the
router, and the chosen experts' feed-forward on Q4_K weights. Each call checks
on the host that its tensors are device tensors of the types and shapes it
reads and writes; ids and weights stay on the device.
"""

from __future__ import annotations

import torch

from .kv import _ROW, _check, _ints, _raw_stream, _workspace, lib

XQ_SOFTMAX, XQ_SIGMOID = range(2)
_SCORES = {"softmax": XQ_SOFTMAX, "sigmoid": XQ_SIGMOID}


def _matrix(t, what: str, index: int):
    """(pointer, type, row stride) of [rows, columns]."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s: expected a torch.Tensor" % what)
    kind, st = _ROW.get(t.dtype), t.stride()
    if kind is None:
        raise ValueError("%s: %s is not supported" % (what, t.dtype))
    if t.get_device() != index or len(st) != 2 or st[1] != 1:
        raise ValueError("%s: expected [rows, columns] with contiguous columns on device %d" % (what, index))
    return t.data_ptr(), kind, st[0] if t.shape[0] != 1 else 0


def _index(x):
    index = x.get_device() if isinstance(x, torch.Tensor) else -1
    if index < 0:
        raise ValueError("x: must be a device tensor")
    return index


def _choice(ids, weights, tokens: int, index: int):
    """(pointers, used) of ids and weights [tokens, used]."""
    if not isinstance(ids, torch.Tensor) or not isinstance(weights, torch.Tensor):
        raise TypeError("ids and weights: expected torch.Tensors")
    if ids.dim() != 2 or ids.shape[0] != tokens or ids.shape != weights.shape:
        raise ValueError("ids and weights: expected [%d, used]" % tokens)
    n = ids.numel()
    return _ints(ids, "ids", index, n), _ints(weights, "weights", index, n, torch.float32), ids.shape[1]


def xq_moe_route_workspace_bytes(tokens: int, experts: int) -> int:
    return lib().xq_moe_route_workspace_bytes(tokens, experts)


def xq_moe_route(ids, weights, x, router, bias=None, score: str = "softmax", normalize: bool = True,
                 scale: float = 1.0, workspace=None, stream=None) -> None:
    """The experts of the highest scores for each token of x [tokens, K]: ids
    int32 and weights f32 [tokens, used], from router [experts, K]."""
    index = _index(x)
    xp, x_kind, x_row = _matrix(x, "x", index)
    rp, r_kind, _ = _matrix(router, "router", index)
    tokens, k = x.shape
    experts = router.shape[0]
    if router.shape[1] != k or not router.is_contiguous():
        raise ValueError("router: expected contiguous [experts, %d]" % k)
    if score not in _SCORES:
        raise ValueError("score: expected softmax or sigmoid, got %r" % (score,))
    ip, wp, used = _choice(ids, weights, tokens, index)
    bp = None if bias is None else _ints(bias, "bias", index, experts, torch.float32)
    sp, sb = _workspace(workspace, index)
    _check(lib().xq_moe_route(ip, wp, xp, x_kind, x_row, rp, r_kind, bp, tokens, experts, used, k, _SCORES[score],
                              1 if normalize else 0, scale, sp, sb, _raw_stream(stream, index)),
           "xq_moe_route")


def xq_moe_q4k_workspace_bytes(tokens: int, used: int, hidden: int, ffn: int) -> int:
    return lib().xq_moe_q4k_workspace_bytes(tokens, used, hidden, ffn)


def xq_moe_q4k(y, x, gate, up, down, ids, weights, experts: int, ffn: int, workspace=None, stream=None) -> None:
    """The chosen experts' feed-forward of x [tokens, hidden] and its weighted
    sum into y; gate, up and down are slabs of Q4_K bytes, `experts` experts of
    [ffn, hidden], [ffn, hidden] and [hidden, ffn]."""
    index = _index(x)
    xp, x_kind, x_row = _matrix(x, "x", index)
    yp, y_kind, y_row = _matrix(y, "y", index)
    if y.shape != x.shape or y_kind != x_kind:
        raise ValueError("y and x differ in shape or type")
    tokens, hidden = x.shape
    ip, wp, used = _choice(ids, weights, tokens, index)
    need, slabs = experts * ffn * (hidden // 256) * 144, []
    for t, what in ((gate, "gate"), (up, "up"), (down, "down")):
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s: expected a torch.Tensor" % what)
        if t.get_device() != index or not t.is_contiguous():
            raise ValueError("%s: expected a contiguous tensor on device %d" % (what, index))
        if t.nbytes < need:
            raise ValueError("%s: holds %d bytes, the layout needs %d" % (what, t.nbytes, need))
        slabs.append(t.data_ptr())
    sp, sb = _workspace(workspace, index)
    _check(lib().xq_moe_q4k(yp, y_row, xp, x_row, x_kind, *slabs, ip, wp, tokens, used, experts, hidden, ffn, sp, sb,
                            _raw_stream(stream, index)),
           "xq_moe_q4k")
