"""The mixture-of-experts layer's part of the C ABI on the host: sizes, and what it refuses before any HIP call."""
import pytest
import torch

import quantized_decode_mat_amd as xq

A, WS, BIG = 0x7F0000000000, 0x7F0000100000, 1 << 40
NULL, SHAPE, ALIGN = xq.XQ_E_NULL, xq.XQ_E_SHAPE, xq.XQ_E_ALIGN

ROUTE = [("ids", A), ("weights", A), ("x", A), ("x_type", xq.XQ_BF16), ("x_row", 2048), ("router", A),
         ("router_type", xq.XQ_BF16), ("bias", None), ("tokens", 3), ("experts", 64), ("used", 8), ("K", 2048),
         ("score", 0), ("normalize", 1), ("scale", 1.0), ("ws", WS), ("ws_bytes", BIG), ("stream", None)]
LAYER = [("y", A), ("y_row", 2048), ("x", A), ("x_row", 2048), ("io", xq.XQ_BF16), ("gate", A), ("up", A), ("down", A),
         ("ids", A), ("weights", A), ("tokens", 3), ("used", 8), ("experts", 64), ("hidden", 2048), ("ffn", 1536),
         ("ws", WS), ("ws_bytes", BIG), ("stream", None)]


def call(name, defaults, change):
    args = [change[k] if k in change else v for k, v in defaults]
    assert set(change) <= {k for k, _ in defaults}
    s = getattr(xq.lib(), name)(*[None if a == "null" else a for a in args])
    return s, xq.xq_last_error()


@pytest.mark.parametrize("change,status,text", [
    *[(dict([(k, "null")]), NULL, "%s is NULL" % k) for k in ("ids", "weights", "x", "router")],
    (dict(ws=None), NULL, "workspace is NULL"),
    (dict(x_type=3), SHAPE, "x_type=3"),
    (dict(router_type=-1), SHAPE, "router_type=-1"),
    (dict(tokens=0), SHAPE, "tokens=0"),
    (dict(tokens=513), SHAPE, "tokens=513"),
    (dict(experts=0), SHAPE, "experts=0"),
    (dict(experts=1025), SHAPE, "experts=1025"),
    (dict(used=0), SHAPE, "used=0"),
    (dict(used=65, experts=128), SHAPE, "used=65"),
    (dict(used=5, experts=4), SHAPE, "used=5"),
    (dict(K=4), SHAPE, "K=4"),
    (dict(K=2044), SHAPE, "K=2044"),
    (dict(K=1 << 21, x_row=1 << 21), SHAPE, "K=2097152"),
    (dict(score=2), SHAPE, "score=2"),
    (dict(normalize=2), SHAPE, "normalize=2"),
    (dict(scale=float("inf")), SHAPE, "scale=inf"),
    (dict(x_row=2040), SHAPE, "x row stride=2040"),
    (dict(x_row=-1, tokens=1), SHAPE, "x row stride=-1"),
    (dict(ws_bytes=96 * 1024 + 4 * 3 * 64 - 1), SHAPE, "workspace_bytes"),
    (dict(ids=A + 2), ALIGN, "ids"),
    (dict(weights=A + 2), ALIGN, "weights"),
    (dict(x=A + 8), ALIGN, "x or its rows"),
    (dict(x_row=2052), ALIGN, "x or its rows"),
    (dict(router=A + 8), ALIGN, "router"),
    (dict(bias=A + 2), ALIGN, "bias"),
    (dict(ws=WS + 128), ALIGN, "workspace"),
])
def test_route_refusals(change, status, text):
    s, err = call("xq_moe_route", ROUTE, change)
    assert s == status and text in err, err


@pytest.mark.parametrize("change,status,text", [
    *[(dict([(k, "null")]), NULL, "%s is NULL" % k) for k in ("y", "x", "gate", "up", "down", "ids", "weights")],
    (dict(ws=None), NULL, "workspace is NULL"),
    (dict(io=3), SHAPE, "io=3"),
    (dict(tokens=0), SHAPE, "tokens*used"),
    (dict(used=0), SHAPE, "tokens*used"),
    (dict(tokens=65, used=8), SHAPE, "tokens*used = 65*8"),
    (dict(tokens=1 << 40, used=1 << 40), SHAPE, "tokens*used"),
    (dict(experts=0), SHAPE, "experts=0"),
    (dict(experts=1025), SHAPE, "experts=1025"),
    (dict(hidden=2000), SHAPE, "hidden=2000"),
    (dict(hidden=33024), SHAPE, "hidden=33024"),
    (dict(ffn=0), SHAPE, "ffn=0"),
    (dict(ffn=1408), SHAPE, "ffn=1408"),
    (dict(y_row=2047), SHAPE, "y row stride=2047"),
    (dict(x_row=0), SHAPE, "x row stride=0"),
    (dict(ws_bytes=1 << 16), SHAPE, "workspace_bytes"),
    (dict(y=A + 1), ALIGN, "y not aligned"),
    (dict(x=A + 2), ALIGN, "x or its rows"),
    (dict(x_row=2049), ALIGN, "x or its rows"),
    *[(dict([(k, A + 8)]), ALIGN, "%s not 16" % k) for k in ("gate", "up", "down")],
    (dict(ids=A + 1), ALIGN, "ids"),
    (dict(weights=A + 1), ALIGN, "weights"),
    (dict(ws=WS + 64), ALIGN, "workspace"),
])
def test_layer_refusals(change, status, text):
    s, err = call("xq_moe_q4k", LAYER, change)
    assert s == status and text in err, err


def test_workspaces():
    assert xq.xq_moe_route_workspace_bytes(3, 64) == 96 * 1024 + 4 * 3 * 64
    assert xq.xq_moe_route_workspace_bytes(0, 64) == xq.xq_moe_route_workspace_bytes(513, 64) == 0
    assert xq.xq_moe_route_workspace_bytes(1, 1025) == 0
    for bad in ((0, 1, 256, 256), (513, 1, 256, 256), (1, 513, 256, 256), (1, 1, 128, 256), (1, 1, 256, 33024)):
        assert xq.xq_moe_q4k_workspace_bytes(*bad) == 0
    # behind other calls' counters: room for every pair's h at least
    for tokens, used, hidden, ffn in ((1, 1, 256, 256), (64, 8, 4096, 14336), (1, 512, 32768, 32768)):
        n = xq.xq_moe_q4k_workspace_bytes(tokens, used, hidden, ffn)
        assert n >= 96 * 1024 + 4 * tokens * used * ffn and n % 256 == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 256)
    ids, w = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2)
    with pytest.raises(ValueError, match="x: must be a device tensor"):
        xq.xq_moe_route(ids, w, x, torch.zeros(4, 256))
    with pytest.raises(ValueError, match="x: must be a device tensor"):
        xq.xq_moe_q4k(x, x, x, x, x, ids, w, 4, 256)
