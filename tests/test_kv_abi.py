"""The paged cache's part of the C ABI on the host: sizes, and what it refuses
before any HIP call (no GPU is touched by these tests)."""
import ctypes

import pytest
import torch

import quantized_decode_mat_amd as xq
from quantized_decode_mat_amd.kv import _KV, _Rope

# Fake device addresses: nothing is dereferenced or launched.
A = 0x7F0000000000
WS = 0x7F0000100000
BIG = 1 << 40


def kv(**change):
    f = dict(k=A, v=A, layers=1, pages=100, kv_heads=8, page=16, dim=128, dtype=xq.XQ_BF16, k_scale=1.0, v_scale=1.0,
             k_stride=(0, 16384, 2048, 128), v_stride=(0, 16384, 2048, 128))
    f.update(change)
    for name in ("k_stride", "v_stride"):
        f[name] = (ctypes.c_int64 * 4)(*f[name])
    return _KV(**f)


def rope(**change):
    f = dict(freq=A, rot=128, axes=3, adjacent=0, sections=(24, 20, 20, 0))
    f.update(change)
    f["sections"] = (ctypes.c_int64 * 4)(*f["sections"])
    return _Rope(**f)


DEFAULTS = {
    "xq_attn_decode": [("out", A), ("q", A), ("io", xq.XQ_BF16), ("seqs", 2), ("heads", 32), ("out_row", 4096),
                       ("out_head", 128), ("q_row", 4096), ("q_head", 128), ("kv", None), ("tables", A), ("width", 8),
                       ("stride", 8), ("lens", A), ("scale", 0.1), ("window", 0), ("sinks", 0), ("max_len", 128),
                       ("ws", WS), ("ws_bytes", BIG), ("stream", None)],
    "xq_attn_prefill": [("out", A), ("q", A), ("io", xq.XQ_BF16), ("rows", 64), ("seqs", 2), ("heads", 32),
                        ("out_row", 4096), ("out_head", 128), ("q_row", 4096), ("q_head", 128), ("kv", None),
                        ("tables", A), ("width", 8), ("stride", 8), ("lens", A), ("starts", A), ("max_chunk", 40),
                        ("scale", 0.1), ("window", 0), ("sinks", 0), ("stream", None)],
    "xq_rope": [("out", A), ("out_type", xq.XQ_F32), ("out_row", 4096), ("out_head", 128), ("x", A),
                ("x_type", xq.XQ_F32), ("x_row", 4096), ("x_head", 128), ("tokens", 5), ("heads", 32), ("dim", 128),
                ("pos", A), ("pos_stride", 5), ("rope", None), ("inverse", 0), ("stream", None)],
    "xq_rope_append": [("q_out", A), ("out_type", xq.XQ_F32), ("out_row", 4096), ("out_head", 128), ("kv", None),
                       ("q", A), ("q_row", 6144), ("q_head", 128), ("k", A), ("k_row", 6144), ("k_head", 128), ("v", A),
                       ("v_row", 6144), ("v_head", 128), ("x_type", xq.XQ_F32), ("tokens", 5), ("heads", 32), ("pos", A),
                       ("pos_stride", 5), ("rope", None), ("slots", A), ("stream", None)],
    "xq_cache_copy": [("kv", None), ("src", A), ("dst", A), ("n", 3), ("stream", None)],
    "xq_cache_free": [("kv", None), ("refs", A), ("tables", A), ("slots", 4), ("width", 8), ("stride", 8), ("lens", A),
                      ("rows", A), ("n", 3), ("stream", None)],
    "xq_cache_fork": [("kv", None), ("refs", A), ("tables", A), ("slots", 4), ("width", 8), ("stride", 8), ("lens", A),
                      ("parents", A), ("children", A), ("n", 3), ("status", A), ("ws", WS), ("ws_bytes", BIG),
                      ("stream", None)],
    "xq_cache_compact": [("kv", None), ("refs", A), ("tables", A), ("slots", 4), ("width", 8), ("stride", 8),
                         ("status", A), ("ws", WS), ("ws_bytes", BIG), ("stream", None)],
}


def call(name, change):
    change = dict(change)
    cache = kv(**{k[3:]: change.pop(k) for k in list(change) if k.startswith("kv_")})
    turn = rope(**{k[2:]: change.pop(k) for k in list(change) if k.startswith("r_")})
    args = []
    for key, value in DEFAULTS[name]:
        value = change.pop(key) if key in change else value
        if key == "kv" and value is None:
            value = ctypes.byref(cache)
        if key == "rope" and value is None:
            value = ctypes.byref(turn)
        args.append(None if value == "null" else value)
    assert not change, change
    s = getattr(xq.lib(), name)(*args)
    return s, xq.xq_last_error()


NULL, SHAPE, ALIGN = xq.XQ_E_NULL, xq.XQ_E_SHAPE, xq.XQ_E_ALIGN
KV_REFUSED = [
    (dict(kv="null"), NULL, "kv is NULL"),
    (dict(kv_k=0), NULL, "kv k is NULL"),
    (dict(kv_v=0), NULL, "kv v is NULL"),
    (dict(kv_dtype=xq.XQ_F32), SHAPE, "dtype=0"),
    (dict(kv_layers=0), SHAPE, "layers=0"),
    (dict(kv_pages=0), SHAPE, "pages=0"),
    (dict(kv_page=0), SHAPE, "page=0"),
    (dict(kv_pages=1 << 30, kv_page=2), SHAPE, "pages=1073741824"),
    (dict(kv_kv_heads=0), SHAPE, "kv_heads=0"),
    (dict(kv_dim=8), SHAPE, "dim=8"),
    (dict(kv_dim=272), SHAPE, "dim=272"),
    (dict(kv_dim=100), SHAPE, "dim=100"),
    (dict(kv_k_scale=0.0), SHAPE, "scales"),
    (dict(kv_v_scale=float("inf")), SHAPE, "scales"),
    (dict(kv_k_scale=float("nan")), SHAPE, "scales"),
    (dict(kv_k_stride=(0, -16, 16, 16)), SHAPE, "stride 1"),
    (dict(kv_k=A + 8), ALIGN, "kv k not 16"),
    (dict(kv_v=A + 2), ALIGN, "kv v not 16"),
    (dict(kv_v_stride=(0, 16384, 2048, 132)), ALIGN, "stride 3"),
]


@pytest.mark.parametrize("name", [n for n in DEFAULTS if n != "xq_rope"])
@pytest.mark.parametrize("change,status,text", KV_REFUSED)
def test_cache_refusals(name, change, status, text):
    s, err = call(name, change)
    assert s == status and text in err, err


TABLES = [
    (dict(tables="null"), NULL, "tables is NULL"),
    (dict(width=0), SHAPE, "table width=0"),
    (dict(stride=7), SHAPE, "table stride=7"),
    (dict(tables=A + 1), ALIGN, "tables not 4"),
]
ATTENTION = TABLES + [
    (dict(out="null"), NULL, "out is NULL"),
    (dict(q="null"), NULL, "q is NULL"),
    (dict(lens="null"), NULL, "lens is NULL"),
    (dict(io=xq.XQ_E4M3), SHAPE, "io=3"),
    (dict(io=7), SHAPE, "io=7"),
    (dict(heads=30), SHAPE, "heads=30"),
    (dict(heads=0), SHAPE, "heads=0"),
    (dict(heads=8 * 257), SHAPE, "heads/kv_heads=257"),
    (dict(seqs=0), SHAPE, "seqs"),
    (dict(seqs=1 << 20), SHAPE, "seqs"),
    (dict(window=-1), SHAPE, "window=-1"),
    (dict(window=(1 << 30) + 1), SHAPE, "window"),
    (dict(sinks=-1), SHAPE, "sinks=-1"),
    (dict(scale=float("nan")), SHAPE, "scale"),
    (dict(kv_layers=2), SHAPE, "layers=2"),
    (dict(q_row=-16), SHAPE, "q has a negative"),
    (dict(out_head=-16), SHAPE, "out has a negative"),
    (dict(q=A + 8), ALIGN, "q not 16"),
    (dict(out=A + 8), ALIGN, "out not 16"),
    (dict(q_head=132), ALIGN, "q strides"),
    (dict(out_row=4100), ALIGN, "out strides"),
    (dict(lens=A + 2), ALIGN, "lens not 4"),
]


@pytest.mark.parametrize("name", ["xq_attn_decode", "xq_attn_prefill"])
@pytest.mark.parametrize("change,status,text", ATTENTION)
def test_attention_refusals(name, change, status, text):
    s, err = call(name, change)
    assert s == status and text in err, err


@pytest.mark.parametrize("change,status,text", [
    (dict(max_len=0), SHAPE, "max_len=0"),
    (dict(max_len=(1 << 30) + 1), SHAPE, "max_len"),
    (dict(max_len=1 << 20, ws="null", ws_bytes=0), NULL, "workspace is NULL"),
    (dict(max_len=1 << 20, ws_bytes=1000), SHAPE, "workspace_bytes=1000"),
    (dict(max_len=1 << 20, ws=WS + 16), ALIGN, "workspace not 256"),
])
def test_decode_refusals(change, status, text):
    s, err = call("xq_attn_decode", change)
    assert s == status and text in err, err


@pytest.mark.parametrize("change,status,text", [
    (dict(io=xq.XQ_F32), SHAPE, "io=0"),
    (dict(io=xq.XQ_F16), SHAPE, "kv dtype=1"),
    (dict(starts="null"), NULL, "starts is NULL"),
    (dict(starts=A + 2), ALIGN, "starts not 4"),
    (dict(rows=0), SHAPE, "rows"),
    (dict(rows=1 << 27), SHAPE, "rows"),
    (dict(max_chunk=0), SHAPE, "max_chunk=0"),
    (dict(max_chunk=65), SHAPE, "max_chunk=65"),
    (dict(rows=1 << 25, max_chunk=1 << 25, seqs=1 << 10), SHAPE, "too many workgroups"),
])
def test_prefill_refusals(change, status, text):
    s, err = call("xq_attn_prefill", change)
    assert s == status and text in err, err


ROPE = [
    (dict(pos="null"), NULL, "pos is NULL"),
    (dict(rope="null"), NULL, "rope is NULL"),
    (dict(r_freq=0), NULL, "freq is NULL"),
    (dict(out_type=xq.XQ_E4M3), SHAPE, "out_type=3"),
    (dict(x_type=4), SHAPE, "x_type=4"),
    (dict(r_rot=4), SHAPE, "rot=4"),
    (dict(r_rot=136), SHAPE, "rot=136"),
    (dict(r_rot=60), SHAPE, "rot=60"),
    (dict(r_axes=0), SHAPE, "axes=0"),
    (dict(r_axes=5), SHAPE, "axes=5"),
    (dict(r_adjacent=2), SHAPE, "adjacent=2"),
    (dict(r_sections=(65, 0, -1, 0)), SHAPE, "sections[0]=65"),
    (dict(r_sections=(24, 20, 19, 1)), SHAPE, "sum to 63"),
    (dict(tokens=0), SHAPE, "tokens"),
    (dict(tokens=1 << 31), SHAPE, "tokens"),
    (dict(heads=0), SHAPE, "heads"),
    (dict(pos_stride=-1), SHAPE, "pos has a negative"),
    (dict(pos=A + 2), ALIGN, "pos not 4"),
    (dict(r_freq=A + 4), ALIGN, "freq not 8"),
]


@pytest.mark.parametrize("name", ["xq_rope", "xq_rope_append"])
@pytest.mark.parametrize("change,status,text", ROPE)
def test_rope_refusals(name, change, status, text):
    s, err = call(name, change)
    assert s == status and text in err, err


@pytest.mark.parametrize("name,change,status,text", [
    ("xq_rope", dict(out="null"), NULL, "out is NULL"),
    ("xq_rope", dict(x="null"), NULL, "x is NULL"),
    ("xq_rope", dict(dim=132, r_rot=128), SHAPE, "dim=132"),
    ("xq_rope", dict(dim=2048), SHAPE, "dim=2048"),
    ("xq_rope", dict(inverse=2), SHAPE, "inverse=2"),
    ("xq_rope", dict(x_row=-1), SHAPE, "x has a negative"),
    ("xq_rope", dict(x=A + 2), ALIGN, "x not aligned"),
    ("xq_rope", dict(out=A + 1), ALIGN, "out not aligned"),
    ("xq_rope_append", dict(q_out="null"), NULL, "q_out is NULL"),
    ("xq_rope_append", dict(q="null"), NULL, "q is NULL"),
    ("xq_rope_append", dict(k="null"), NULL, "k is NULL"),
    ("xq_rope_append", dict(v="null"), NULL, "v is NULL"),
    ("xq_rope_append", dict(slots="null"), NULL, "slots is NULL"),
    ("xq_rope_append", dict(kv_layers=3), SHAPE, "layers=3"),
    ("xq_rope_append", dict(v_head=-1), SHAPE, "v has a negative"),
    ("xq_rope_append", dict(k=A + 2), ALIGN, "k not aligned"),
    ("xq_rope_append", dict(slots=A + 4), ALIGN, "slots not 8"),
])
def test_rope_own_refusals(name, change, status, text):
    s, err = call(name, change)
    assert s == status and text in err, err


@pytest.mark.parametrize("name", ["xq_cache_free", "xq_cache_fork", "xq_cache_compact"])
@pytest.mark.parametrize("change,status,text", TABLES + [
    (dict(refs="null"), NULL, "refs is NULL"),
    (dict(refs=A + 2), ALIGN, "refs not 4"),
    (dict(slots=0), SHAPE, "slots=0"),
    (dict(slots=(1 << 20) + 1), SHAPE, "slots"),
])
def test_pages_refusals(name, change, status, text):
    s, err = call(name, change)
    assert s == status and text in err, err


@pytest.mark.parametrize("name,change,status,text", [
    ("xq_cache_copy", dict(src="null"), NULL, "src is NULL"),
    ("xq_cache_copy", dict(dst="null"), NULL, "dst is NULL"),
    ("xq_cache_copy", dict(n=-1), SHAPE, "n=-1"),
    ("xq_cache_copy", dict(n=1 << 31), SHAPE, "n="),
    ("xq_cache_copy", dict(src=A + 2), ALIGN, "src not 4"),
    ("xq_cache_free", dict(lens="null"), NULL, "lens is NULL"),
    ("xq_cache_free", dict(rows="null"), NULL, "rows is NULL"),
    ("xq_cache_free", dict(n=(1 << 20) + 1), SHAPE, "n="),
    ("xq_cache_fork", dict(parents="null"), NULL, "parents is NULL"),
    ("xq_cache_fork", dict(children="null"), NULL, "children is NULL"),
    ("xq_cache_fork", dict(status="null"), NULL, "status is NULL"),
    ("xq_cache_fork", dict(n=5), SHAPE, "n=5"),
    ("xq_cache_fork", dict(ws="null"), NULL, "workspace is NULL"),
    ("xq_cache_fork", dict(ws_bytes=100), SHAPE, "workspace_bytes=100"),
    ("xq_cache_fork", dict(ws=WS + 4), ALIGN, "workspace not 256"),
    ("xq_cache_compact", dict(status="null"), NULL, "status is NULL"),
    ("xq_cache_compact", dict(ws="null"), NULL, "workspace is NULL"),
    ("xq_cache_compact", dict(ws_bytes=100), SHAPE, "workspace_bytes=100"),
    ("xq_cache_compact", dict(status=A + 1), ALIGN, "status not 4"),
])
def test_pages_own_refusals(name, change, status, text):
    s, err = call(name, change)
    assert s == status and text in err, err


def test_empty_lists_do_nothing():
    assert call("xq_cache_copy", dict(n=0, src="null", dst="null"))[0] == xq.XQ_OK
    assert call("xq_cache_free", dict(n=0, rows="null"))[0] == xq.XQ_OK


def test_workspace_sizes():
    """96 KiB of counters at the same place for every plan; nothing where nothing is split or nothing is sound."""
    need = lambda seqs, heads, max_len, window=0, sinks=0, **c: xq.lib().xq_attn_decode_workspace_bytes(
        seqs, heads, ctypes.byref(kv(**c)), max_len, window, sinks)
    assert need(1, 32, 100) == 0                      # one step of one workgroup
    assert need(2, 32, 131072) > 96 * 1024
    assert need(200, 32, 4096) == 0                   # more (sequence, kv head) pairs than a round of workgroups
    assert need(2, 32, 131072, 128) < need(2, 32, 131072, 1024) < need(2, 32, 131072)
    assert need(0, 32, 100) == 0 and need(1, 31, 100) == 0 and need(1, 32, 0) == 0 and need(1, 32, 4096, dim=8) == 0
    ws = xq.xq_cache_workspace_bytes
    assert ws(1000, 10) > 96 * 1024 + 4 * 3 * 1000 and ws(0, 1) == 0 and ws(1, 0) == 0


def test_binding_refuses_host_and_wrong_tensors():
    x = torch.zeros(2, 4, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        xq.xq_kv_cache(torch.zeros(4, 1, 16, 16, dtype=torch.bfloat16), torch.zeros(4, 1, 16, 16, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="torch.Tensor"):
        xq.xq_kv_cache([1], [2])
    with pytest.raises(ValueError, match="device tensor"):
        xq.xq_rope_plan(torch.ones(8, dtype=torch.float64), [8])
    with pytest.raises(ValueError, match="device tensor"):
        xq.xq_rope(x, x, None, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="a GPU is there")
@pytest.mark.parametrize("name", list(DEFAULTS))
def test_device_gate_without_gpu(name):
    s, err = call(name, {})
    assert s == xq.XQ_E_DEVICE, err
