"""The binding on a PyTorch that lacks the types of a 4-bit cache: it loads, and the other caches are described as ever."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
import torch
for name in ("float4_e2m1fn_x2", "float8_e8m0fnu"):
    if hasattr(torch, name):
        delattr(torch, name)
import quantized_decode_mat_amd as xq
from quantized_decode_mat_amd import kv
kv._device = lambda t, what: None      # (what a device tensor is described by, of one on the host)
for dtype, code in ((torch.bfloat16, xq.XQ_BF16), (torch.float16, xq.XQ_F16), (torch.float8_e4m3fn, xq.XQ_E4M3)):
    pool = torch.zeros(2, 3, 4, 16, 64).to(dtype)
    cache = xq.xq_kv_cache(pool, pool)
    assert cache._c.dtype == code and cache.dim == 64 and cache.layer(1).pages == 3
    assert list(cache._c.k_stride) == [3 * 4 * 16 * 64, 4 * 16 * 64, 16 * 64, 64]
for dtype in (torch.uint8, torch.float32):
    try:
        xq.xq_kv_cache(torch.zeros(3, 4, 16, 64, dtype=dtype), torch.zeros(3, 4, 16, 64, dtype=dtype))
    except ValueError as e:
        assert "not supported" in str(e)
    else:
        raise AssertionError("a cache of %s was taken" % dtype)
"""


def test_without_the_4_bit_types():
    r = subprocess.run([sys.executable, "-c", SOURCE], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
