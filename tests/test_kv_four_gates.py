"""The 4-bit cache on the host: what is refused before any HIP call, and which bytes of a row each lane loads."""
import ctypes
import os
import subprocess

import pytest
import torch

import quantized_decode_mat_amd as xq
from quantized_decode_mat_amd.kv import _KV
from test_kv_abi import A, ALIGN, BIG, DEFAULTS, NULL, SHAPE, call, rope

DEFAULTS.setdefault("xq_cache_read", [("k_out", A), ("k_row", 1024), ("k_head", 128), ("v_out", A), ("v_row", 1024),
                                      ("v_head", 128), ("out_type", xq.XQ_BF16), ("kv", None), ("slots", A),
                                      ("tokens", 5), ("stream", None)])
CALLS = ["xq_attn_decode", "xq_attn_prefill", "xq_rope_append", "xq_cache_read", "xq_cache_copy", "xq_cache_fork",
         "xq_cache_compact"]


def four(change):
    f = dict(k=A, v=A, layers=1, pages=100, kv_heads=8, page=16, dim=128, dtype=xq.XQ_E2M1, k_scale=1.0, v_scale=1.0,
             k_stride=(0, 16384, 2048, 128), v_stride=(0, 16384, 2048, 128), k_exp=A, v_exp=A,
             k_exp_stride=(0, 512, 64, 4), v_exp_stride=(0, 512, 64, 4))
    f.update(change)
    for name in ("k_stride", "v_stride", "k_exp_stride", "v_exp_stride"):
        f[name] = (ctypes.c_int64 * 4)(*f[name])
    return _KV(**f)


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("change,status,text", [
    (dict(k_exp=0), NULL, "k_exp is NULL"),
    (dict(v_exp=0), NULL, "v_exp is NULL"),
    (dict(dim=112), SHAPE, "dim=112 of XQ_E2M1"),
    (dict(dim=288), SHAPE, "dim=288"),
    (dict(dtype=5), SHAPE, "dtype=5"),
    (dict(k_exp_stride=(0, 512, -64, 4)), SHAPE, "exponents' stride 2 is negative"),
    (dict(k_exp=A + 2), ALIGN, "k_exp not 4-byte"),
    (dict(v_exp=A + 1), ALIGN, "v_exp not 4-byte"),
    (dict(v_exp_stride=(0, 512, 64, 3)), ALIGN, "exponents' stride 3"),
    (dict(k_stride=(0, 16384, 2048, 144)), ALIGN, "stride 3 not a multiple of 16 bytes"),
    (dict(k=A + 8), ALIGN, "k not 16-byte"),
])
def test_refusals(name, change, status, text):
    s, err = call(name, dict(kv=ctypes.byref(four(change))))
    assert s == status and text in err, err


@pytest.mark.parametrize("change,status,text", [
    (dict(k_out="null"), NULL, "k_out is NULL"),
    (dict(v_out="null"), NULL, "v_out is NULL"),
    (dict(slots="null"), NULL, "slots is NULL"),
    (dict(out_type=3), SHAPE, "out_type=3"),
    (dict(tokens=0), SHAPE, "tokens"),
    (dict(tokens=1 << 28), SHAPE, "tokens"),
    (dict(k_row=-1), SHAPE, "k_out has a negative stride"),
    (dict(v_head=-1), SHAPE, "v_out has a negative stride"),
    (dict(k_out=A + 1), ALIGN, "k_out"),
    (dict(v_out=A + 1), ALIGN, "v_out"),
    (dict(slots=A + 4), ALIGN, "slots not 8-byte"),
    (dict(kv_layers=2, ), SHAPE, "layers=2"),
])
def test_read_refusals(change, status, text):
    s, err = call("xq_cache_read", change)
    assert s == status and text in err, err


def test_chunks_of_f32_are_refused():
    s, err = call("xq_attn_prefill", dict(kv=ctypes.byref(four({})), io=xq.XQ_F32))
    assert s == SHAPE and "io=0" in err


def test_pages_over_64_gib_are_counted_in_bytes():
    far = (0, 1 << 31, 2048, 128)
    s, err = call("xq_attn_decode", dict(kv=ctypes.byref(four(dict(k_stride=far)))))
    assert s == SHAPE and "64 GiB" in err
    near = (0, (1 << 37) // 99 // 32 * 32 - 4096, 2048, 128)
    s, err = call("xq_attn_decode", dict(kv=ctypes.byref(four(dict(k_stride=near)))))
    assert "64 GiB" not in err, err


def test_workspace_is_the_other_types_own():
    """The plan's size depends on the type's residency alone."""
    for dim in (32, 64, 96, 128, 192, 256):
        kv = four(dict(dim=dim))
        n = xq.lib().xq_attn_decode_workspace_bytes(2, 32, ctypes.byref(kv), 131072, 0, 0)
        assert n > 96 * 1024


SOURCE = r"""
#include <cstdio>
#include <cstring>
#include "kv_lanes.h"
static int bad = 0;
template <int DP, bool FULL> static void check(int dim) {
  char seen[256] = {};
  for (int s = 0; s < xq::decode4_k_loads(DP); ++s)
    for (int g = 0; g < 4; ++g) {
      const int d = xq::decode4_k_dim<DP, FULL>(s, g, dim), n = 2 * xq::decode4_k_bytes(DP);
      if (d < 0 || d + n > dim || d % n) std::printf("dim %d: reads %d..%d\n", dim, d, d + n - 1), ++bad;
      else std::memset(seen + d, 1, n);
    }
  for (int d = 0; d < dim; ++d) if (!seen[d]) std::printf("dim %d of %d is not read\n", d, dim), ++bad;
}
int main() {
  check<64, true>(64); check<64, false>(32); check<64, false>(64);
  check<128, true>(128); check<128, false>(96); check<128, false>(128);
  check<192, true>(192); check<192, false>(160); check<192, false>(192);
  check<256, true>(256); check<256, false>(224); check<256, false>(256);
  return bad != 0;
}
"""


def test_lanes_load_a_row_of_4_bits(tmp_path):
    src = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_decode_mat_amd", "csrc")
    (tmp_path / "lanes.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-I", src, str(tmp_path / "lanes.cpp"), "-o", str(tmp_path / "lanes")], check=True)
    r = subprocess.run([str(tmp_path / "lanes")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_binding_refuses_wrong_tensors():
    x = torch.zeros(4, 2, 16, 64, dtype=torch.uint8).view(torch.float4_e2m1fn_x2)
    with pytest.raises(ValueError, match="device tensor"):
        xq.xq_kv_cache(x, x)
