"""Edges of the paged cache's calls: what lies beside a row, scales of zero,
small weights, starts that do not fit, sizes past a launch's."""
import pytest
import torch

import kv_reference as ref
import quantized_decode_mat_amd as xq
from test_gpu_kv_attention import _device, check_decode, check_prefill, decode, prefill, setup  # noqa: F401
from test_gpu_kv_prefill_large import copies

pytestmark = pytest.mark.gpu
DEV = "cuda"


def beside(s, fill):
    """The same cache as slices of rows of 256, with `fill` in what is beside them."""
    kv = []
    for x in (s["k"], s["v"]):
        wide = torch.full((*x.shape[:3], 256), fill, device=DEV).to(x.dtype)
        wide[..., :x.shape[3]] = x
        kv.append(wide[..., :x.shape[3]])
    return dict(s, k=kv[0], v=kv[1], kv=xq.xq_kv_cache(*kv, *s["scales"]))


@pytest.mark.parametrize("cache,io", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "f16")])
@pytest.mark.parametrize("dim", [176, 192])
def test_what_lies_beside_a_row_has_no_influence(cache, io, dim):
    lens = [517, 90, 3]
    s = setup(lens, 6, 2, dim, 16, cache, io, "hnd", poison=False)
    results = []
    for fill in (0.0, float("nan")):
        t = beside(s, fill)
        decode(t, 0, 0, 517)
        check_decode(t, lens, 0, 0, "decode")
        results.append(t["out"].clone())
        prefill(t, [1, 1, 1], 0, 0)
        check_prefill(t, lens, [1, 1, 1], [0, 1, 2, 3], 0, 0, "single rows")
        results.append(t["out"].clone())
    assert torch.equal(results[0], results[2]) and torch.equal(results[1], results[3])


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("cache,io,scale,k_scale", [("bf16", "bf16", 0.0, 1.0), ("f16", "f16", 0.0, 1.0),
                                                   ("e4m3", "bf16", 0.0, 0.75), ("e4m3", "f16", 1e-30, 1e-20)])
def test_scale_of_zero(cache, io, scale, k_scale, many):
    """Every visible token weighs the same."""
    n = copies([64, 129], 4, 2) if many else 1
    lens, chunks = [300, 129] * n, [64, 129] * n
    s = setup(lens, 4, 2, 80, 16, cache, io, "hnd", rows=193 * n)
    s["scale"], s["scales"] = scale, (k_scale, s["scales"][1])
    s["kv"] = xq.xq_kv_cache(s["k"], s["v"], *s["scales"])
    starts = prefill(s, chunks, 50, 2)
    check_prefill(s, lens, chunks, starts, 50, 2, "scale of zero")
