"""Sizes and scales that the paged cache's kernels cannot take are refused on
the host, before any HIP call."""
import pytest

import quantized_decode_mat_amd as xq
from test_kv_abi import SHAPE, call


@pytest.mark.parametrize("name", ["xq_attn_decode", "xq_attn_prefill"])
@pytest.mark.parametrize("scale,k_scale", [(1e30, 1e10), (-1e30, 1e10), (3e38, 1.0), (1.0, 3e38)])
def test_scales_whose_product_overflows(name, scale, k_scale):
    s, err = call(name, dict(scale=scale, kv_k_scale=k_scale))
    assert s == SHAPE and "above f32's range" in err, err


@pytest.mark.parametrize("name,change", [
    # 2^20 units of 256 heads, 16 at a time
    ("xq_attn_decode", dict(seqs=1 << 20, heads=256, kv_kv_heads=1)),
    # 2^16 sequences of 2^8 tiles of 128 rows
    ("xq_attn_prefill", dict(seqs=1 << 16, heads=1, kv_kv_heads=1, rows=1 << 15, max_chunk=1 << 15)),
])
def test_more_workgroups_than_a_launch_counts(name, change):
    s, err = call(name, change)
    assert s == SHAPE and "too many workgroups" in err, err


def test_counters_stay_in_the_first_96_kib():
    """Where every call that shares a workspace keeps what has to stay zero."""
    sizes = [xq.xq_gemv_q4k_q8k_workspace_bytes(256 * n) for n in range(1, 16385)]
    assert sizes == [128 * min(n, 768) for n in range(1, 16385)]


@pytest.mark.parametrize("name", ["xq_cache_copy", "xq_cache_free", "xq_cache_fork", "xq_cache_compact"])
def test_more_layers_than_a_page_move_counts(name):
    s, err = call(name, dict(kv_layers=(1 << 24) + 1))
    assert s == SHAPE and "layers=16777217" in err, err
