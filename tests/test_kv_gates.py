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
