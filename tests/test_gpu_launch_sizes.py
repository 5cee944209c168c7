"""More threads than a launch counts are refused, not left out."""
import pytest
import torch

import quantized_decode_mat_amd as xq

pytestmark = pytest.mark.gpu


def test_rows_of_more_threads_than_a_launch_counts():
    """A wave a row: 2^26 rows are 2^32 threads."""
    n, k = (1 << 26) + 64, 256
    w = torch.empty(n * 144, dtype=torch.uint8, device="cuda")
    x = torch.zeros(xq.xq_q8k_bytes(1, k), dtype=torch.uint8, device="cuda")
    y = torch.full((n,), 7.0, device="cuda")
    with pytest.raises(xq.XQError, match="xq_gemv_q4k") as refused:
        xq.xq_gemv_q4k(y, w, x, n, k)
    assert refused.value.status == xq.XQ_E_LAUNCH
    torch.cuda.synchronize()
    assert (y == 7.0).all()
