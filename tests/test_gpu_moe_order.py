"""The router's order where scores in f32 are alike."""
import pytest
import torch

import quantized_decode_mat_amd as xq
from test_gpu_kv_four import _device  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda"


def order(logits, score, bias):
    """The router's ids for one row of these logits, as many as it takes (64)."""
    n, used = len(logits), min(len(logits), 64)
    x = torch.zeros(1, 8, device=DEV)
    x[0, 0] = 1
    router = torch.zeros(n, 8, device=DEV)
    router[:, 0] = torch.tensor(logits, device=DEV)
    ids = torch.full((1, used), -1, dtype=torch.int32, device=DEV)
    weights = torch.zeros(1, used, device=DEV)
    ws = torch.zeros(xq.xq_moe_route_workspace_bytes(1, n), dtype=torch.uint8, device=DEV)
    xq.xq_moe_route(ids, weights, x, router, bias=bias, score=score, normalize=False, workspace=ws)
    torch.cuda.synchronize()
    return ids[0].tolist()


@pytest.mark.parametrize("more", [0, 90, 900])
def test_order_of_scores_that_round_to_one(more):
    """Softmax without a bias goes by the logits; with one, of zeros too, by its scores, of which those e^-104 below the
    highest are 0 and go by their index. Sigmoid's scores are 1 from logits of 17.4 on (exp(-17.4) < 2^-25)."""
    logits = [-300.0, 1.0, -150.0, -200.0, 0.0, -120.0, -2.0] + [-400.0] * more
    n = len(logits)
    rest = list(range(7, min(n, 64)))
    zeros = torch.zeros(n, device=DEV)
    assert order(logits, "softmax", None) == [1, 4, 6, 5, 2, 3, 0] + rest
    assert order(logits, "softmax", zeros) == [1, 4, 6, 0, 2, 3, 5] + rest
    logits = [17.5, 1.0, 30.0, 20.0, 0.0, 100.0, -2.0] + [-400.0] * more
    for bias in (None, zeros):
        assert order(logits, "sigmoid", bias) == [0, 2, 3, 5, 1, 4, 6] + rest
