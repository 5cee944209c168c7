"""Experts by rows where down takes a token's blocks four steps of 16 at a time: as many as that or fewer, in one turn and
with the next row's weights under way, and more, several turns a row; with one row a wave and with several. Tolerances
are test_gpu_moe's."""
import pytest
import torch

from test_gpu_kv_four import _device  # noqa: F401
from test_gpu_moe import check, run, state

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("case", [
    # tokens, used, experts, hidden, ffn, io
    (1, 8, 16, 4096, 2048, "bf16"),   # 64 blocks, two rows a wave
    (1, 8, 8, 2048, 2048, "f32"),     # the same, one row
    (5, 7, 64, 2048, 2048, "f16"),    # 56 blocks, six rows
    (1, 7, 7, 6400, 1792, "f32"),     # 49 blocks, four rows, the last of them past the end for some
    (3, 3, 16, 2048, 7168, "f32"),    # 84 blocks: two turns, four rows
    (1, 5, 5, 4352, 11264, "bf16"),   # 220 blocks: four turns, three rows
], ids=lambda c: "-".join(str(x) for x in c))
def test_down_by_rows(case):
    c = dict(zip(("tokens", "used", "experts", "hidden", "ffn", "io"), case))
    s = state(c, 3)
    run(c, s)
    check(c, s, "layer")
    first = s["y"].clone()
    s["full"][:, :c["hidden"]] = 5.0
    run(c, s)
    torch.cuda.synchronize()
    assert torch.equal(s["y"], first), "the same call gave other bits"
    s["ids"][0, 1], s["ids"][-1, -1] = -1, c["experts"]       # slots that are left out
    run(c, s)
    check(c, s, "layer with slots left out")
