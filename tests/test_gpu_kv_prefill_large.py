"""Chunked attention where the rows are many: the tiles of 128 rows, which the
smaller cases (up to 512 tiles of 16 rows) do not reach. The same cases, each
repeated until there are more."""
import pytest
import torch

import test_gpu_kv_attention as small
from test_gpu_kv_attention import DEV, _device, check_prefill, prefill, setup  # noqa: F401

pytestmark = pytest.mark.gpu


def copies(chunks, heads, kv_heads):
    tiles = len(chunks) * kv_heads * -(-max(chunks) * (heads // kv_heads) // 16)
    return 512 // tiles + 1


@pytest.mark.parametrize("case", small.PREFILL, ids=lambda c: "-".join(str(x) for x in c[2:]))
def test_prefill(case):
    lens, chunks, heads, kv_heads, dim, page, cache, io, order, window, sinks = case
    n = copies(chunks, heads, kv_heads)
    lens, chunks = lens * n, chunks * n
    s = setup(lens, heads, kv_heads, dim, page, cache, io, order, rows=sum(chunks) + 7)
    starts = prefill(s, chunks, window, sinks, first=4)
    check_prefill(s, lens, chunks, starts, window, sinks, "prefill")
    first = s["out"].clone()
    prefill(s, chunks, window, sinks, first=4)
    assert torch.equal(s["out"], first), "the same call gave other bits"


def test_bad_pages():
    n = copies([100, 200, 20], 4, 2)
    lens, chunks = [300, 200, 20] * n, [100, 200, 20] * n
    s = setup(lens, 4, 2, 64, 16, "bf16", "bf16", "hnd", rows=320 * n)
    s["table"][0, 3], s["table"][0, 17], s["table"][2, :] = -1, s["k"].shape[0], -1
    starts = prefill(s, chunks, 0, 0)
    check_prefill(s, lens, chunks, starts, 0, 0, "bad pages")
    assert (s["out"][300:320] == 0).all()


def test_negative_scale():
    n = copies([64, 129], 4, 2)
    for k in (1, n):
        lens, chunks = [100, 129] * k, [64, 129] * k
        s = setup(lens, 4, 2, 64, 16, "f16", "f16", "hnd", rows=193 * k)
        s["scale"] = -0.2
        starts = prefill(s, chunks, 50, 2)
        check_prefill(s, lens, chunks, starts, 50, 2, "negative scale")


@pytest.mark.parametrize("cache,io", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("dim", [64, 80, 128, 256])
@pytest.mark.parametrize("many", [False, True])
def test_unseen_tokens_have_no_influence(cache, io, dim, many):
    """Later tokens of the chunk, and tokens before the window, hold NaN and infinities in k and v."""
    n = copies([400, 60], 4, 2) if many else 1
    lens, chunks, window, sinks = [400, 90] * n, [400, 60] * n, 70, 3
    make = lambda: setup(lens, 4, 2, dim, 16, cache, io, "hnd", rows=460 * n, poison=False)
    s, clean = make(), make()
    prefill(clean, chunks, window, sinks)
    bad = 250  # sequence 0's token; rows 250..319 see it
    p = int(s["table"][0, bad // 16])
    for x in (s["k"], s["v"]):
        x[p, :, bad % 16] = torch.full_like(x[p, :, bad % 16].float(), float("nan")).to(x.dtype)
    if cache != "e4m3":
        s["v"][int(s["table"][0, 399 // 16]), :, 399 % 16, ::2] = float("inf")
    prefill(s, chunks, window, sinks)
    torch.cuda.synchronize()
    got = s["out"]
    assert torch.equal(got[:250], clean["out"][:250]) and torch.equal(got[320:399], clean["out"][320:399])
    assert got[250:320].isnan().all() and torch.equal(got[400:], clean["out"][400:])
    if cache != "e4m3":
        assert (got[399, :, ::2] == float("inf")).all()
        assert torch.equal(got[399, :, 1::2], clean["out"][399, :, 1::2])
