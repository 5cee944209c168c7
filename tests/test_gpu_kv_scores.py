"""Attention at scores of any size: the largest weighs 1 whatever f32's step is there, equal ones share, and what lies
between two scores is not lost in their last bits.

q and k are small whole numbers (halves of them) times powers of two, so that a product's f32 sum is exact. Two scores are
then either equal or as far apart as the definition in 64 bits has them, up to the scale's roundings (three) and one of the
difference's product: 5 half steps of a distance, of which distances above 110 do not count (a weight below 2^-158).

A weight below 2^-126 is no normal number of f32, and the exponential gives 0 for it. Each such token's term is below
2^-126 |v| (the weights' sum is 1 at least), so n tokens add at most n 2^-126 max |v| that is not there."""
import pytest
import torch

import four_reference as four
import kv_reference as ref
import test_gpu_kv_attention as others
import test_gpu_kv_four as bits4
from test_gpu_kv_attention import _device, decode  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda"
CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def setup(cache, lens, heads, kv_heads, dim, page, io, order, rows=None):
    if cache == "e2m1":
        return bits4.setup(lens, heads, kv_heads, dim, page, io, order, rows=rows)
    return others.setup(lens, heads, kv_heads, dim, page, cache, io, order, rows=rows)


def keys(s, b, k):
    """Sequence b's keys become k [n, kv_heads, dim]."""
    j = torch.arange(len(k), device=DEV)
    at, slot = s["table"][b].long()[j // s["page"]], j % s["page"]
    if "k_exp" in s:
        codes, powers, _ = four.encode(k)
        s["k"][at, :, slot] = codes
        s["k_exp"][at, :, slot, :k.shape[-1] // 32] = powers
        assert torch.equal(four.values(codes, powers), k)
    else:
        x = k.float().to(s["k"].dtype)
        assert torch.equal(x.double(), k)
        raw = lambda t: t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
        raw(s["k"])[at, :, slot] = raw(x)


def check(s, b, rows, pos, n, weight_error, what, window=0, sinks=0):
    torch.cuda.synchronize()
    table = s["table"][b]
    if "k_exp" in s:
        (k, there), (v, _) = (four.rows_of(s[x], s[x + "_exp"], table, n, s["page"]) for x in "kv")
    else:
        (k, there), (v, _) = (ref.rows_of(s[x], table, n, s["page"]) for x in "kv")
    want, mag, _ = ref.attend(s["q"][rows], k * s["scales"][0], v * s["scales"][1], there, pos, s["scale"], window, sinks)
    tol = ref.attend_tolerance(want, mag, torch.full_like(want[..., :1], 5 * 110), s["io"], weight_error, n)
    tol = tol + n * 2.0 ** -126 * float((v * s["scales"][1]).abs().max())
    err = (s["out"][rows].double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), "%s: %d of %d outside, worst %.3g of the tolerance" % (
        what, int(bad.sum()), bad.numel(), float((err / tol).nan_to_num(9e9).max()))


def single_error(cache, io):
    return (2.0 ** -24 if io == "f32" else 2.0 ** -16) if cache == "e2m1" else others.weight_error(cache, io)


def far_apart(s, lens, size, by, kv_heads, dim, io, seed=5):
    """Keys and queries whose scores are up to `size`, whole numbers of a step that is over 100 where they differ."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    size_of = lambda *shape: torch.tensor(CODES, dtype=torch.float64, device=DEV)[torch.randint(0, 8, shape, device=DEV, generator=g)]
    sign = torch.randint(0, 2, (kv_heads, dim), device=DEV, generator=g).double() * 2 - 1
    rows, heads = s["q"].shape[:2]
    lift_q, lift_k = 0, 0
    if by == "rows":   # by the values themselves: q up to 2^13 in f16, to 2^60 beyond, k to the largest power
        lift_q, lift_k = 13 if io == "f16" else 60, 11
    top = 0.0
    for b, n in enumerate(lens):
        if n == 0:
            continue
        k = size_of(n, kv_heads, dim) * (torch.randint(0, 2, (n, kv_heads, dim), device=DEV, generator=g) * 2 - 1)
        if b % 3 == 1:
            k[:] = -6 * sign           # all alike, and far below 0
        else:
            for j in {0, n // 3, n // 2, n - 1} if b % 2 else {n // 2}:
                k[j] = 6 * sign
        keys(s, b, k * 2.0 ** lift_k)
        top = max(top, float(k.abs().sum(-1).max()))
    q = torch.randint(1, 4, (rows, heads, dim), device=DEV, generator=g) * sign.repeat_interleave(heads // kv_heads, 0)
    s["q"].copy_(q * 2.0 ** lift_q)
    assert torch.equal(s["q"].double(), q * 2.0 ** lift_q)
    s["scale"] = size / (2 * top) if by == "scale" else 2.0 ** -3


@pytest.mark.parametrize("size,by", [(1e4 * 4608, "scale"), (1e9, "scale"), (2.0 ** 33, "scale"), (1e20, "scale"),
                                     (1e30, "scale"), (-2.0 ** 33, "scale"), (0, "rows")])
@pytest.mark.parametrize("cache,io,dim", [("e2m1", "f32", 128), ("e2m1", "bf16", 64), ("e2m1", "f16", 192), ("e2m1", "f32", 256),
                                          ("bf16", "f32", 128), ("e4m3", "f16", 128)])
def test_single_tokens_of_far_scores(cache, io, dim, size, by):
    if by == "rows" and cache == "e4m3":
        pytest.skip("its largest value is 448")
    lens = [1, 700, 2600, 300, 1, 0, 3]
    s = setup(cache, lens, 8, 2, dim, 16, io, "hnd")
    far_apart(s, lens, size, by, 2, dim, io)
    for most in (2600, 700 * 2600):    # other splits
        decode(s, 0, 0, most)
        for b, n in enumerate(lens):
            if n:
                check(s, b, slice(b, b + 1), torch.tensor([n - 1], device=DEV), n, single_error(cache, io),
                      "sequence %d of %d, planned for %d" % (b, n, most))


def close_by(s, lens, kv_heads, dim, io, seed=6):
    """Scores of 2^21 and beside them halves up to 48, times the scale: in other heads and rows their negatives, and 2^-7 of
    them."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rows, heads = s["q"].shape[:2]
    for b, n in enumerate(lens):
        k = torch.zeros(n, kv_heads, dim, dtype=torch.float64, device=DEV)
        k[..., 0] = 64
        k[..., 32:40] = torch.tensor(CODES, dtype=torch.float64, device=DEV)[torch.randint(0, 8, (n, kv_heads, 8), device=DEV, generator=g)]
        if n:
            keys(s, b, k)
    q = torch.zeros(rows, heads, dim, dtype=torch.float64, device=DEV)
    large = torch.tensor([2.0 ** 15, -2.0 ** 15, 2.0 ** 8], dtype=torch.float64, device=DEV)
    q[..., 0] = large[torch.randint(0, 3, (rows, heads), device=DEV, generator=g)]
    q[..., 32:40] = 1
    s["q"].copy_(q)


@pytest.mark.parametrize("scale", [0.25, 0.34, 0.5, 1.0, 16.0, -1.0])
@pytest.mark.parametrize("io,dim", [("f32", 128), ("bf16", 64), ("f16", 192)])
def test_single_tokens_of_close_scores(io, dim, scale):
    lens = [1, 700, 2600, 300, 0]
    s = setup("e2m1", lens, 8, 2, dim, 16, io, "nhd")
    close_by(s, lens, 2, dim, io)
    s["scale"] = scale
    for most in (2600, 2600 * 700):
        decode(s, 0, 0, most)
        for b, n in enumerate(lens):
            if n:
                check(s, b, slice(b, b + 1), torch.tensor([n - 1], device=DEV), n, single_error("e2m1", io),
                      "sequence %d of %d, planned for %d" % (b, n, most))


def chunk(s, lens, chunks, what, window=0, sinks=0):
    starts = others.prefill(s, chunks, window, sinks)
    for b, (n, c) in enumerate(zip(lens, chunks)):
        if c:
            check(s, b, slice(starts[b], starts[b + 1]), torch.arange(n - c, n, device=DEV), n, ref.half_step(s["io"]),
                  "%s, sequence %d, %d of %d tokens" % (what, b, c, n), window, sinks)


FEW = ([70, 300, 5], [70, 33, 1], 8, 2)   # on the single tokens' kernel


@pytest.mark.parametrize("size,by", [(1e4 * 4608, "scale"), (2.0 ** 33, "scale"), (1e30, "scale"), (0, "rows")])
@pytest.mark.parametrize("io,dim", [("bf16", 128), ("f16", 64), ("f16", 256)])
def test_few_rows_of_far_scores(io, dim, size, by):
    lens, chunks, heads, kv_heads = FEW
    s = setup("e2m1", lens, heads, kv_heads, dim, 16, io, "hnd", rows=sum(chunks))
    far_apart(s, lens, size, by, kv_heads, dim, io)
    chunk(s, lens, chunks, "few rows")


@pytest.mark.parametrize("scale", [0.34, 1.0, 16.0])
@pytest.mark.parametrize("io,dim", [("bf16", 128), ("f16", 64)])
def test_few_rows_of_close_scores(io, dim, scale):
    lens, chunks, heads, kv_heads = FEW
    s = setup("e2m1", lens, heads, kv_heads, dim, 16, io, "hnd", rows=sum(chunks))
    close_by(s, lens, kv_heads, dim, io)
    s["scale"] = scale
    chunk(s, lens, chunks, "few rows", 60, 3)


MANY = ([1200, 900], [1100, 700], 8, 4)   # on the tiles of 128 rows
CACHES = [("e2m1", "bf16", 128), ("e2m1", "f16", 64), ("e2m1", "f16", 192), ("bf16", "bf16", 128), ("f16", "f16", 96),
          ("f16", "f16", 256), ("e4m3", "bf16", 64), ("e4m3", "f16", 128)]


@pytest.mark.parametrize("size,by", [(1e4 * 4608, "scale"), (1e9, "scale"), (2.0 ** 33, "scale"), (1e30, "scale"),
                                     (-1e12, "scale"), (1e38, "scale"), (0, "rows")])
@pytest.mark.parametrize("cache,io,dim", CACHES)
def test_tiles_of_far_scores(cache, io, dim, size, by):
    if by == "rows" and cache == "e4m3":
        pytest.skip("its largest value is 448")
    lens, chunks, heads, kv_heads = MANY
    s = setup(cache, lens, heads, kv_heads, dim, 16, io, "hnd", rows=sum(chunks))
    far_apart(s, lens, size, by, kv_heads, dim, io)
    chunk(s, lens, chunks, "tiles")


@pytest.mark.parametrize("cache,io,dim", CACHES)
def test_tiles_of_single_tokens(cache, io, dim):
    """A window of 1: every row sees itself alone, at 2^33 and more."""
    lens, chunks, heads, kv_heads = MANY
    s = setup(cache, lens, heads, kv_heads, dim, 24, io, "nhd", rows=sum(chunks))
    s["scale"] = 2.0 ** 33
    chunk(s, lens, chunks, "window of 1", 1)


@pytest.mark.parametrize("scale", [0.25, 0.34, 0.5, 1.0, 16.0, -1.0])
@pytest.mark.parametrize("cache,io,dim", CACHES)
def test_tiles_of_close_scores(cache, io, dim, scale):
    lens, chunks, heads, kv_heads = MANY
    s = setup(cache, lens, heads, kv_heads, dim, 16, io, "hnd", rows=sum(chunks))
    close_by(s, lens, kv_heads, dim, io)
    s["scale"] = scale
    chunk(s, lens, chunks, "tiles")
    s["out"][:] = 0
    chunk(s, lens, chunks, "tiles, window", 200, 3)
