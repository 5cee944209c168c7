"""Attention over the paged cache against its definition in 64 bits, element by
element. Tolerances count roundings (kv_reference.attend_tolerance): the result's,
the weights' (two 16-bit pieces for a 16-bit output of a bfloat16 cache, three for an
f32 one, two of f16; one rounding in the chunked form), the scores' and the sums'
in f32. What lies in unused slots, unused pages and unseen tokens is NaN."""
import pytest
import torch

import kv_reference as ref
import quantized_decode_mat_amd as xq

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def setup(lens, heads, kv_heads, dim, page, cache, io, order, rows=None, seed=1, spare=3, poison=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    width = max(1, max(need)) + 1
    table = torch.full((len(lens), width + 2), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        at += n
    k = ref.pool(pages, kv_heads, page, dim, cache, order, g, DEV)
    v = ref.pool(pages, kv_heads, page, dim, cache, order, g, DEV)
    if poison:
        nan = float("nan")
        for b, n in enumerate(lens):
            if n % page:
                last = int(table[b, n // page])
                for x in (k, v):
                    x[last, :, n % page:] = torch.full_like(x[last, :, n % page:].float(), nan).to(x.dtype)
        for p in perm[at:]:
            for x in (k, v):
                x[p] = torch.full_like(x[p].float(), nan).to(x.dtype)
    scales = (0.75, 1.25) if cache == "e4m3" else (1.0, 1.0)
    rows = len(lens) if rows is None else rows
    # q and out are slices of wider rows
    wide = torch.randn(rows, heads + 3, dim, device=DEV, generator=g).to(ref.TYPES[io])
    out = torch.full((rows, heads + 1, dim), 7.0, dtype=ref.TYPES[io], device=DEV)
    return dict(kv=xq.xq_kv_cache(k, v, *scales), k=k, v=v, scales=scales, table=table.to(DEV)[:, :width],
                lens=torch.tensor(lens, dtype=torch.int32, device=DEV), q=wide[:, 1:heads + 1],
                full=out, out=out[:, :heads], page=page, scale=dim ** -0.5, io=io, cache=cache)


def expect(s, b, rows, pos, n, window, sinks):
    k, there = ref.rows_of(s["k"], s["table"][b], n, s["page"])
    v, _ = ref.rows_of(s["v"], s["table"][b], n, s["page"])
    return ref.attend(s["q"][rows], k * s["scales"][0], v * s["scales"][1], there, pos, s["scale"], window, sinks)


def compare(s, got, want, mag, slack, weight_error, n, what):
    tol = ref.attend_tolerance(want, mag, slack, s["io"], weight_error, n)
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), "%s: %d of %d outside, worst %.3g of the tolerance" % (
        what, int(bad.sum()), bad.numel(), float((err / tol).nan_to_num(9e9).max()))


def weight_error(cache, io):
    if cache == "bf16":
        return 2.0 ** -24 if io == "f32" else 2.0 ** -16
    return 2.0 ** -22


def decode(s, window, sinks, max_len, workspace=None, **kw):
    seqs, heads = s["q"].shape[:2]
    need = xq.xq_attn_decode_workspace_bytes(seqs, heads, s["kv"], max_len, window, sinks)
    if workspace is None and need:
        workspace = torch.zeros(need, dtype=torch.uint8, device=DEV)
    xq.xq_attn_decode(s["out"], s["q"], s["kv"], s["table"], s["lens"], s["scale"], window=window, sinks=sinks,
                      max_len=max_len, workspace=workspace, **kw)
    return workspace


def check_decode(s, lens, window, sinks, what):
    torch.cuda.synchronize()
    heads = s["q"].shape[1]
    assert (s["full"][:, heads:] == 7.0).all(), "%s: wrote past the heads" % what
    for b, n in enumerate(lens):
        pos = torch.tensor([n - 1], device=DEV)
        want, mag, slack = expect(s, b, slice(b, b + 1), pos, n, window, sinks)
        compare(s, s["out"][b:b + 1], want, mag, slack, weight_error(s["cache"], s["io"]), n,
                "%s, sequence %d of %d tokens" % (what, b, n))


DECODE = [
    # lens, heads, kv_heads, dim, page, cache, io, order, window, sinks
    ([1, 0, 2, 31, 32, 33], 8, 2, 128, 16, "bf16", "f32", "hnd", 0, 0),
    ([129, 517, 1, 0, 1000], 8, 8, 64, 1, "f16", "f16", "nhd", 0, 0),
    ([2500, 700], 5, 1, 80, 24, "e4m3", "bf16", "hnd", 0, 0),
    ([2500, 700, 90], 16, 2, 256, 8, "bf16", "bf16", "nhd", 300, 7),
    ([1300, 64], 20, 1, 96, 64, "f16", "f32", "hnd", 128, 0),
    ([1300, 64, 5], 6, 2, 192, 128, "e4m3", "f32", "nhd", 1, 3),
    ([777, 1], 4, 4, 16, 16, "bf16", "f16", "hnd", 50, 200),
    ([3000, 41, 0], 33, 1, 112, 32, "f16", "bf16", "nhd", 0, 0),
    ([3000, 2999], 8, 1, 192, 16, "bf16", "f32", "hnd", 2000, 1500),
    ([900], 16, 1, 256, 16, "f16", "f32", "hnd", 0, 0),
]


@pytest.mark.parametrize("case", DECODE, ids=lambda c: "-".join(str(x) for x in c[1:]))
def test_decode(case):
    lens, heads, kv_heads, dim, page, cache, io, order, window, sinks = case
    s = setup(lens, heads, kv_heads, dim, page, cache, io, order)
    ws = decode(s, window, sinks, max(lens))
    check_decode(s, lens, window, sinks, "decode")
    first = s["out"].clone()
    if ws is not None:
        assert not ws[:96 * 1024].any(), "arrival counters left standing"
    # again, on the same workspace and under a longer plan
    s["full"][:, :heads] = 0
    decode(s, window, sinks, max(lens), ws)
    assert torch.equal(s["out"], first), "the same call gave other bits"
    decode(s, window, sinks, 40 * max(lens))
    check_decode(s, lens, window, sinks, "decode, planned for more")


def test_decode_bad_pages_and_lengths():
    lens = [300, 200, 100]
    s = setup(lens, 4, 2, 64, 16, "bf16", "f32", "hnd", spare=2)
    pages = s["k"].shape[0]
    # a hole, pages past the pool, and a row without any page
    s["table"][0, 3], s["table"][0, 7] = -1, pages
    s["table"][1, 0], s["table"][1, 1] = 2 ** 31 - 1, -2 ** 31
    s["table"][2, :] = -5
    decode(s, 0, 0, 300)
    check_decode(s, lens, 0, 0, "bad pages")
    assert (s["out"][2] == 0).all()
    # lengths past the table, past max_len and below zero
    s = setup(lens, 4, 2, 64, 16, "bf16", "f32", "hnd", spare=2, poison=False)
    room = s["table"].shape[1] * 16
    s["lens"].copy_(torch.tensor([2 ** 31 - 1, 200, -4], dtype=torch.int32))
    decode(s, 0, 0, 10 ** 6)
    check_decode(s, [room, 200, 0], 0, 0, "long lengths")
    decode(s, 0, 0, 150)
    check_decode(s, [150, 150, 0], 0, 0, "max_len")


def test_decode_far_scores_and_values():
    """Scores hundreds apart, in either order, and values next to the type's largest."""
    lens = [640, 640]
    s = setup(lens, 4, 1, 128, 32, "bf16", "f32", "hnd", poison=False)
    j = torch.arange(640, device=DEV)
    rising = torch.where(torch.tensor([True, False], device=DEV)[:, None], j, 639 - j).float() / 64
    for b in range(2):
        p = s["table"][b].long()[j // 32]
        s["k"][p, :, j % 32] = (rising[b][:, None, None] * s["q"][b, :1].float()).to(torch.bfloat16)
        s["v"][p, :, j % 32] = (s["v"][p, :, j % 32].float() * 1e30).to(torch.bfloat16)
    s["q"] *= 4
    decode(s, 0, 0, 640)
    check_decode(s, lens, 0, 0, "far scores")


def test_decode_nan_and_infinity_that_are_seen():
    s = setup([100, 100], 4, 2, 64, 16, "f16", "f16", "hnd", poison=False)
    p = int(s["table"][0, 2])
    s["v"][p, 0, 5, 3] = float("inf")
    s["v"][p, 1, 5, 9] = float("nan")
    decode(s, 0, 0, 100)
    torch.cuda.synchronize()
    out = s["out"].float()
    assert (out[0, :2, 3] == float("inf")).all() and out[0, 2:, 9].isnan().all()
    out[0, :2, 3], out[0, 2:, 9] = 0, 0
    assert out.isfinite().all()
    s["k"][p, 0, 5, 3] = float("nan")
    decode(s, 0, 0, 100)
    assert s["out"][0, :2].isnan().all() and s["out"][1].isfinite().all()


def test_decode_past_32_bit_offsets():
    """Pages that begin past 2^32 elements of the pool."""
    page, kv_heads, dim = 64, 8, 128
    pages = (1 << 32) // (page * kv_heads * dim) + 200
    k = torch.empty(pages, kv_heads, page, dim, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    g = torch.Generator(device=DEV).manual_seed(3)
    ids = [pages - 1, 5, pages - 190, pages - 7, 0]
    for p in ids:
        k[p] = torch.randn(kv_heads, page, dim, device=DEV, generator=g)
        v[p] = torch.randn(kv_heads, page, dim, device=DEV, generator=g)
    lens = [page * len(ids) - 3]
    q = torch.randn(1, 16, dim, device=DEV, generator=g)
    out = torch.zeros(1, 17, dim, device=DEV)
    out[:, 16:] = 7.0
    s = dict(kv=xq.xq_kv_cache(k, v), k=k, v=v, scales=(1.0, 1.0), page=page, scale=dim ** -0.5, io="f32", cache="bf16",
             table=torch.tensor([ids], dtype=torch.int32, device=DEV), q=q, full=out, out=out[:, :16],
             lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    decode(s, 0, 0, lens[0])
    check_decode(s, lens, 0, 0, "far pages")


def test_decode_in_a_graph_on_another_stream():
    lens = [1500, 0, 700]
    s = setup(lens, 8, 2, 128, 16, "bf16", "f32", "hnd")
    ws = decode(s, 0, 0, 1500)
    torch.cuda.synchronize()
    want = s["out"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        decode(s, 0, 0, 1500, ws)
    for _ in range(4):
        s["full"][:, :8] = 5.0
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s["out"], want)
        decode(s, 0, 0, 1500, ws)
        torch.cuda.synchronize()
        assert torch.equal(s["out"], want)


PREFILL = [
    # lens, chunks, heads, kv_heads, dim, page, cache, io, order, window, sinks
    ([70, 5, 300], [70, 1, 33], 8, 2, 128, 16, "bf16", "bf16", "hnd", 0, 0),
    ([700, 129, 64], [200, 129, 64], 4, 4, 64, 24, "f16", "f16", "nhd", 0, 0),
    ([700, 129, 64], [200, 129, 64], 4, 1, 64, 24, "e4m3", "f16", "hnd", 100, 5),
    ([1100, 300], [256, 299], 5, 1, 80, 64, "e4m3", "bf16", "nhd", 0, 0),
    ([1100, 300, 2], [256, 299, 2], 6, 2, 96, 128, "bf16", "bf16", "nhd", 1, 70),
    ([500, 400], [130, 3], 4, 2, 256, 8, "bf16", "bf16", "hnd", 65, 200),
    ([500, 1], [500, 1], 3, 1, 192, 16, "f16", "f16", "hnd", 64, 0),
    ([900], [150], 20, 1, 16, 1, "f16", "f16", "nhd", 333, 64),
    ([900, 77], [64, 77], 2, 1, 256, 32, "e4m3", "f16", "hnd", 0, 0),
    ([0, 40, 0], [0, 40, 0], 8, 8, 112, 16, "bf16", "bf16", "hnd", 0, 0),
]


def prefill(s, chunks, window, sinks, first=0, most=None):
    starts = [first]
    for c in chunks:
        starts.append(starts[-1] + c)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    xq.xq_attn_prefill(s["out"], s["q"], s["kv"], s["table"], s["lens"], s["starts"], most or max(chunks), s["scale"],
                       window=window, sinks=sinks)
    return starts


def check_prefill(s, lens, chunks, starts, window, sinks, what):
    torch.cuda.synchronize()
    heads = s["q"].shape[1]
    assert (s["full"][:, heads:] == 7.0).all(), "%s: wrote past the heads" % what
    assert (s["full"][:starts[0]] == 7.0).all() and (s["full"][starts[-1]:] == 7.0).all(), "%s: other rows" % what
    for b, (n, c) in enumerate(zip(lens, chunks)):
        if c == 0:
            continue
        rows = slice(starts[b], starts[b + 1])
        pos = torch.arange(n - c, n, device=DEV)
        want, mag, slack = expect(s, b, rows, pos, n, window, sinks)
        compare(s, s["out"][rows], want, mag, slack, ref.half_step(s["io"]), n,
                "%s, sequence %d, %d of %d tokens" % (what, b, c, n))


@pytest.mark.parametrize("case", PREFILL, ids=lambda c: "-".join(str(x) for x in c[2:]))
def test_prefill(case):
    lens, chunks, heads, kv_heads, dim, page, cache, io, order, window, sinks = case
    s = setup(lens, heads, kv_heads, dim, page, cache, io, order, rows=sum(chunks) + 7)
    starts = prefill(s, chunks, window, sinks, first=4)
    check_prefill(s, lens, chunks, starts, window, sinks, "prefill")
    first = s["out"].clone()
    prefill(s, chunks, window, sinks, first=4)
    assert torch.equal(s["out"], first), "the same call gave other bits"


def test_prefill_bad_pages_and_starts():
    lens, chunks = [300, 200, 20], [100, 200, 20]
    s = setup(lens, 4, 2, 64, 16, "bf16", "bf16", "hnd", rows=320)
    s["table"][0, 3], s["table"][0, 17], s["table"][2, :] = -1, s["k"].shape[0], -1
    starts = prefill(s, chunks, 0, 0)
    check_prefill(s, lens, chunks, starts, 0, 0, "bad pages")
    assert (s["out"][300:] == 0).all()
    # fewer tokens in the cache than in the chunk: the first rows see nothing
    s = setup([10, 64], 4, 2, 64, 16, "bf16", "bf16", "hnd", rows=200)
    starts = prefill(s, [30, 64], 0, 0)
    check_prefill(s, [10, 64], [30, 64], starts, 0, 0, "short cache")
    assert (s["out"][:20] == 0).all()
    # starts outside the rows, descending, and a chunk above max_chunk
    s = setup([64, 64, 64], 4, 2, 64, 16, "bf16", "bf16", "hnd", rows=100)
    s["starts"] = torch.tensor([-5, 40, 20, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    xq.xq_attn_prefill(s["out"], s["q"], s["kv"], s["table"], s["lens"], s["starts"], 40, s["scale"])
    torch.cuda.synchronize()
    assert (s["full"][60:] == 7.0).all() and s["out"][:60].isfinite().all()


@pytest.mark.parametrize("cache,io", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16")])
def test_prefill_unseen_tokens_have_no_influence(cache, io):
    """Later tokens of the chunk, and tokens before the window, hold NaN and infinities in k and v."""
    lens, chunks, window, sinks = [400, 90], [400, 60], 70, 3
    s = setup(lens, 4, 2, 96, 16, cache, io, "hnd", rows=460, poison=False)
    clean = setup(lens, 4, 2, 96, 16, cache, io, "hnd", rows=460, poison=False)
    starts = prefill(clean, chunks, window, sinks)
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


def test_prefill_and_decode_agree():
    """The last row of a chunk is the single token's result."""
    lens = [333, 64, 1]
    s = setup(lens, 8, 2, 128, 16, "f16", "f16", "hnd")
    decode(s, 90, 4, 333)
    one = s["out"].clone()
    prefill(s, [1, 1, 1], 90, 4)
    torch.cuda.synchronize()
    check_prefill(s, lens, [1, 1, 1], [0, 1, 2, 3], 90, 4, "single rows")
    assert (one.double() - s["out"].double()).abs().max() < 2.0 ** -9


def test_prefill_in_a_graph():
    lens, chunks = [300, 64], [100, 64]
    s = setup(lens, 8, 2, 128, 16, "bf16", "bf16", "hnd", rows=164)
    prefill(s, chunks, 0, 0)
    torch.cuda.synchronize()
    want = s["out"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        xq.xq_attn_prefill(s["out"], s["q"], s["kv"], s["table"], s["lens"], s["starts"], 100, s["scale"])
    for _ in range(3):
        s["full"][:, :8] = 5.0
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s["out"], want)
