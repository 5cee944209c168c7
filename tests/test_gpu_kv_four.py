"""The 4-bit cache: the append's codes and powers against the definition in 64 bits (equal, byte for byte), tokens
read back, attention element by element with the tolerances of kv_reference (which count roundings), its pages.

Weights enter their product with v as bf16 pieces: two (2^-16) for a 16-bit output, three (2^-24) for f32's; a chunk's
as one rounding of its type. q is exact in its pieces. Unused slots, pages and unseen tokens hold NaN (power 255)."""
import importlib.util
import os

import pytest
import torch

import four_reference as four
import kv_reference as ref
import quantized_decode_mat_amd as xq
from test_gpu_kv_attention import _device, check_decode, check_prefill, compare, decode, prefill  # noqa: F401
from test_gpu_kv_rope_pages import check_rope, freqs, positions

pytestmark = pytest.mark.gpu
DEV = "cuda"


def setup(lens, heads, kv_heads, dim, page, io, order, rows=None, seed=1, spare=3, poison=True, layers=()):
    g = torch.Generator(device=DEV).manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    width = max(1, max(need)) + 1
    table, at = torch.full((len(lens), width), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        at += n
    k, k_exp = four.pool(pages, kv_heads, page, dim, order, g, DEV, layers)
    v, v_exp = four.pool(pages, kv_heads, page, dim, order, g, DEV, layers)
    if poison:
        for x in (k_exp, v_exp):
            for b, n in enumerate(lens):
                if n % page:
                    x[..., int(table[b, n // page]), :, n % page:, :] = 255
            for p in perm[at:]:
                x[..., p, :, :, :] = 255
    rows = len(lens) if rows is None else rows
    wide = torch.randn(rows, heads + 3, dim, device=DEV, generator=g).to(ref.TYPES[io])
    out = torch.full((rows, heads + 1, dim), 7.0, dtype=ref.TYPES[io], device=DEV)
    scales = (0.75, 1.25)
    return dict(kv=four.cache(xq, k, k_exp, v, v_exp, scales), k=k, v=v, k_exp=k_exp, v_exp=v_exp, scales=scales,
                table=table.to(DEV), lens=torch.tensor(lens, dtype=torch.int32, device=DEV), q=wide[:, 1:heads + 1],
                full=out, out=out[:, :heads], page=page, scale=dim ** -0.5, io=io)


def check_rows(s, got, rows, b, pos, n, window, sinks, weight_error, what):
    torch.cuda.synchronize()
    want, mag, slack = four.attend(s, rows, b, pos, n, window, sinks)
    compare(s, got, want, mag, slack, weight_error, n, what)


def check_single(s, lens, window, sinks, what):
    torch.cuda.synchronize()
    assert (s["full"][:, s["q"].shape[1]:] == 7.0).all(), what
    for b, n in enumerate(lens):
        check_rows(s, s["out"][b:b + 1], slice(b, b + 1), b, torch.tensor([n - 1], device=DEV), n, window, sinks,
                   2.0 ** -24 if s["io"] == "f32" else 2.0 ** -16, "%s, sequence %d of %d" % (what, b, n))


def check_chunks(s, lens, chunks, starts, window, sinks, what):
    torch.cuda.synchronize()
    heads = s["q"].shape[1]
    assert (s["full"][:, heads:] == 7.0).all(), what
    assert (s["full"][:starts[0]] == 7.0).all() and (s["full"][starts[-1]:] == 7.0).all(), "%s: other rows" % what
    for b, (n, c) in enumerate(zip(lens, chunks)):
        if c:
            rows = slice(starts[b], starts[b + 1])
            check_rows(s, s["out"][rows], rows, b, torch.arange(n - c, n, device=DEV), n, window, sinks,
                       ref.half_step(s["io"]), "%s, sequence %d, %d of %d tokens" % (what, b, c, n))


# ---------------------------------------------------------------- append and read

APPEND = [
    # tokens, heads, kv_heads, dim, rot, sections, adjacent, page, src, io, order
    (1, 4, 1, 64, 64, [32], False, 16, "f32", "f32", "hnd"),
    (37, 8, 2, 128, 128, [24, 20, 20], False, 16, "bf16", "bf16", "nhd"),
    (37, 6, 3, 96, 48, [24], True, 24, "f16", "f32", "hnd"),
    (19, 5, 5, 32, 24, [4, 8], False, 1, "f32", "f16", "nhd"),
    (9, 2, 1, 160, 80, [10, 10, 10, 10], True, 8, "bf16", "f32", "hnd"),
    (65, 16, 2, 256, 256, [128], False, 64, "f16", "f16", "nhd"),
    (2100, 3, 1, 224, 8, [4], False, 32, "f32", "bf16", "hnd"),
    (300, 1, 1, 192, 192, [96], True, 16, "bf16", "bf16", "hnd"),
    (4097, 4, 2, 128, 128, [24, 20, 20], False, 16, "bf16", "bf16", "nhd"),  # four tokens a workgroup
    (5002, 1, 1, 32, 16, [8], True, 64, "f32", "f16", "hnd"),
    (4099, 3, 9, 256, 200, [60, 40], False, 8, "f16", "f32", "hnd"),         # more than 256 quarters a token
]


def append_state(case, seed=1):
    tokens, heads, kv_heads, dim, rot, sections, adjacent, page, src, io, order = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    pages = -(-tokens // page) + 3
    k, k_exp = four.pool(pages, kv_heads, page, dim, order, g, DEV)
    v, v_exp = four.pool(pages, kv_heads, page, dim, order, g, DEV)
    x = torch.randn(tokens, heads + 2 * kv_heads, dim, device=DEV, generator=g).to(ref.TYPES[src])
    return dict(k=k, v=v, k_exp=k_exp, v_exp=v_exp, x=x, pos=positions(len(sections), tokens, 150000, seed),
                plan=xq.xq_rope_plan(freqs(rot), sections, adjacent), page=page, pages=pages,
                slots=torch.randperm(pages * page, device=DEV, generator=g)[:tokens],
                out=torch.full((tokens, heads + 1, dim), 7.0, dtype=ref.TYPES[io], device=DEV))


def append(s, heads, kv_heads, scales):
    kv = four.cache(xq, s["k"], s["k_exp"], s["v"], s["v_exp"], scales)
    x = s["x"]
    xq.xq_rope_append(s["out"][:, :heads], kv, x[:, :heads], x[:, heads:heads + kv_heads], x[:, heads + kv_heads:],
                      s["pos"], s["plan"], s["slots"])
    torch.cuda.synchronize()
    return kv


def check_append(s, before, heads, kv_heads, sections, adjacent, scales, rows=None):
    """Every byte of the pool: the appended rows' as defined, all others as they were."""
    x, dim = s["x"].double(), s["x"].shape[-1]
    turned = ref.rotate(x[:, heads:heads + kv_heads], s["pos"], s["plan"].freq, sections, adjacent, False)
    rows = torch.ones(len(x), dtype=torch.bool, device=DEV) if rows is None else rows
    at, slot = s["slots"][rows] // s["page"], s["slots"][rows] % s["page"]
    for name, value, scale in (("k", turned, scales[0]), ("v", x[:, heads + kv_heads:], scales[1])):
        codes, powers, nan = four.encode(value[rows] / torch.tensor(scale, dtype=torch.float32).double())
        want, want_exp = before[name].clone(), before[name + "_exp"].clone()
        want[at, :, slot] = codes
        want_exp[at, :, slot, :dim // 32] = powers
        got, got_exp = s[name].clone(), s[name + "_exp"]
        assert torch.equal(got_exp, want_exp), "%s: %d powers differ" % (name, int((got_exp != want_exp).sum()))
        # (a block that holds a NaN is NaN whatever its codes)
        hidden = nan.repeat_interleave(16, -1)
        got[at, :, slot], want[at, :, slot] = got[at, :, slot].masked_fill(hidden, 0), codes.masked_fill(hidden, 0)
        assert torch.equal(got, want), "%s: %d bytes of codes differ" % (name, int((got != want).sum()))


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(str(x) for x in c))
def test_append(case):
    tokens, heads, kv_heads, dim, rot, sections, adjacent, page, src, io, order = case
    for scales in ((0.75, 1.25), (1.0, 1.0)):
        s = append_state(case)
        if tokens > 4:
            s["slots"][3], s["slots"][1] = -1, page * s["pages"]
        before = {n: s[n].clone() for n in ("k", "v", "k_exp", "v_exp")}
        append(s, heads, kv_heads, scales)
        assert (s["out"][:, heads:] == 7.0).all()
        check_rope(s["out"][:, :heads], s["x"][:, :heads], s["pos"], s["plan"], sections, adjacent, False, io)
        ok = (s["slots"] >= 0) & (s["slots"] < page * s["pages"])
        check_append(s, before, heads, kv_heads, sections, adjacent, scales, ok)


def test_append_borders_zeros_and_what_is_not_finite():
    """Values on the borders between codes (times a scale that they divide by exactly), blocks of zeros, far sizes,
    infinities (they saturate) and NaN (its block is NaN)."""
    case = (40, 1, 1, 128, 8, [4], False, 16, "f32", "f32", "hnd")
    s = append_state(case)
    s["pos"].zero_()                                        # the angle is 0: k comes as it is
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 6.5, 0.0], device=DEV)
    near = torch.cat([borders, torch.nextafter(borders, borders + 9), torch.nextafter(borders, borders - 9)])
    x = torch.zeros(40, 3, 128, device=DEV)
    for t in range(12):
        for w, scale in ((1, 0.75), (2, 1.25)):
            x[t, w, :30] = near * 2.0 ** (t - 6)
            x[t, w, 32:62] = -near * 2.0 ** (3 * t - 20)
            x[t, w, 64:94] = near * 2.0 ** (t - 6) * scale  # exact: 2 and 3 bits more
            x[t, w, 94] = 6.9 * 2.0 ** (t - 6) * scale
    for t, top in enumerate([7.0, 6.9999995, 3.5, 65504.0, 49152.0, 57343.9, 57344.0, 3e38, 1e-30, 2.0 ** -22, 1.4e-45]):
        x[12 + t, :, 32] = top
        x[12 + t, :, 33:40] = top / 3
        x[12 + t, :, 70] = -top
    x[25, 1, 5], x[25, 2, 40] = float("inf"), -float("inf")
    x[26, 1, 5], x[26, 2, 40] = float("nan"), float("nan")
    x[27] = -0.0
    s["x"] = x
    for scales in ((1.0, 1.0), (0.75, 1.25), (3e-39, 1e30)):
        before = {n: s[n].clone() for n in ("k", "v", "k_exp", "v_exp")}
        kv = append(s, 1, 1, scales)
        check_append(s, before, 1, 1, [4], False, scales)
        back = torch.empty(2, 40, 1, 128, device=DEV)
        xq.xq_cache_read(back[0], back[1], kv, s["slots"])
        assert back[0, 26, 0, :32].isnan().all() and back[1, 26, 0, 32:64].isnan().all()
        assert back[0, 25, 0, :32].isnan().all()            # an infinity turned: 0 times it is NaN
        assert int(back.isnan().sum()) == 96


@pytest.mark.parametrize("rot,src", [(128, "bf16"), (40, "f32"), (72, "f16")])
def test_append_with_q_in_place(rot, src):
    """q_out is q, among k and v in one product's output."""
    s = append_state((70, 6, 2, 128, rot, [rot // 2], False, 16, src, src, "hnd"))
    before = {n: s[n].clone() for n in ("k", "v", "k_exp", "v_exp")}
    x = s["x"].clone()
    s["out"] = s["x"]
    append(s, 6, 2, (0.75, 1.25))
    check_rope(s["x"][:, :6], x[:, :6], s["pos"], s["plan"], [rot // 2], False, False, src)
    assert torch.equal(s["x"][:, 6:], x[:, 6:])
    check_append(dict(s, x=x), before, 6, 2, [rot // 2], False, (0.75, 1.25))


def test_append_of_unaligned_rows():
    case = (21, 2, 2, 64, 32, [16], False, 16, "bf16", "f32", "hnd")
    s = append_state(case)
    flat = torch.zeros(21 * 6 * 67 + 1, dtype=torch.bfloat16, device=DEV)
    odd = flat[1:].as_strided((21, 6, 64), (6 * 67, 67, 1))
    odd.copy_(s["x"])
    s["x"] = odd
    before = {n: s[n].clone() for n in ("k", "v", "k_exp", "v_exp")}
    append(s, 2, 2, (0.75, 1.25))
    check_append(s, before, 2, 2, [16], False, (0.75, 1.25))


@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3", "e2m1"])
@pytest.mark.parametrize("io", ["f32", "bf16", "f16"])
def test_read(kind, io):
    g = torch.Generator(device=DEV).manual_seed(4)
    pages, heads, page, dim, scales = 9, 3, 8, 96, (0.7, 1.3)
    if kind == "e2m1":
        k, k_exp = four.pool(pages, heads, page, dim, "nhd", g, DEV)
        v, v_exp = four.pool(pages, heads, page, dim, "nhd", g, DEV)
        kv, values = four.cache(xq, k, k_exp, v, v_exp, scales), [four.values(k, k_exp), four.values(v, v_exp)]
    else:
        k, v = (ref.pool(pages, heads, page, dim, kind, "nhd", g, DEV) for _ in range(2))
        kv, values = xq.xq_kv_cache(k, v, *scales), [ref.as_f64(k), ref.as_f64(v)]
    slots = torch.tensor([5, 71, 0, 5, -1, 72, 2 ** 40, -2 ** 62, 33], device=DEV)
    for wide in (dim, dim + 1):
        outs = [torch.full((9, heads + 1, wide), 7.0, dtype=ref.TYPES[io], device=DEV) for _ in range(2)]
        got = [x[:, :heads, :dim] for x in outs]
        xq.xq_cache_read(got[0], got[1], kv, slots)
        torch.cuda.synchronize()
        ok = (slots >= 0) & (slots < 72)
        at = slots.clamp(0, 71)
        for x, y, z, scale in zip(got, values, outs, scales):
            want = (y[at // page, :, at % page].float() * scale).to(ref.TYPES[io])
            want[~ok] = 0
            assert torch.equal(x, want)
            assert (z[:, heads:] == 7.0).all() and (z[:, :, dim:] == 7.0).all()


# ---------------------------------------------------------------- attention

DECODE = [
    # lens, heads, kv_heads, dim, page, io, order, window, sinks
    ([1, 0, 2, 31, 32, 33], 8, 2, 128, 16, "f32", "hnd", 0, 0),
    ([129, 517, 1, 0, 1000], 8, 8, 64, 1, "f16", "nhd", 0, 0),
    ([2500, 700], 5, 1, 32, 24, "bf16", "hnd", 0, 0),
    ([2500, 700, 90], 16, 2, 256, 8, "bf16", "nhd", 300, 7),
    ([1300, 64], 20, 1, 96, 64, "f32", "hnd", 128, 0),
    ([1300, 64, 5], 6, 2, 192, 128, "f32", "nhd", 1, 3),
    ([777, 1], 4, 4, 160, 16, "f16", "hnd", 50, 200),
    ([3000, 41, 0], 33, 1, 224, 32, "bf16", "nhd", 0, 0),
    ([3000, 2999], 8, 1, 192, 16, "f16", "hnd", 2000, 1500),
    ([900], 16, 1, 256, 16, "f32", "hnd", 0, 0),
    ([5000, 60], 7, 1, 128, 16, "f32", "nhd", 0, 0),
    ([400] * 70, 8, 8, 128, 16, "bf16", "hnd", 0, 0),
]


@pytest.mark.parametrize("case", DECODE, ids=lambda c: "-".join(str(x) for x in c[1:]))
def test_decode(case):
    lens, heads, kv_heads, dim, page, io, order, window, sinks = case
    s = setup(lens, heads, kv_heads, dim, page, io, order)
    ws = decode(s, window, sinks, max(lens))
    check_single(s, lens, window, sinks, "decode")
    first = s["out"].clone()
    if ws is not None:
        assert not ws[:96 * 1024].any(), "arrival counters left standing"
    s["full"][:, :heads] = 0
    decode(s, window, sinks, max(lens), ws)
    assert torch.equal(s["out"], first), "the same call gave other bits"
    decode(s, window, sinks, 40 * max(lens))
    check_single(s, lens, window, sinks, "decode, planned for more")


def test_decode_bad_pages_and_lengths():
    lens = [300, 200, 100]
    s = setup(lens, 4, 2, 64, 16, "f32", "hnd", spare=2)
    pages = s["k"].shape[0]
    s["table"][0, 3], s["table"][0, 7] = -1, pages
    s["table"][1, 0], s["table"][1, 1] = 2 ** 31 - 1, -2 ** 31
    s["table"][2, :] = -5
    decode(s, 0, 0, 300)
    check_single(s, lens, 0, 0, "bad pages")
    assert (s["out"][2] == 0).all()
    s = setup(lens, 4, 2, 64, 16, "f32", "hnd", spare=2, poison=False)
    room = s["table"].shape[1] * 16
    s["lens"].copy_(torch.tensor([2 ** 31 - 1, 200, -4], dtype=torch.int32))
    decode(s, 0, 0, 10 ** 6)
    check_single(s, [room, 200, 0], 0, 0, "long lengths")


def test_decode_nan_that_is_seen():
    s = setup([100, 100], 4, 2, 64, 16, "f16", "hnd", poison=False)
    p = int(s["table"][0, 2])
    s["v_exp"][p, 0, 5, 1] = 255
    decode(s, 0, 0, 100)
    out = s["out"].float()
    assert out[0, :2, 32:].isnan().all()
    out[0, :2, 32:] = 0
    assert out.isfinite().all()
    s["k_exp"][p, 0, 5, 0] = 255
    decode(s, 0, 0, 100)
    assert s["out"][0, :2].isnan().all() and s["out"][0, 2:].isfinite().all() and s["out"][1].isfinite().all()


@pytest.mark.parametrize("low,high", [(104, 112), (132, 140), (2, 4), (237, 241)])
def test_powers_at_the_ends(low, high):
    """The smallest and largest powers that the append stores, and those that are read beside them: 700 tokens of up to
    6 * 2^114 add up to less than 2^127."""
    g = torch.Generator(device=DEV).manual_seed(2)
    s = setup([700], 4, 2, 128, 16, "f32", "hnd")
    for x in (s["k_exp"], s["v_exp"]):
        new = torch.randint(low, high + 1, x.shape, device=DEV, dtype=torch.int32, generator=g).to(torch.uint8)
        x.copy_(torch.where(x == 255, x, new))
    # scores of a size that f32 holds
    s["scale"] = 2.0 ** min(100, 127 - high)
    s["q"] *= 0.05
    decode(s, 0, 0, 700)
    check_single(s, [700], 0, 0, "powers %d..%d" % (low, high))


def test_read_of_all_powers():
    g = torch.Generator(device=DEV).manual_seed(2)
    k, k_exp = four.pool(16, 1, 16, 32, "hnd", g, DEV)
    v, v_exp = four.pool(16, 1, 16, 32, "hnd", g, DEV)
    byte = torch.arange(256, device=DEV).clamp(max=250).view(16, 1, 16).to(torch.uint8)
    k_exp[..., 0], v_exp[..., 0] = byte, 250 - byte
    got = [torch.empty(256, 1, 32, device=DEV) for _ in range(2)]
    xq.xq_cache_read(got[0], got[1], four.cache(xq, k, k_exp, v, v_exp, (1.0, 1.0)), torch.arange(256, device=DEV))
    for x, want in zip(got, (four.values(k, k_exp), four.values(v, v_exp))):
        want = want.view(256, 1, 32)
        normal = (want == 0) | (want.abs() >= 2.0 ** -126)
        assert torch.equal(x.double()[normal], want[normal])


def test_decode_past_32_bit_offsets():
    """Pages whose codes begin past 2^32 bytes of the pool."""
    page, kv_heads, dim = 64, 8, 128
    pages = (1 << 33) // (page * kv_heads * dim) + 200
    g = torch.Generator(device=DEV).manual_seed(3)
    k, v = (torch.empty(pages, kv_heads, page, dim // 2, dtype=torch.uint8, device=DEV) for _ in range(2))
    k_exp, v_exp = (torch.full((pages, kv_heads, page, 4), 255, dtype=torch.uint8, device=DEV) for _ in range(2))
    ids = [pages - 1, 5, pages - 190, pages - 7, 0]
    for p in ids:
        for codes, exps in ((k, k_exp), (v, v_exp)):
            one = four.pool(1, kv_heads, page, dim, "hnd", g, DEV)
            codes[p], exps[p] = one[0][0], one[1][0]
    lens = [page * len(ids) - 3]
    q = torch.randn(1, 16, dim, device=DEV, generator=g)
    out = torch.full((1, 17, dim), 7.0, device=DEV)
    s = dict(kv=four.cache(xq, k, k_exp, v, v_exp, (1.0, 1.0)), k=k, v=v, k_exp=k_exp, v_exp=v_exp, scales=(1.0, 1.0),
             page=page, scale=dim ** -0.5, io="f32", table=torch.tensor([ids], dtype=torch.int32, device=DEV), q=q,
             full=out, out=out[:, :16], lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    decode(s, 0, 0, lens[0])
    check_single(s, lens, 0, 0, "far pages")


def test_decode_in_a_graph_on_another_stream():
    lens = [1500, 0, 700]
    s = setup(lens, 8, 2, 128, 16, "f32", "hnd")
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


def test_decode_at_once_on_two_streams():
    """A call whose parts are joined, one whose are not, and one of many parts, each on two streams."""
    runs = []
    for lens, heads, io in (([5000, 300], 8, "f32"), ([700, 40], 8, "bf16"), ([9000], 4, "f16")):
        a, b = (setup(lens, heads, 2, 128, 16, io, "hnd", seed=seed) for seed in (1, 2))
        runs.append((lens, a, b, decode(a, 0, 0, max(lens)), decode(b, 0, 0, max(lens))))
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for lens, a, b, wa, wb in runs:
        a["full"][:, :a["q"].shape[1]] = 5.0
        b["full"][:, :b["q"].shape[1]] = 5.0
    torch.cuda.synchronize()
    for _ in range(10):
        for lens, a, b, wa, wb in runs:
            decode(a, 0, 0, max(lens), wa, stream=one)
            decode(b, 0, 0, max(lens), wb, stream=two)
    for lens, a, b, wa, wb in runs:
        check_single(a, lens, 0, 0, "first stream")
        check_single(b, lens, 0, 0, "second stream")


@pytest.mark.parametrize("scale", [-0.11, 0.0, 1e-30, -1e-40])
def test_scales_of_scores(scale):
    """Negative: the order of the scores turns round; 0: all tokens weigh the same."""
    lens = [1900, 33, 0, 600]
    s = setup(lens, 8, 2, 128, 16, "f32", "nhd")
    s["scale"] = scale
    decode(s, 0, 0, 1900)
    check_single(s, lens, 0, 0, "scale %g" % scale)
    decode(s, 100, 3, 1900)
    check_single(s, lens, 100, 3, "scale %g, window" % scale)
    for lens, chunks, heads in (([300, 90], [200, 60], 4), ([900, 1000], [900, 1000], 16)):
        s = setup(lens, heads, 4, 64, 16, "bf16", "hnd", rows=sum(chunks))
        s["scale"] = scale
        starts = prefill(s, chunks, 70, 3)
        check_chunks(s, lens, chunks, starts, 70, 3, "chunk, scale %g" % scale)


CHUNK = [
    # lens, chunks, heads, kv_heads, dim, page, io, order, window, sinks, copies
    ([70, 5, 300], [70, 1, 33], 8, 2, 128, 16, "bf16", "hnd", 0, 0),
    ([700, 129, 64], [200, 129, 64], 4, 4, 64, 24, "f16", "nhd", 0, 0),
    ([700, 129, 64], [200, 129, 64], 4, 1, 64, 24, "bf16", "hnd", 100, 5),
    ([1100, 300], [256, 299], 5, 1, 160, 64, "bf16", "nhd", 0, 0),
    ([1100, 300, 2], [256, 299, 2], 6, 2, 96, 128, "f16", "nhd", 1, 70),
    ([500, 400], [130, 3], 4, 2, 256, 8, "bf16", "hnd", 65, 200),
    ([500, 1], [500, 1], 3, 1, 192, 16, "f16", "hnd", 64, 0),
    ([900], [150], 20, 1, 32, 1, "f16", "nhd", 333, 64),
    ([900, 77], [64, 77], 2, 1, 256, 32, "f16", "hnd", 0, 0),
    ([0, 40, 0], [0, 40, 0], 8, 8, 224, 16, "bf16", "hnd", 0, 0),
    # enough rows for the tiles of 128
    ([1200, 900, 1100], [1200, 700, 1100], 8, 4, 128, 16, "bf16", "nhd", 0, 0),
    ([1200, 900, 1100], [1200, 700, 1100], 8, 4, 128, 64, "f16", "hnd", 200, 70),
    ([1200, 900, 1100], [1200, 700, 1100], 4, 4, 64, 24, "f16", "hnd", 0, 0),
    ([1200, 900], [1100, 700], 10, 5, 96, 16, "bf16", "hnd", 0, 0),
    ([1500, 900], [1500, 900], 6, 6, 192, 16, "bf16", "hnd", 100, 3),
    ([1500, 900], [1500, 900], 6, 6, 224, 16, "f16", "nhd", 0, 0),
    ([1500, 900], [1500, 900], 6, 6, 256, 16, "f16", "nhd", 700, 1),
]


@pytest.mark.parametrize("case", CHUNK, ids=lambda c: "-".join(str(x) for x in c[2:]) + "-%d" % c[0][0])
def test_chunk(case):
    lens, chunks, heads, kv_heads, dim, page, io, order, window, sinks = case
    s = setup(lens, heads, kv_heads, dim, page, io, order, rows=sum(chunks) + 7)
    starts = prefill(s, chunks, window, sinks, first=4)
    check_chunks(s, lens, chunks, starts, window, sinks, "chunk")
    first = s["out"].clone()
    prefill(s, chunks, window, sinks, first=4)
    assert torch.equal(s["out"], first), "the same call gave other bits"


@pytest.mark.parametrize("io", ["bf16", "f16"])
@pytest.mark.parametrize("lens,chunks,heads", [([400, 90], [400, 60], 4), ([900, 1000], [900, 1000], 16)])
def test_chunk_unseen_tokens_have_no_influence(io, lens, chunks, heads):
    """A token behind some rows' window and ahead of others is NaN in k, and in half of v's blocks."""
    window, sinks, bad = 70, 3, 250
    rows = sum(chunks)
    s = setup(lens, heads, 4, 64, 16, io, "hnd", rows=rows, poison=False)
    clean = setup(lens, heads, 4, 64, 16, io, "hnd", rows=rows, poison=False)
    prefill(clean, chunks, window, sinks)
    p = int(s["table"][0, bad // 16])
    s["v_exp"][p, :, bad % 16, 1] = 255
    prefill(s, chunks, window, sinks)
    torch.cuda.synchronize()
    got, want = s["out"], clean["out"]
    assert torch.equal(got[:bad], want[:bad]) and torch.equal(got[bad + window:], want[bad + window:])
    assert got[bad:bad + window, :, 32:].isnan().all() and torch.equal(got[bad:bad + window, :, :32], want[bad:bad + window, :, :32])
    s["k_exp"][p, :, bad % 16, 0] = 255
    prefill(s, chunks, window, sinks)
    torch.cuda.synchronize()
    assert torch.equal(got[:bad], want[:bad]) and torch.equal(got[bad + window:], want[bad + window:])
    assert got[bad:bad + window].isnan().all()


def test_chunk_in_a_graph_and_bad_pages():
    lens, chunks = [300, 200, 20], [100, 200, 20]
    s = setup(lens, 4, 2, 64, 16, "bf16", "hnd", rows=320)
    s["table"][0, 3], s["table"][0, 17], s["table"][2, :] = -1, s["k"].shape[0], -1
    starts = prefill(s, chunks, 0, 0)
    check_chunks(s, lens, chunks, starts, 0, 0, "bad pages")
    assert (s["out"][300:] == 0).all()
    want = s["out"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        xq.xq_attn_prefill(s["out"], s["q"], s["kv"], s["table"], s["lens"], s["starts"], 200, s["scale"])
    for _ in range(3):
        s["full"][:, :4] = 5.0
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s["out"], want)


# ---------------------------------------------------------------- pages

@pytest.mark.parametrize("order,dim", [("hnd", 128), ("nhd", 192), ("hnd", 32)])
def test_pages_move_with_their_powers(order, dim):
    """Copy, fork and compact against the same moves of bytes."""
    g = torch.Generator(device=DEV).manual_seed(5)
    k, k_exp = four.pool(24, 2, 16, dim, order, g, DEV, (3,))
    v, v_exp = four.pool(24, 2, 16, dim, order, g, DEV, (3,))
    kv = four.cache(xq, k, k_exp, v, v_exp, (1.0, 1.0))
    pool = dict(k=k, v=v, k_exp=k_exp, v_exp=v_exp)
    ints = dict(dtype=torch.int32, device=DEV)

    def moved(before, pairs):
        for name, x in pool.items():
            want = before[name].clone()
            for a, b in pairs:
                want[:, b] = before[name][:, a]
            assert torch.equal(x, want), name

    before = {n: x.clone() for n, x in pool.items()}
    xq.xq_cache_copy(kv, torch.tensor([3, 7, 99, 4], **ints), torch.tensor([5, 0, 1, 4], **ints))
    moved(before, [(3, 5), (7, 0)])
    refs, tables, lens = torch.zeros(24, **ints), torch.full((4, 6), -1, **ints), torch.zeros(4, **ints)
    tables[0, :3], lens[0] = torch.tensor([20, 11, 17], **ints), 40
    refs[[20, 11, 17]] = 1
    status = torch.zeros(2, **ints)
    ws = torch.zeros(xq.xq_cache_workspace_bytes(24, 4), dtype=torch.uint8, device=DEV)
    before = {n: x.clone() for n, x in pool.items()}
    xq.xq_cache_fork(kv, refs, tables, lens, torch.tensor([0], **ints), torch.tensor([2], **ints), status, workspace=ws)
    assert status.tolist() == [0, 0] and tables[2].tolist() == [20, 11, 0, -1, -1, -1]
    moved(before, [(17, 0)])
    before = {n: x.clone() for n, x in pool.items()}
    xq.xq_cache_compact(kv, refs, tables, status, workspace=ws)
    assert status.tolist() == [0, 4] and tables[0, :3].tolist() == [3, 1, 2]
    moved(before, [(11, 1), (17, 2), (20, 3)])


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_prompt_then_tokens(io):
    """A prompt's append and chunk attention, then single tokens appended and attended to, as a server runs them."""
    heads, kv_heads, dim, page, prompt, more = 8, 2, 128, 16, 75, 6
    g = torch.Generator(device=DEV).manual_seed(6)
    k, k_exp = four.pool(8, kv_heads, page, dim, "hnd", g, DEV)
    v, v_exp = four.pool(8, kv_heads, page, dim, "hnd", g, DEV)
    scales = (0.5, 2.0)
    kv = four.cache(xq, k, k_exp, v, v_exp, scales)
    table = torch.tensor([[5, 0, 7, 2, 4, 1]], dtype=torch.int32, device=DEV)
    plan = xq.xq_rope_plan(freqs(dim), [dim // 2])
    s = dict(k=k, v=v, k_exp=k_exp, v_exp=v_exp, table=table, page=page, scale=dim ** -0.5, scales=scales, kv=kv)
    ws = torch.zeros(xq.xq_attn_decode_workspace_bytes(1, heads, kv, 96), dtype=torch.uint8, device=DEV)
    n = 0
    for count in [prompt] + [1] * more:
        t = torch.bfloat16 if count > 1 else ref.TYPES[io]
        x = torch.randn(count, heads + 2 * kv_heads, dim, device=DEV, generator=g)
        j = torch.arange(n, n + count, device=DEV)
        slots = table[0].long()[j // page] * page + j % page
        q = torch.empty(count, heads, dim, dtype=t, device=DEV)
        xq.xq_rope_append(q, kv, x[:, :heads], x[:, heads:heads + kv_heads], x[:, heads + kv_heads:], j.int(), plan, slots)
        n += count
        lens = torch.tensor([n], dtype=torch.int32, device=DEV)
        out = torch.empty_like(q)
        if count > 1:
            starts = torch.tensor([0, count], dtype=torch.int32, device=DEV)
            xq.xq_attn_prefill(out, q, kv, table, lens, starts, count, s["scale"])
        else:
            xq.xq_attn_decode(out, q, kv, table, lens, s["scale"], max_len=96, workspace=ws)
        s.update(q=q, io="bf16" if t == torch.bfloat16 else "f32")
        check_rows(s, out, slice(0, count), 0, j, n, 0, 0, 2.0 ** -8 if count > 1 else 2.0 ** -16 if io == "bf16" else 2.0 ** -24,
                   "%d tokens of %d" % (count, n))
        # what the codes hold: a block's largest is 3.5 of its powers at least, and a value is off by 1 at most (half of
        # the widest gap, or 7 that saturates)
        back = torch.empty(2, count, kv_heads, dim, device=DEV)
        xq.xq_cache_read(back[0], back[1], kv, slots)
        top = x[:, heads + kv_heads:].abs().unflatten(-1, (-1, 32)).amax(-1, keepdim=True).expand(-1, -1, -1, 32).flatten(-2)
        assert ((back[1] - x[:, heads + kv_heads:]).abs() <= top * (2 / 7 + 1e-6)).all()


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
def test_attention_layer(window, sinks):
    """The example's layer with its cache in 4 bits: its rows are attention over what the cache holds, through a prompt,
    single tokens, a fork and a compaction."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_layer.py")
    spec = importlib.util.spec_from_file_location("attention_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    layer = example.Layer(window=window, sinks=sinks, four_bits=True)
    g = torch.Generator(device=DEV).manual_seed(3)
    draw = lambda n: torch.randn(n, layer.hidden, device=DEV, generator=g)

    def holds(out, q, rows, io):
        raw = {n: getattr(layer.kv, n).view(torch.uint8) for n in ("k", "v", "k_exp", "v_exp")}
        s = dict(raw, table=layer.tables, page=layer.page, scale=layer.scale, scales=(1.0, 1.0), q=q)
        for t, (slot, pos) in enumerate(rows):
            n = layer.lens.tolist()[slot]
            want, mag, slack = four.attend(s, slice(t, t + 1), slot, torch.tensor([pos], device=DEV), n, window, sinks)
            tol = ref.attend_tolerance(want, mag, slack, io, 2.0 ** -8 if io == "bf16" else 2.0 ** -24, n)
            # A weight is f32, of the largest's 1: below 2^-126 it may count as 0, which takes up to 2^-126 |v| a token from
            # a sum that is divided by 1 or more. (Scores reach 100 here and many v are 0, so such weights stand alone.)
            v, _ = four.rows_of(s["v"], s["v_exp"], s["table"][slot], n, s["page"])
            tol = tol + 2.0 ** -126 * n * v.abs().max()
            assert ((out[t:t + 1].double() - want).abs() <= tol).all(), (slot, pos)

    last = lambda slots: [(s, layer.lens[s].item() - 1) for s in slots]
    y, out, q = layer.prompt(draw(103), [(0, 70), (1, 33)])
    holds(out, q, [(0, p) for p in range(70)] + [(1, p) for p in range(33)], "bf16")
    y, out, q = layer.step(draw(2), [0, 1])
    holds(out, q, last([0, 1]), "f32")
    layer.fork([0, 0], [2, 3])
    y, out, q = layer.step(draw(4), [0, 1, 2, 3])
    holds(out, q, last(range(4)), "f32")
    layer.fork([3], [1])
    layer.compact()
    y, out, q = layer.step(draw(4), [0, 1, 2, 3])
    holds(out, q, last(range(4)), "f32")
    assert y.isfinite().all()
