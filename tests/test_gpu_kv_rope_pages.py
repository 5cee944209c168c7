"""Rotary positions against the formula in 64 bits (and the gradient against
differences), the append, and the pages' management against a host model."""
import random

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


def freqs(rot, base=500000.0):
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    return base ** (-2.0 * i / rot)


def positions(axes, tokens, far, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    pos = torch.randint(0, 1000, (axes, tokens), device=DEV, generator=g, dtype=torch.int32)
    pos[0] = far + torch.arange(tokens, device=DEV, dtype=torch.int32)
    return pos


ROPE = [
    # tokens, heads, dim, rot, sections, adjacent, x type, out type, first position
    (1, 1, 8, 8, [4], False, "f32", "f32", 0),
    (7, 32, 128, 128, [64], False, "f32", "f32", 199000),
    (33, 5, 96, 64, [12, 10, 10], True, "bf16", "bf16", 1000000),
    (5, 3, 80, 40, [0, 20], False, "f16", "f32", 77),
    (1030, 8, 64, 64, [8, 8, 8, 8], True, "bf16", "f16", 5),
    (2, 2, 256, 256, [100, 20, 8], False, "f32", "bf16", -3),
    (3, 300, 1024, 1024, [512], False, "bf16", "bf16", 2000000000),
]


def rope_case(tokens, heads, dim, rot, sections, adjacent, xt, ot, far, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    wide = torch.randn(tokens, heads + 2, dim + 8, device=DEV, generator=g).to(ref.TYPES[xt])
    return (wide[:, 1:heads + 1, 8:], positions(len(sections), tokens, far, seed),
            xq.xq_rope_plan(freqs(rot), sections, adjacent))


def check_rope(got, x, pos, plan, sections, adjacent, inverse, ot, scale=1.0):
    x = x.double()
    want = ref.rotate(x, pos, plan.freq, sections, adjacent, inverse)
    angle = float(pos.double().abs().max() * plan.freq.max())
    tol = ref.rotate_tolerance(x, want, "f32", plan.freq.numel(), adjacent, angle)
    tol = tol / scale + ref.half_step(ot) * (want / scale).abs() * 1.01 + ref.smallest(ot) + 2.0 ** -23 * (want / scale).abs()
    err = (ref.as_f64(got) - want / scale).abs()
    assert (err <= tol).all(), "worst %.3g of the tolerance" % float((err / tol).nan_to_num(9e9).max())


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", ROPE, ids=lambda c: "-".join(str(x) for x in c))
def test_rope(case, inverse):
    tokens, heads, dim, rot, sections, adjacent, xt, ot, far = case
    x, pos, plan = rope_case(*case)
    out = torch.full((tokens, heads + 1, dim), 7.0, dtype=ref.TYPES[ot], device=DEV)
    xq.xq_rope(out[:, :heads], x, pos if plan.axes > 1 else pos[0], plan, inverse=inverse)
    torch.cuda.synchronize()
    assert (out[:, heads:] == 7.0).all()
    check_rope(out[:, :heads], x, pos, plan, sections, adjacent, inverse, ot)


def test_rope_unaligned_rows():
    """Rows that begin at any element."""
    x, pos, plan = rope_case(9, 3, 64, 32, [16], False, "bf16", "f32", 11)
    flat = torch.zeros(9 * 3 * 67 + 1, dtype=torch.bfloat16, device=DEV)
    odd = flat[1:].as_strided((9, 3, 64), (3 * 67, 67, 1))
    odd.copy_(x)
    res = torch.zeros(9 * 3 * 65 + 3, dtype=torch.float32, device=DEV)
    out = res[3:].as_strided((9, 3, 64), (3 * 65, 65, 1))
    xq.xq_rope(out, odd, pos, plan)
    torch.cuda.synchronize()
    check_rope(out, odd, pos, plan, [16], False, False, "f32")


def test_rope_in_place_and_back():
    x, pos, plan = rope_case(65, 4, 128, 96, [20, 14, 14], True, "f32", "f32", 5000)
    y = x.contiguous()
    xq.xq_rope(y, y, pos, plan)
    check_rope(y, x, pos, plan, [20, 14, 14], True, False, "f32")
    xq.xq_rope(y, y, pos, plan, inverse=True)
    torch.cuda.synchronize()
    # two rotations, 8 half steps of a pair's magnitude each, at most 5.5
    assert (y - x).abs().max() <= 2 * 8 * 2.0 ** -24 * 2 * float(x.abs().max())


@pytest.mark.parametrize("adjacent", [False, True])
def test_rope_gradient_against_differences(adjacent):
    """g . (f(x + h d) - f(x - h d)) / 2h = d . f_inverse(g), f being linear."""
    args = (17, 4, 64, 48, [8, 8, 8], adjacent, "f32", "f32", 300)
    x, pos, plan = rope_case(*args)
    g, d = rope_case(*args, seed=2)[0], rope_case(*args, seed=3)[0]
    up, down, back = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    h = 0.5
    xq.xq_rope(up, (x + h * d), pos, plan)
    xq.xq_rope(down, (x - h * d), pos, plan)
    xq.xq_rope(back, g, pos, plan, inverse=True)
    left = float((g.double() * (up.double() - down.double())).sum() / (2 * h))
    right = float((d.double() * back.double()).sum())
    # each of the 4352 terms off by at most 8 half steps of 2 * 6 * 6 (|x|, |g|, |d| below 6)
    assert abs(left - right) <= x.numel() * 2 * 8 * 2.0 ** -24 * 72


APPEND = [
    # tokens, heads, kv_heads, dim, rot, sections, adjacent, page, src, io, cache, order
    (1, 4, 1, 64, 64, [32], False, 16, "f32", "f32", "bf16", "hnd"),
    (40, 6, 2, 128, 128, [24, 20, 20], False, 24, "f32", "bf16", "bf16", "nhd"),
    (33, 5, 1, 80, 40, [20], True, 1, "bf16", "f16", "f16", "hnd"),
    (300, 8, 8, 96, 48, [6, 6, 6, 6], True, 64, "f16", "f32", "e4m3", "nhd"),
    (9, 3, 3, 256, 128, [60, 4], False, 8, "bf16", "bf16", "e4m3", "hnd"),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(str(x) for x in c))
def test_append(case):
    tokens, heads, kv_heads, dim, rot, sections, adjacent, page, src, io, cache, order = case
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(tokens, heads + 2 * kv_heads, dim, device=DEV, generator=g).to(ref.TYPES[src])
    pages = -(-tokens // page) + 3
    k, v = (ref.pool(pages, kv_heads, page, dim, cache, order, g, DEV) for _ in range(2))
    k0, v0 = ref.as_f64(k).clone(), ref.as_f64(v).clone()
    scales = (0.05, 0.04) if cache == "e4m3" else (1.0, 2.0)
    kv = xq.xq_kv_cache(k, v, *scales)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(1))[:tokens].to(DEV)
    if tokens > 8:  # tokens without a place, and places that do not exist
        slots[3], slots[5], slots[7] = -1, pages * page, 1 << 40
    pos, plan = positions(len(sections), tokens, 4000, 1), xq.xq_rope_plan(freqs(rot), sections, adjacent)
    q, ks, vs = x[:, :heads], x[:, heads:heads + kv_heads], x[:, heads + kv_heads:]
    out = torch.empty(tokens, heads, dim, dtype=ref.TYPES[io], device=DEV)
    xq.xq_rope_append(out, kv, q, ks, vs, pos, plan, slots)
    torch.cuda.synchronize()
    check_rope(out, q, pos, plan, sections, adjacent, False, io)
    keep = (slots >= 0) & (slots < pages * page)
    at, place = slots[keep] // page, slots[keep] % page
    got_k, got_v = ref.as_f64(k), ref.as_f64(v)
    check_rope(got_k[at, :, place], ks[keep], pos[:, keep], plan, sections, adjacent, False, cache, scales[0])
    want = vs[keep].double() / scales[1]
    if cache == "e4m3":
        want = want.clamp(-448, 448)
    assert ((got_v[at, :, place] - want).abs() <= ref.half_step(cache) * want.abs() * 1.01 + ref.smallest(cache) + 2.0 ** -23 * want.abs()).all()
    k0[at, :, place], v0[at, :, place] = got_k[at, :, place], got_v[at, :, place]
    assert torch.equal(k0, got_k) and torch.equal(v0, got_v), "other slots changed"


def test_append_8_bit_extremes():
    """Values past the type's largest are clamped, NaN stays."""
    k = torch.zeros(1, 1, 16, 16, device=DEV).to(torch.float8_e4m3fn)
    v = torch.zeros(1, 1, 16, 16, device=DEV).to(torch.float8_e4m3fn)
    x = torch.zeros(2, 3, 16, device=DEV)
    x[0, 2, :6] = torch.tensor([1e9, -1e9, 448.0, -449.0, float("inf"), float("nan")], device=DEV)
    x[1, 2, :3] = torch.tensor([-0.0, 2.0 ** -9, 2.0 ** -11], device=DEV)
    plan = xq.xq_rope_plan(freqs(16), [8])
    pos = torch.zeros(2, dtype=torch.int32, device=DEV)
    out = torch.empty(2, 1, 16, device=DEV)
    xq.xq_rope_append(out, xq.xq_kv_cache(k, v), x[:, :1], x[:, 1:2], x[:, 2:], pos, plan,
                      torch.tensor([3, 4], device=DEV))
    torch.cuda.synchronize()
    got = v.float()[0, 0]
    assert got[3, :5].tolist() == [448.0, -448.0, 448.0, -448.0, 448.0] and got[3, 5].isnan()
    assert got[4, :3].tolist() == [0.0, 2.0 ** -9, 0.0]


# ---- pages

def cache(layers, pages, kv_heads, page, dim, kind, order, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    k, v = (ref.pool(pages, kv_heads, page, dim, kind, order, g, DEV, layers) for _ in range(2))
    return xq.xq_kv_cache(k, v), k, v


def raw(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


POOLS = [(1, 40, 2, 16, 64, "bf16", "hnd"), (3, 40, 1, 8, 16, "e4m3", "nhd"), (2, 300, 3, 1, 80, "f16", "nhd"),
         (2, 64, 8, 24, 128, "bf16", "hnd")]


@pytest.mark.parametrize("case", POOLS, ids=lambda c: "-".join(str(x) for x in c))
def test_copy(case):
    kv, k, v = cache(*case)
    pages = case[1]
    ids = random.Random(1).sample(range(pages), 30)
    src, dst = ids[:15] + [-1, 0, pages, ids[3]], ids[15:] + [0, -2, 1, ids[3]]
    want = [raw(x).clone() for x in (k, v)]
    for w in want:
        w[:, ids[15:]] = w[:, ids[:15]]
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    xq.xq_cache_copy(kv, t(src), t(dst))
    torch.cuda.synchronize()
    assert torch.equal(raw(k), want[0]) and torch.equal(raw(v), want[1])
    xq.xq_cache_copy(kv, t([]), t([]))


def test_copy_strided_pool():
    """A cache that is a slice of a larger pool's heads."""
    g = torch.Generator(device=DEV).manual_seed(1)
    big = torch.randn(2, 12, 5, 16, 64, device=DEV, generator=g).to(torch.bfloat16)
    k, v = big[:, :, 1:3], big[:, :, 3:5]
    want = big.clone()
    want[:, 7, 1:] = want[:, 2, 1:]
    xq.xq_cache_copy(xq.xq_kv_cache(k, v), torch.tensor([2], dtype=torch.int32, device=DEV),
                     torch.tensor([7], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert torch.equal(big, want)


def filled(rng, pages, page, slots, width, rows):
    """Tables whose first `rows` rows hold sequences."""
    ids = rng.sample(range(pages), pages)
    refs, tables, lens = [0] * pages, [[-1] * width for _ in range(slots)], [0] * slots
    for r in range(rows):
        n = rng.choice([0, 1, page, rng.randint(1, width * page), rng.randint(1, page * 3)])
        need = -(-n // page)
        if need > min(len(ids) // 2, width):
            n = need = 0
        lens[r] = n
        for i in range(need):
            tables[r][i] = ids.pop()
            refs[tables[r][i]] = 1
    return refs, tables, lens


class Device:
    def __init__(self, refs, tables, lens):
        t = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
        slots, width = len(lens), len(tables[0])
        self.wide = torch.full((slots, width + 3), -9, dtype=torch.int32, device=DEV)
        self.refs, self.tables, self.lens = t(refs), self.wide[:, :width], t(lens)
        self.tables.copy_(t(tables))
        self.status = t([5, 5])
        self.ws = torch.zeros(xq.xq_cache_workspace_bytes(len(refs), slots), dtype=torch.uint8, device=DEV)

    def check(self, model, kv_pairs):
        torch.cuda.synchronize()
        assert self.refs.tolist() == model.refs
        assert self.tables.tolist() == model.tables
        assert self.lens.tolist() == model.lens
        assert (self.wide[:, self.tables.shape[1]:] == -9).all()
        for x, w in kv_pairs:
            for a, b in model.copies:
                w[:, b] = w[:, a]
            assert torch.equal(raw(x), w)
        assert not self.ws[:96 * 1024].any()


@pytest.mark.parametrize("case", POOLS, ids=lambda c: "-".join(str(x) for x in c))
@pytest.mark.parametrize("seed", [1, 2])
def test_free_fork_compact(case, seed):
    rng = random.Random(seed)
    kv, k, v = cache(*case)
    layers, pages, _, page, _, _, _ = case
    slots, width = 24, 9
    refs, tables, lens = filled(rng, pages, page, slots, width, 12)
    d, m = Device(refs, tables, lens), ref.Pages(refs, tables, lens, page)
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    for _ in range(3):
        pairs = [(x, raw(x).clone()) for x in (k, v)]
        m.copies = []
        kids = rng.sample(range(12, slots), 9)
        parents = [rng.randrange(0, 12) for _ in kids]
        rows = kids + [kids[0], -1, slots]
        m.free(rows)
        xq.xq_cache_free(kv, d.refs, d.tables, d.lens, t(rows))
        # a child twice, rows out of range, a child that is not empty, a fork of an empty child
        parents += [0, -1, 3, 2, kids[0]]
        kids2 = kids + [kids[1], 13, slots, 1, next(r for r in range(12, slots) if r not in kids)]
        want = m.fork(parents, kids2)
        xq.xq_cache_fork(kv, d.refs, d.tables, d.lens, t(parents), t(kids2), d.status, workspace=d.ws)
        d.check(m, pairs)
        assert d.status.tolist() == want
    gone = rng.sample(range(slots), 8)
    m.free(gone)
    xq.xq_cache_free(kv, d.refs, d.tables, d.lens, t(gone))
    pairs = [(x, raw(x).clone()) for x in (k, v)]
    m.copies = []
    want = m.compact()
    xq.xq_cache_compact(kv, d.refs, d.tables, d.status, workspace=d.ws)
    d.check(m, pairs)
    assert d.status.tolist() == want
    # twice more: nothing is left to move
    m.copies = []
    xq.xq_cache_compact(kv, d.refs, d.tables, d.status, workspace=d.ws)
    d.check(m, [(x, raw(x).clone()) for x in (k, v)])


def test_fork_runs_out_of_pages():
    kv, k, v = cache(1, 8, 1, 16, 64, "bf16", "hnd")
    tables = [[0, 3, 4], [5, -1, -1]] + [[-1] * 3 for _ in range(6)]
    refs, lens = [1, 0, 1, 1, 1, 1, 0, 1], [40, 32, 0, 0, 0, 0, 0, 0]
    d, m = Device(refs, tables, lens), ref.Pages(refs, tables, lens, 16)
    pairs = [(x, raw(x).clone()) for x in (k, v)]
    parents, kids = [0, 1, 0, 0, 2], [4, 5, 6, 7, 3]  # row 1 is shorter than its length: refused
    want = m.fork(parents, kids)
    assert want == [2, 1]
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    xq.xq_cache_fork(kv, d.refs, d.tables, d.lens, t(parents), t(kids), d.status, workspace=d.ws)
    d.check(m, pairs)
    assert d.status.tolist() == want


def test_many_pages_and_rows():
    """More pages and rows than one workgroup has threads."""
    rng = random.Random(4)
    kv, k, v = cache(1, 5000, 1, 2, 16, "bf16", "hnd")
    refs, tables, lens = filled(rng, 5000, 2, 2600, 5, 1250)
    d, m = Device(refs, tables, lens), ref.Pages(refs, tables, lens, 2)
    pairs = [(x, raw(x).clone()) for x in (k, v)]
    kids = list(range(1250, 2500))
    parents = [rng.randrange(1250) for _ in kids]
    want = m.fork(parents, kids)
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    xq.xq_cache_fork(kv, d.refs, d.tables, d.lens, t(parents), t(kids), d.status, workspace=d.ws)
    d.check(m, pairs)
    assert d.status.tolist() == want
    gone = rng.sample(range(2500), 1500)
    m.free(gone)
    xq.xq_cache_free(kv, d.refs, d.tables, d.lens, t(gone))
    pairs, m.copies = [(x, raw(x).clone()) for x in (k, v)], []
    want = m.compact()
    xq.xq_cache_compact(kv, d.refs, d.tables, d.status, workspace=d.ws)
    d.check(m, pairs)
    assert d.status.tolist() == want


def test_pages_in_a_graph():
    """Free and fork captured, replayed: the same lowest pages each time."""
    kv, k, v = cache(2, 40, 2, 16, 64, "bf16", "hnd")
    rng = random.Random(7)
    refs, tables, lens = filled(rng, 40, 16, 12, 6, 6)
    d = Device(refs, tables, lens)
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    kids, parents = t([6, 7, 8, 9]), t([0, 1, 0, 2])

    def step():
        xq.xq_cache_free(kv, d.refs, d.tables, d.lens, kids)
        xq.xq_cache_fork(kv, d.refs, d.tables, d.lens, parents, kids, d.status, workspace=d.ws)

    step()
    torch.cuda.synchronize()
    want = [x.clone() for x in (d.refs, d.tables, d.lens, raw(k), raw(v))]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (d.refs, d.tables, d.lens, raw(k), raw(v))))
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (d.refs, d.tables, d.lens, raw(k), raw(v))))
