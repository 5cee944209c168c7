"""The mixture-of-experts layer against its definition in 64 bits, element by element.

The router: a logit is off by at most its sum's roundings, (K + 8) half steps of f32 of the terms' magnitudes (a chain in
any order); ids are the oracle's wherever the keys lie further apart than that.

The layer: x^ is exact (its two roundings are done the same way here, on the host). h is off by the sums' roundings and
those of silu; where that can move an element's quotient h / d over a border between two codes, the code may be either:
one step d there, times |down|. Beside that the scale's own error and f32's sums."""
import pytest
import torch

import four_reference as four
import kv_reference as ref
import quantized_decode_mat_amd as xq
from test_gpu_kv_four import _device  # noqa: F401
from test_gpu_kv_rope_pages import freqs

pytestmark = pytest.mark.gpu
DEV = "cuda"
F = 2.0 ** -24


def slab(rows, columns, g):
    n = rows * columns // 256
    raw = torch.randint(0, 256, (n, 144), device=DEV, generator=g, dtype=torch.int32).to(torch.uint8)
    d = (torch.rand(n, device=DEV, generator=g) + 0.5) * 1.2e-4
    raw[:, 0:2] = d.half().view(torch.uint8).view(n, 2)
    raw[:, 2:4] = (7.5 * d).half().view(torch.uint8).view(n, 2)
    return raw.view(-1)


def weights64(raw, rows, columns):
    """Q4_K rows in 64 bits: values, and the magnitudes of the two terms that each is the difference of."""
    b = raw.view(rows, columns // 256, 144)
    half = lambda i: b[..., i:i + 2].contiguous().view(torch.float16).double()
    i = b.int()
    w, mag = [], []
    for j in range(8):
        if j < 4:
            sc, m = i[..., 4 + j] & 63, i[..., 8 + j] & 63
        else:
            sc = (i[..., 8 + j] & 15) | (i[..., j] >> 6 << 4)
            m = (i[..., 8 + j] >> 4) | (i[..., 4 + j] >> 6 << 4)
        q = i[..., 16 + 32 * (j // 2):48 + 32 * (j // 2)]
        q = (q >> 4 if j % 2 else q & 15).double()
        a, c = half(0) * sc[..., None] * q, half(2) * m[..., None]
        w.append(a - c)
        mag.append(a + c)
    return torch.cat(w, -1).flatten(1), torch.cat(mag, -1).flatten(1)


def q8k(x):
    """x [rows, columns] f32 on the host: codes and scales."""
    b = x.float().cpu().unflatten(-1, (-1, 256))
    d = b.abs().amax(-1, keepdim=True) * torch.tensor(1.0 / 127.0, dtype=torch.float32)
    codes = torch.where(d > 0, torch.round(b / torch.where(d > 0, d, torch.ones_like(d))), torch.zeros_like(b))
    return codes.double().to(DEV), d.double().to(DEV)


def layer64(c, s):
    """y and its tolerance."""
    T, U, E, K, N = c["tokens"], c["used"], c["experts"], c["hidden"], c["ffn"]
    codes, d = q8k(s["x"])
    x = (codes * d).flatten(1)
    y, tol = (torch.zeros(T, K, dtype=torch.float64, device=DEV) for _ in range(2))
    ids, w = s["ids"].cpu().tolist(), s["weights"].double()
    part = lambda name, e, rows, columns: weights64(s[name].view(E, -1)[e], rows, columns)
    for e in range(E):
        at = [(t, k) for t in range(T) for k in range(U) if ids[t][k] == e]
        if not at:
            continue
        (gw, gm), (uw, um), (dw, dm) = part("gate", e, N, K), part("up", e, N, K), part("down", e, K, N)
        for t, k in at:
            g, u = gw @ x[t], uw @ x[t]
            steps = (K // 256 + 32) * F
            g_off, u_off = gm @ x[t].abs() * steps, um @ x[t].abs() * steps
            sig = 1 / (1 + torch.exp(-g))
            h = g * sig * u
            off = 1.1 * g_off * (u.abs() + u_off) + (g * sig).abs() * u_off + 12 * F * h.abs() + 1e-37
            hb, ob = h.view(-1, 256), off.view(-1, 256)
            top = hb.abs().amax(1, keepdim=True)
            scale = top / 127
            ratio = (ob.amax(1, keepdim=True) / top.clamp(min=1e-300)) + 3 * F   # of the scale's error
            z = torch.where(scale > 0, hb / scale.clamp(min=1e-300), torch.zeros_like(hb))
            code = torch.round(z)
            slack = ob / scale.clamp(min=1e-300) + z.abs() * (ratio + 2 * F)
            either = ((z - code).abs() + slack >= 0.5).double()
            hq = (code * scale).flatten()
            err = (either * scale + code.abs() * scale * ratio).flatten()
            wk = float(w[t, k])
            y[t] += wk * (dw @ hq)
            tol[t] += abs(wk) * (dw.abs() @ err + dm @ (hq.abs() + err) * ((N // 256 + U + 32) * F))
    kind = c["io"]
    return y, 1.01 * tol + ref.half_step(kind) * y.abs() + ref.smallest(kind)


def state(c, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    T, U, E, K, N = c["tokens"], c["used"], c["experts"], c["hidden"], c["ffn"]
    s = dict(gate=slab(E * N, K, g), up=slab(E * N, K, g), down=slab(E * K, N, g))
    wide = torch.randn(T, K + 16, device=DEV, generator=g).to(ref.TYPES[c["io"]])
    s["x"] = wide[:, :K]
    s["full"] = torch.full((T, K + 3), 7.0, dtype=ref.TYPES[c["io"]], device=DEV)
    s["y"] = s["full"][:, :K]
    s["ids"] = torch.stack([torch.randperm(E, device=DEV, generator=g)[:U] for _ in range(T)]).int()
    s["weights"] = torch.rand(T, U, device=DEV, generator=g) + 0.1
    s["ws"] = torch.zeros(xq.xq_moe_q4k_workspace_bytes(T, U, K, N), dtype=torch.uint8, device=DEV)
    return s


def run(c, s, **kw):
    xq.xq_moe_q4k(s["y"], s["x"], s["gate"], s["up"], s["down"], s["ids"], s["weights"], c["experts"], c["ffn"],
                  workspace=s["ws"], **kw)


def check(c, s, what=""):
    torch.cuda.synchronize()
    assert (s["full"][:, c["hidden"]:] == 7.0).all(), "%s: wrote past the rows" % what
    want, tol = layer64(c, s)
    err = (s["y"].double() - want).abs()
    assert (err <= tol).all(), "%s: worst %.3g of the tolerance" % (what, float((err / tol).nan_to_num(9e9).max()))


LAYERS = [
    # tokens, used, experts, hidden, ffn, io
    (1, 8, 64, 2048, 1536, "bf16"),
    (1, 1, 1, 256, 256, "f32"),
    (1, 4, 9, 1280, 768, "f16"),
    (1, 2, 8, 4096, 2560, "f32"),
    (1, 3, 4, 4352, 256, "bf16"),       # rows of 17 blocks: two units
    (1, 8, 16, 256, 11264, "bf16"),     # h past 80 KiB of LDS: by tiles
    (2, 3, 60, 768, 512, "f32"),
    (5, 6, 64, 2048, 1280, "f16"),
    (7, 1, 8, 8448, 512, "bf16"),       # three units
    (3, 2, 8, 1024, 1792, "f32"),
    (9, 4, 8, 512, 768, "bf16"),
    (16, 2, 8, 1024, 1280, "f32"),
    (40, 2, 2, 512, 256, "f16"),
    (33, 3, 5, 256, 2304, "bf16"),
    (512, 1, 3, 256, 256, "f32"),
    (16, 8, 128, 768, 256, "bf16"),
    (64, 8, 128, 256, 512, "f16"),
    (1, 1, 2, 32768, 256, "bf16"),      # the widest, every way
    (2, 2, 5, 32768, 256, "f32"),
    (1, 2, 2, 256, 32768, "f16"),
    (3, 1, 2, 256, 32768, "f32"),
    (5, 1, 2, 32768, 512, "bf16"),
    (1, 512, 1024, 256, 256, "f32"),    # all 512 slots a token's
    (16, 2, 8, 2304, 2048, "f32"),      # many pairs of larger experts: tiles
    (40, 2, 2, 2048, 2304, "f16"),      # 40 pairs an expert: three passes
    (33, 3, 5, 1024, 2304, "bf16"),
    (9, 4, 8, 2048, 2816, "bf16"),
    (512, 1, 3, 2048, 1024, "f32"),
    (64, 8, 64, 1024, 1024, "f16"),
    (512, 1, 1, 768, 512, "bf16"),
    (17, 1, 2, 32768, 256, "f32"),
]


@pytest.mark.parametrize("case", LAYERS, ids=lambda c: "-".join(str(x) for x in c))
def test_layer(case):
    c = dict(zip(("tokens", "used", "experts", "hidden", "ffn", "io"), case))
    s = state(c)
    run(c, s)
    check(c, s, "layer")
    first = s["y"].clone()
    s["ws"].fill_(0xff)                                      # nothing is kept from one call for the next
    s["ws"][:96 * 1024] = 0
    s["full"][:, :c["hidden"]] = 5.0
    run(c, s)
    assert torch.equal(s["y"], first), "the same call gave other bits"
    assert not s["ws"][:96 * 1024].any(), "wrote where other calls keep counters"


@pytest.mark.parametrize("tokens,experts,width", [(1, 16, 512), (3, 16, 512), (12, 6, 512), (100, 6, 1024)])  # the last by tiles
def test_slots_left_out_and_experts_named_twice(tokens, experts, width):
    c = dict(tokens=tokens, used=4, experts=experts, hidden=width, ffn=width, io="f32")
    s = state(c, 2)
    s["ids"][0] = torch.tensor([-1, 3, 3, experts], dtype=torch.int32)
    if tokens > 1:
        s["ids"][1] = torch.tensor([2 ** 31 - 1, -2 ** 31, -1, experts], dtype=torch.int32)
        s["weights"][1] = float("nan")                       # nothing of them is read
        s["ids"][2] = 5
    run(c, s)
    if tokens > 1:
        torch.cuda.synchronize()
        assert (s["y"][1] == 0).all()
        s["weights"][1] = 0
    check(c, s)


@pytest.mark.parametrize("tokens,experts", [(1, 2), (6, 12), (96, 4)])  # the last by tiles
def test_rows_of_zeros_and_large_weights(tokens, experts):
    """x of zeros gives zeros; q8_K blocks of zeros beside others; weights at the header's ends."""
    c = dict(tokens=tokens, used=2, experts=experts, hidden=1024, ffn=768, io="f32")
    s = state(c, 3)
    s["x"][0] = 0
    if tokens > 1:
        s["x"][1, 256:512] = 0
        s["x"][2] *= 1e4
        s["x"][3] *= 1e-6
    for name in ("gate", "up", "down"):
        raw = s[name].view(-1, 144)
        raw[::3, 4:] = 255                                   # the largest codes, scales and mins
        raw[1::3, 4:] = 0
    run(c, s)
    torch.cuda.synchronize()
    assert (s["y"][0] == 0).all()
    check(c, s)


def test_layer_in_a_graph_on_another_stream():
    # (the fourth with more LDS than a launch has by itself, the last by tiles)
    for tokens, hidden, ffn in ((1, 512, 768), (4, 512, 768), (20, 512, 768), (2, 256, 20480), (40, 1024, 2048)):
        c = dict(tokens=tokens, used=3, experts=12, hidden=hidden, ffn=ffn, io="bf16")
        s = state(c, 4)
        run(c, s)
        torch.cuda.synchronize()
        want = s["y"].clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            run(c, s)
        for _ in range(3):
            s["full"][:, :hidden] = 5.0
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(s["y"], want)
            run(c, s)
            torch.cuda.synchronize()
            assert torch.equal(s["y"], want)


@pytest.mark.parametrize("tokens,hidden,ffn", [(1, 512, 768), (5, 512, 768), (60, 1024, 2048)])  # the last by tiles
def test_layer_in_place(tokens, hidden, ffn):
    c = dict(tokens=tokens, used=3, experts=6, hidden=hidden, ffn=ffn, io="bf16")
    s = state(c, 11)
    run(c, s)
    torch.cuda.synchronize()
    want = s["y"].clone()
    s["y"] = s["x"]
    run(c, s)
    torch.cuda.synchronize()
    assert torch.equal(s["x"], want)


def test_two_layers_at_once():
    """Two streams, each with its own workspace, and x of one in both."""
    g = torch.Generator(device=DEV).manual_seed(6)
    runs = []
    for tokens, experts in ((1, 8), (3, 40), (48, 8)):  # the last by tiles
        c = dict(tokens=tokens, used=4, experts=experts, hidden=1024, ffn=768, io="bf16")
        a = state(c, 7)
        b = dict(a, ids=torch.randint(0, experts, (tokens, 4), device=DEV, generator=g, dtype=torch.int32),
                 full=a["full"].clone(), ws=torch.zeros_like(a["ws"]))
        b["y"] = b["full"][:, :1024]
        runs.append((c, a, b))
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(8):
        for c, a, b in runs:
            run(c, a, stream=one)
            run(c, b, stream=two)
    for c, a, b in runs:
        check(c, a)
        check(c, b)


# ---------------------------------------------------------------- router

ROUTES = [
    # tokens, experts, used, K, x type, router type, score, bias, normalize
    (1, 64, 8, 2048, "bf16", "bf16", "softmax", False, True),
    (1, 1, 1, 8, "f32", "f32", "sigmoid", False, True),
    (3, 5, 5, 264, "f16", "f32", "softmax", True, False),
    (5, 65, 6, 512, "f32", "bf16", "sigmoid", True, True),
    (17, 128, 8, 4096, "bf16", "f16", "softmax", False, False),
    (64, 200, 64, 1000, "f16", "f16", "sigmoid", False, True),
    (9, 1024, 32, 520, "bf16", "bf16", "softmax", True, True),
    (512, 8, 2, 256, "f32", "f32", "softmax", False, True),
    (512, 1024, 64, 8, "f32", "bf16", "sigmoid", True, True),
    (2, 6, 2, 1048576, "f32", "f32", "softmax", False, True),
]


def route_state(case, seed=1):
    T, E, U, K, xt, rt, score, bias, normalize = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(x=torch.randn(T, K + 16, device=DEV, generator=g).to(ref.TYPES[xt])[:, :K],
             router=(2 * torch.randn(E, K, device=DEV, generator=g) * K ** -0.5).to(ref.TYPES[rt]),
             bias=torch.randn(E, device=DEV, generator=g) * 0.2 if bias else None)
    s["ids"] = torch.full((T + 1, U), 77, dtype=torch.int32, device=DEV)
    s["weights"] = torch.full((T + 1, U), 7.0, device=DEV)
    s["ws"] = torch.zeros(xq.xq_moe_route_workspace_bytes(T, E), dtype=torch.uint8, device=DEV)
    return s


def route(case, s, scale=1.5, **kw):
    T = case[0]
    xq.xq_moe_route(s["ids"][:T], s["weights"][:T], s["x"], s["router"], bias=s["bias"], score=case[6],
                    normalize=case[8], scale=scale, workspace=s["ws"], **kw)


def check_route(case, s, scale=1.5):
    T, E, U, K, xt, rt, score, bias, normalize = case
    torch.cuda.synchronize()
    assert (s["ids"][T:] == 77).all() and (s["weights"][T:] == 7.0).all()
    x, r = s["x"].double(), s["router"].double()
    logits = torch.mm(x, r.t().contiguous())
    off = torch.mm(x.abs(), r.abs().t().contiguous()) * ((K + 8) * F)
    # a score's relative error: exp of its logit's, the sum's alike, and 8 roundings
    p = torch.softmax(logits, -1) if score == "softmax" else torch.sigmoid(logits)
    rel = off + off.amax(-1, keepdim=True) + 8 * F if score == "softmax" else off + 8 * F
    key = p + (s["bias"].double() if bias else 0) if score == "sigmoid" or bias else logits
    slack = p * rel + F * key.abs() if score == "sigmoid" or bias else off
    ids, got = s["ids"][:T].long(), s["weights"][:T].double()
    assert (ids >= 0).all() and (ids < E).all()
    assert all(len(set(row)) == U for row in ids.tolist())
    # in order, and nothing that is left out is above what is chosen, but for the slack
    k, sl = key.gather(1, ids), slack.gather(1, ids)
    assert (k[:, :-1] + sl[:, :-1] >= k[:, 1:] - sl[:, 1:]).all()
    rest = (key - slack).scatter(1, ids, -float("inf"))
    assert (rest.amax(-1) <= (k + sl).amin(-1)).all()
    best = key.sort(dim=-1, descending=True, stable=True)[1][:, :U]
    assert (best == ids).float().mean() > 0.99
    want = p.gather(1, ids)
    total = want.sum(-1, keepdim=True) if normalize else 1.0
    want = want / total * scale
    bound = want * (rel.gather(1, ids) + (rel.gather(1, ids).amax(-1, keepdim=True) if normalize else 0) + (U + 4) * F)
    assert ((got - want).abs() <= bound + 1e-40).all()


@pytest.mark.parametrize("case", ROUTES, ids=lambda c: "-".join(str(x) for x in c))
def test_route(case):
    s = route_state(case)
    route(case, s)
    check_route(case, s)
    assert not s["ws"][:96 * 1024].any(), "arrival counters left standing"
    first = s["ids"].clone(), s["weights"].clone()
    s["ids"].fill_(77)
    route(case, s)
    assert torch.equal(s["ids"], first[0]) and torch.equal(s["weights"], first[1])


@pytest.mark.parametrize("experts,used", [(8, 3), (70, 40), (1000, 64)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_of_equal_scores(experts, used, score):
    """Equal keys go by their index: all experts alike, then two kinds of them."""
    case = (2, experts, used, 256, "f32", "f32", score, False, True)
    s = route_state(case)
    s["router"][:] = s["router"][:1].clone()
    route(case, s)
    torch.cuda.synchronize()
    assert (s["ids"][:2] == torch.arange(used, device=DEV)).all()
    assert ((s["weights"][:2] * used / 1.5 - 1).abs() <= (experts + 40) * F).all()
    s["x"][:] = s["x"].abs()
    s["router"][:] = -1.0
    s["router"][1::3] = 1.0
    route(case, s)
    torch.cuda.synchronize()
    high = list(range(1, experts, 3))
    assert s["ids"][0].tolist() == (high + [e for e in range(experts) if e % 3 != 1])[:used]


def test_route_zeros_and_what_is_not_finite():
    """Minus zero is zero; NaN ranks below everything, minus infinity among it; far logits."""
    case = (4, 8, 8, 256, "f32", "f32", "sigmoid", False, False)
    s = route_state(case)
    s["x"][:], s["router"][:] = 0, 0
    s["x"][:, 0] = 1
    s["router"][:, 0] = torch.tensor([-0.0, 0.0, float("nan"), 500.0, -500.0, float("-inf"), float("inf"), -0.0])
    route(case, s, scale=1.0)
    torch.cuda.synchronize()
    assert s["ids"][0].tolist() == [3, 6, 0, 1, 7, 4, 5, 2]
    assert s["weights"][0, :7].tolist() == [1, 1, 0.5, 0.5, 0.5, 0, 0] and s["weights"][0, 7].isnan()
    # softmax of such a row is NaN, in the logits' order
    case = case[:6] + ("softmax", False, True)
    route(case, s, scale=1.0)
    torch.cuda.synchronize()
    assert s["ids"][0].tolist() == [6, 3, 0, 1, 7, 4, 5, 2]
    # a chosen sum of zero gives zeros
    s["router"][:, 0] = -500.0
    case = case[:6] + ("sigmoid", False, True)
    route(case, s)
    torch.cuda.synchronize()
    assert (s["weights"][:4] == 0).all()


# ---------------------------------------------------------------- together

def test_decode_step_in_a_graph():
    """One step of a layer in 4 bits, as a server captures it: positions and append to the cache, attention, router,
    experts; replayed with new inputs, on one workspace, against the same calls made one by one and the definitions."""
    T, heads, kv_heads, dim, page, E, U, N = 3, 8, 2, 128, 16, 16, 4, 768
    hidden = heads * dim
    g = torch.Generator(device=DEV).manual_seed(9)
    k, k_exp = four.pool(20, kv_heads, page, dim, "hnd", g, DEV)
    v, v_exp = four.pool(20, kv_heads, page, dim, "hnd", g, DEV)
    scales = (0.75, 1.25)
    kv = four.cache(xq, k, k_exp, v, v_exp, scales)
    table = torch.randperm(20, device=DEV, generator=g)[:18].view(T, 6).int()
    lens = torch.tensor([70, 1, 33], dtype=torch.int32, device=DEV)
    plan = xq.xq_rope_plan(freqs(dim), [dim // 2])
    c = dict(tokens=T, used=U, experts=E, hidden=hidden, ffn=N, io="bf16")
    s = state(c, 10)
    router = torch.randn(E, hidden, device=DEV, generator=g).to(torch.bfloat16)
    qkv = torch.empty(T, heads + 2 * kv_heads, dim, dtype=torch.bfloat16, device=DEV)
    q, out = (torch.empty(T, heads, dim, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    y = torch.empty(T, hidden, dtype=torch.bfloat16, device=DEV)
    need = max(xq.xq_attn_decode_workspace_bytes(T, heads, kv, 96), xq.xq_moe_route_workspace_bytes(T, E),
               xq.xq_moe_q4k_workspace_bytes(T, U, hidden, N))
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    pos, slots = torch.empty(T, dtype=torch.int32, device=DEV), torch.empty(T, dtype=torch.int64, device=DEV)

    def step():
        xq.xq_rope_append(q, kv, qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:], pos, plan, slots)
        xq.xq_attn_decode(out, q, kv, table, lens, dim ** -0.5, max_len=96, workspace=ws)
        xq.xq_moe_route(s["ids"], s["weights"], out.view(T, hidden), router, workspace=ws)
        xq.xq_moe_q4k(y, out.view(T, hidden), s["gate"], s["up"], s["down"], s["ids"], s["weights"], E, N, workspace=ws)

    def fresh(seed):
        qkv.copy_(torch.randn(qkv.shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed)))
        j = lens.long() - 1
        pos.copy_(j)
        slots.copy_(table.long()[torch.arange(T, device=DEV), j // page] * page + j % page)

    fresh(1)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (2, 3, 4):
        lens += 1
        fresh(seed)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, s["ids"], s["weights"], y)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, s["ids"], s["weights"], y)))
        a = dict(k=k, v=v, k_exp=k_exp, v_exp=v_exp, table=table, page=page, scale=dim ** -0.5, scales=scales, q=q)
        for b, n in enumerate(lens.tolist()):
            want, mag, slack = four.attend(a, slice(b, b + 1), b, torch.tensor([n - 1], device=DEV), n, 0, 0)
            assert ((out[b:b + 1].double() - want).abs() <= ref.attend_tolerance(want, mag, slack, "bf16", 2.0 ** -16, n)).all()
        assert (s["weights"].sum(-1) - 1).abs().max() < 1e-5
        want, tol = layer64(c, dict(s, x=out.view(T, hidden)))
        assert ((y.double() - want).abs() <= tol).all()
