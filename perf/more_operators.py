"""The 4-bit half of a decode step: what is measured, and the operators' plain forms.

Four operators: attention of one new token per sequence over a paged cache held in 4 bits (``decode``), attention of a
chunk of tokens over it (``chunk``), rotary positions fused with the append to it, and the tokens read back
(``append``), and a mixture-of-experts layer on Q4_K weights for a few tokens, router included (``moe``).

The cache's values: blocks of 32 dims share a power of two (a byte, its exponent + 127), each dim is a sign and one of
0, 0.5, 1, 1.5, 2, 3, 4, 6 (two to a byte, the first in the low bits).
"""

import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one user's chat, some hundred tokens in: the call's latency
        dict(name="decode_one_short", op="decode", seqs=1, longest=700, heads=32, kv_heads=8, dim=128, page=16,
             io="f32", order="hnd", window=0, sinks=0),
        # a ragged serving batch on the 4096-wide layer's heads
        dict(name="decode_batch_ragged", op="decode", seqs=32, longest=4099, heads=32, kv_heads=8, dim=128, page=16,
             io="f16", order="nhd", window=0, sinks=0),
        # two long documents: few rows, so the work has to be split over the length
        dict(name="decode_long", op="decode", seqs=2, longest=131072, heads=32, kv_heads=8, dim=128, page=64,
             io="f32", order="hnd", window=0, sinks=0),
        # a full serving batch, windowed layers with 4 first tokens kept
        dict(name="decode_window", op="decode", seqs=64, longest=16000, heads=64, kv_heads=8, dim=128, page=32,
             io="bf16", order="hnd", window=8192, sinks=4),
        # short turns appended to running chats, small heads, a short window
        dict(name="chunk_turns", op="chunk", seqs=7, chunk=300, longest=1500, heads=16, kv_heads=4, dim=64, page=16,
             io="bf16", order="nhd", window=513, sinks=4),
        # one whole prompt, full causal attention
        dict(name="chunk_prompt", op="chunk", seqs=1, chunk=4096, longest=4096, heads=32, kv_heads=8, dim=128,
             page=64, io="bf16", order="hnd", window=0, sinks=0),
        # a long prompt on a windowed layer
        dict(name="chunk_window", op="chunk", seqs=1, chunk=8192, longest=8192, heads=32, kv_heads=8, dim=128,
             page=64, io="f16", order="hnd", window=2048, sinks=16),
        # positions and append of one decode step of eight users
        dict(name="append_step", op="append", tokens=8, heads=32, kv_heads=8, dim=128, rot=128, page=16, src="f32",
             io="f32", order="hnd", axes=1, pairs="halves"),
        # positions and append of an image-and-text prompt, three axes
        dict(name="append_prompt", op="append", tokens=8192, heads=32, kv_heads=8, dim=128, rot=128, page=16,
             src="bf16", io="bf16", order="nhd", axes=3, pairs="halves"),
        # one user's token through a layer of 64 small experts, 8 of them used
        dict(name="moe_one", op="moe", tokens=1, experts=64, used=8, hidden=2048, ffn=1536, io="bf16",
             score="softmax"),
        # a few users' tokens, which share some experts
        dict(name="moe_few", op="moe", tokens=5, experts=64, used=6, hidden=2048, ffn=1280, io="f16",
             score="sigmoid"),
        # a small batch on eight large experts, every one of which is used
        dict(name="moe_large", op="moe", tokens=16, experts=8, used=2, hidden=4096, ffn=14336, io="bf16",
             score="softmax"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "chunk", "append", "moe", "moe"])
    if op == "moe":
        experts = rng.choice([4, 8, 16, 60, 64, 128])
        hidden, ffn = 256 * _log(rng, 1, 16), 256 * _log(rng, 1, 16)
        tokens, used = _log(rng, 1, 16), rng.randint(1, min(8, experts))
        while min(experts, tokens * used) * hidden * ffn > 8 * 4096 * 14336:
            tokens = -(-tokens // 2)
            ffn = 256 * -(-ffn // 512)
        # 16-bit activations: with f32 ones, a hidden value next to a border of its 8-bit code shows in the output
        return dict(op=op, tokens=tokens, experts=experts, used=used, hidden=hidden, ffn=ffn,
                    io=rng.choice(["bf16", "f16"]), score=rng.choice(["softmax", "sigmoid"]))
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8])
    dim = rng.choice([64, 96, 128, 128, 192, 256])
    order = rng.choice(["hnd", "nhd"])
    if op == "decode":
        longest = _log(rng, 1, 65536)
        most = min(64, max(1, (1 << 30) // (longest * kv_heads * dim * 4)))
        windowed = rng.random() < 0.4
        return dict(op=op, seqs=_log(rng, 1, most), longest=longest, heads=kv_heads * group, kv_heads=kv_heads,
                    dim=dim, page=rng.choice([1, 8, 16, 24, 32, 64, 128]), io=rng.choice(["f32", "bf16", "f16"]),
                    order=order, window=_log(rng, 1, 4096) if windowed else 0,
                    sinks=rng.randint(0, 9) if windowed else 0)
    if op == "chunk":
        longest = _log(rng, 16, 2400)
        windowed = rng.random() < 0.6
        return dict(op=op, seqs=rng.randint(1, 3), chunk=_log(rng, 1, longest), longest=longest,
                    heads=kv_heads * min(group, 4), kv_heads=kv_heads, dim=dim, page=rng.choice([8, 16, 24, 64, 128]),
                    io=rng.choice(["bf16", "f16"]), order=order, window=_log(rng, 1, 4096) if windowed else 0,
                    sinks=rng.randint(0, 70) if windowed else 0)
    return dict(op=op, tokens=_log(rng, 1, 4096), heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                rot=rng.choice([dim, dim // 2, 24]), page=rng.choice([8, 16, 24, 64]),
                src=rng.choice(["f32", "bf16", "f16"]), io=rng.choice(["f32", "bf16", "f16"]), order=order,
                axes=rng.randint(1, 4), pairs=rng.choice(["halves", "adjacent"]))


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _lengths(n, longest):
    """Lengths as a batch has them, a case's own: the longest, then spread over their logarithm."""
    rng = random.Random(64 * longest + n)
    return [longest] + [_log(rng, max(1, longest // 8), longest) for _ in range(n - 1)]


def _chunks(lens, most):
    """How many of each sequence's tokens are new."""
    rng = random.Random(64 * most + len(lens))
    return [min(n, most) if i == 0 else min(n, _log(rng, 1, most)) for i, n in enumerate(lens)]


def _exponent_bytes(dim):
    """Bytes of a row's exponents: one for 32 dims, rows of 4 or 8."""
    return 4 if dim <= 128 else 8


def _encode(x):
    """[..., dim] in 64 or 32 bits -> packed codes [..., dim / 2] and exponents [..., 4 or 8]."""
    blocks = x.unflatten(-1, (-1, 32))
    largest = blocks.abs().amax(-1)
    # frexp: largest = f * 2^e with f in [0.5, 1). The largest rounds to 6 at most: below 7 * 2^(e - 3).
    f, e = torch.frexp(largest)
    e = torch.where(f >= 0.875, e - 2, e - 3).clamp(-23, 13)
    u = torch.ldexp(blocks.abs(), -e[..., None])
    code = torch.zeros_like(u, dtype=torch.uint8)
    for border, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (u >= border if up else u > border)
    code |= torch.signbit(blocks).to(torch.uint8) << 3
    code = code.flatten(-2)
    exps = torch.zeros(*x.shape[:-1], _exponent_bytes(x.shape[-1]), dtype=torch.uint8, device=x.device)
    exps[..., :e.shape[-1]] = (e + 127).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), exps


def _pool(pages, kv_heads, page, dim, order, g, spread):
    """A pool's codes and exponents, seen as [pages, kv_heads, page, .]; "nhd" stores a page token by token."""
    front = (kv_heads, page) if order == "hnd" else (page, kv_heads)
    codes = torch.empty(pages, *front, dim // 2, dtype=torch.uint8, device=DEV)
    exps = torch.empty(pages, *front, _exponent_bytes(dim), dtype=torch.uint8, device=DEV)
    # some channels are larger than others, as keys have them
    channel = torch.exp(spread * torch.randn(dim, device=DEV, generator=g))
    step = max(1, (1 << 25) // (kv_heads * page * dim))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        x = torch.randn(n, *front, dim, device=DEV, generator=g) * channel
        codes[at:at + n], exps[at:at + n] = _encode(x)
    if order == "nhd":
        codes, exps = codes.transpose(1, 2), exps.transpose(1, 2)
    return codes, exps


def _tables(lens, page, spare, rng):
    """Each sequence's pages, in an order that a running server's pool has; -1 where a row ends."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + spare
    ids = list(range(total))
    rng.shuffle(ids)
    rows, at = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32), 0
    for i, n in enumerate(need):
        rows[i, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
        at += n
    return rows.to(DEV), total


def _attention_state(c, seed):
    rng, g = random.Random(seed), _gen(seed)
    lens = _lengths(c["seqs"], c["longest"])
    tables, pages = _tables(lens, c["page"], 3, rng)
    s = dict(c, tables=tables, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), host_lens=lens,
             scale=c["dim"] ** -0.5, k_scale=0.75, v_scale=1.25)
    s["k"], s["k_exp"] = _pool(pages, c["kv_heads"], c["page"], c["dim"], c["order"], g, 0.5)
    s["v"], s["v_exp"] = _pool(pages, c["kv_heads"], c["page"], c["dim"], c["order"], g, 0.0)
    if c["op"] == "decode":
        rows = c["seqs"]
    else:
        chunks = _chunks(lens, c["chunk"])
        starts = [0]
        for n in chunks:
            starts.append(starts[-1] + n)
        rows = starts[-1]
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
        s["host_starts"], s["most"] = starts, max(chunks)
    s["q"] = torch.randn(rows, c["heads"], c["dim"], device=DEV, generator=g).to(TYPES[c["io"]])
    s["out"] = torch.empty_like(s["q"])
    return s


def _sections(rot, axes):
    base = rot // 2 // axes
    return [rot // 2 - base * (axes - 1)] + [base] * (axes - 1)


def _append_state(c, seed):
    rng, g = random.Random(seed), _gen(seed)
    T, H, K, D = c["tokens"], c["heads"], c["kv_heads"], c["dim"]
    s = dict(c, sections=_sections(c["rot"], c["axes"]), k_scale=0.75, v_scale=1.25)
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device=DEV)
    s["freq"] = 500000.0 ** (-2.0 * i / c["rot"])
    # a text of T tokens somewhere in a long context; the other axes are grid places
    first = rng.randint(0, 200000)
    pos = torch.randint(0, 1000, (c["axes"], T), device=DEV, generator=g, dtype=torch.int32)
    pos[0] = first + torch.arange(T, device=DEV, dtype=torch.int32)
    s["pos"] = pos
    # one row of the qkv product's output per token; q, k and v are its slices
    s["qkv"] = torch.randn(T, H + 2 * K, D, device=DEV, generator=g).to(TYPES[c["src"]])
    pages = -(-T // c["page"]) + 2
    s["k"], s["k_exp"] = _pool(pages, K, c["page"], D, c["order"], g, 0.5)
    s["v"], s["v_exp"] = _pool(pages, K, c["page"], D, c["order"], g, 0.0)
    order = list(range(pages))
    rng.shuffle(order)
    t = torch.arange(T)
    s["slots"] = (torch.tensor(order)[t // c["page"]] * c["page"] + t % c["page"]).to(DEV)
    s["out"] = torch.empty(T, H, D, dtype=TYPES[c["io"]], device=DEV)
    s["k_back"] = torch.empty(T, K, D, dtype=torch.bfloat16, device=DEV)
    s["v_back"] = torch.empty(T, K, D, dtype=torch.bfloat16, device=DEV)
    return s


def _q4k(rows, columns, g):
    """Q4_K super-blocks of `rows` x `columns` weights around zero: two f16 scales, 12 bytes of 6-bit scales, nibbles."""
    n = rows * columns // 256
    raw = torch.randint(0, 256, (n, 144), device=DEV, generator=g, dtype=torch.uint8)
    d = (torch.rand(n, device=DEV, generator=g) + 0.5) * 1.2e-4
    raw[:, 0:2] = d.half().view(torch.uint8).view(n, 2)
    raw[:, 2:4] = (7.5 * d).half().view(torch.uint8).view(n, 2)
    return raw.view(-1)


def _moe_state(c, seed):
    g = _gen(seed)
    T, E, K, F = c["tokens"], c["experts"], c["hidden"], c["ffn"]
    s = dict(c, gate=_q4k(E * F, K, g), up=_q4k(E * F, K, g), down=_q4k(E * K, F, g))
    s["x"] = torch.randn(T, K, device=DEV, generator=g).to(TYPES[c["io"]])
    s["router"] = (torch.randn(E, K, device=DEV, generator=g) * K ** -0.5).to(torch.bfloat16)
    # a bias that evens out the experts' loads comes with sigmoid scores
    s["bias"] = 0.1 * torch.randn(E, device=DEV, generator=g) if c["score"] == "sigmoid" else None
    s["factor"] = 2.5 if c["score"] == "sigmoid" else 1.0
    s["ids"] = torch.empty(T, c["used"], dtype=torch.int32, device=DEV)
    s["weights"] = torch.empty(T, c["used"], dtype=torch.float32, device=DEV)
    s["y"] = torch.empty_like(s["x"])
    return s


def prepare(case, seed):
    s = {"decode": _attention_state, "chunk": _attention_state, "append": _append_state,
         "moe": _moe_state}[case["op"]](case, seed)
    if own:
        import quantized_decode_mat_amd as xq
        if "k" in s:
            four, exps = torch.float4_e2m1fn_x2, torch.float8_e8m0fnu
            s["kv"] = xq.xq_kv_cache(s["k"].view(four), s["v"].view(four), s["k_scale"], s["v_scale"],
                                     k_exp=s["k_exp"].view(exps), v_exp=s["v_exp"].view(exps))
        need = 0
        if case["op"] == "append":
            s["rope"] = xq.xq_rope_plan(s["freq"], s["sections"], s["pairs"] == "adjacent")
        elif case["op"] == "decode":
            need = xq.xq_attn_decode_workspace_bytes(case["seqs"], case["heads"], s["kv"], case["longest"],
                                                     case["window"], case["sinks"])
        elif case["op"] == "moe":
            need = max(xq.xq_moe_route_workspace_bytes(case["tokens"], case["experts"]),
                       xq.xq_moe_q4k_workspace_bytes(case["tokens"], case["used"], case["hidden"], case["ffn"]))
        s["ws"] = torch.zeros(need, dtype=torch.uint8, device=DEV) if need else None
    return s


# ---------------------------------------------------------------- the framework's calls

def _own(s):
    import quantized_decode_mat_amd as xq
    op = s["op"]
    if op == "decode":
        xq.xq_attn_decode(s["out"], s["q"], s["kv"], s["tables"], s["lens"], s["scale"], window=s["window"],
                          sinks=s["sinks"], max_len=s["longest"], workspace=s["ws"])
        return s["out"]
    if op == "chunk":
        xq.xq_attn_prefill(s["out"], s["q"], s["kv"], s["tables"], s["lens"], s["starts"], s["most"], s["scale"],
                           window=s["window"], sinks=s["sinks"])
        return s["out"]
    if op == "append":
        H, K = s["heads"], s["kv_heads"]
        x = s["qkv"]
        xq.xq_rope_append(s["out"], s["kv"], x[:, :H], x[:, H:H + K], x[:, H + K:], s["pos"], s["rope"], s["slots"])
        xq.xq_cache_read(s["k_back"], s["v_back"], s["kv"], s["slots"])
        return s["out"], s["k_back"], s["v_back"]
    xq.xq_moe_route(s["ids"], s["weights"], s["x"], s["router"], bias=s["bias"], score=s["score"], normalize=True,
                    scale=s["factor"], workspace=s["ws"])
    xq.xq_moe_q4k(s["y"], s["x"], s["gate"], s["up"], s["down"], s["ids"], s["weights"], s["experts"], s["ffn"],
                  workspace=s["ws"])
    return s["y"], s["ids"], s["weights"]


# ---------------------------------------------------------------- plain forms

_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _decode_rows(codes, exps):
    """Packed codes [..., dim / 2] and exponents -> values in 32 bits, [..., dim]."""
    values = torch.tensor(_VALUES + tuple(-v for v in _VALUES), device=DEV)
    byte = torch.arange(256, device=DEV)
    pairs = torch.stack((values[byte & 15], values[byte >> 4]), -1)
    x = pairs[codes.int()].flatten(-2)
    e = exps[..., :x.shape[-1] // 32].int() - 127
    return torch.ldexp(x.unflatten(-1, (-1, 32)), e[..., None]).flatten(-2)


def _gathered(s, name):
    """[seqs, kv_heads, length, dim] in 32 bits through the table."""
    rows = s["tables"].long().clamp(min=0)
    x = _decode_rows(s[name][rows], s[name + "_exp"][rows])
    x = x.transpose(1, 2).reshape(len(rows), s["kv_heads"], -1, s["dim"])
    return x.mul_(s[name + "_scale"])


def _visible(s, pos, length):
    j = torch.arange(length, device=DEV)
    ok = j <= pos[..., None]
    if s["window"]:
        ok &= (j > pos[..., None] - s["window"]) | (j < s["sinks"])
    return ok


def _softmax_product(scores, ok, v):
    scores = scores.masked_fill_(~ok, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-3e38)
    p = scores.sub_(top).exp_()
    return (p @ v) / p.sum(-1, keepdim=True).clamp(min=1e-38)


def _plain_decode(s):
    k, v = _gathered(s, "k"), _gathered(s, "v")
    B, H, K, D = s["seqs"], s["heads"], s["kv_heads"], s["dim"]
    q = s["q"].float().reshape(B, K, H // K, D)
    ok = _visible(s, s["lens"].long() - 1, k.shape[2])[:, None, None]
    out = _softmax_product((q @ k.transpose(-1, -2)) * s["scale"], ok, v)
    return out.reshape(B, H, D).to(s["q"].dtype)


def _plain_chunk(s):
    k, v = _gathered(s, "k"), _gathered(s, "v")
    B, H, K, D, n = s["seqs"], s["heads"], s["kv_heads"], s["dim"], s["most"]
    starts, lens = s["starts"].long(), s["lens"].long()
    count = starts[1:] - starts[:-1]
    i = torch.arange(n, device=DEV)
    at = (starts[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)          # padded rows repeat a real one
    pos = (lens - count)[:, None] + i
    q = s["q"].float()[at].reshape(B, n, K, H // K, D).permute(0, 2, 3, 1, 4).reshape(B, K, -1, D)
    scores = (q @ k.transpose(-1, -2)).mul_(s["scale"]).view(B, K, H // K, n, -1)
    ok = _visible(s, pos, k.shape[2])[:, None, None]
    ok = ok.expand(-1, 1, H // K, -1, -1).reshape(B, 1, -1, k.shape[2])
    out = _softmax_product(scores.view(B, K, -1, k.shape[2]), ok, v)
    out = out.reshape(B, K, H // K, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, H, D)
    t = torch.arange(s["q"].shape[0], device=DEV)
    b = torch.searchsorted(starts, t, right=True) - 1
    return out[b, t - starts[b]].to(s["q"].dtype)


def _rotated(s, x, cos, sin):
    r = s["rot"]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if s["pairs"] == "adjacent" else (x[..., :r // 2], x[..., r // 2:r])
    y, z = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((y, z), -1).flatten(-2) if s["pairs"] == "adjacent" else torch.cat((y, z), -1)
    return torch.cat((turned, x[..., r:]), -1)


def _plain_append(s):
    axis = torch.repeat_interleave(torch.arange(s["axes"], device=DEV),
                                   torch.tensor(s["sections"], device=DEV), output_size=s["rot"] // 2)
    a = s["pos"].double()[axis].t() * s["freq"]                          # far positions need 64 bits
    cos, sin = a.cos()[:, None], a.sin()[:, None]
    H, K = s["heads"], s["kv_heads"]
    x = s["qkv"]
    out = _rotated(s, x[:, :H].float(), cos.float(), sin.float()).to(TYPES[s["io"]])
    # a value next to a border between two codes needs 64 bits
    k = _rotated(s, x[:, H:H + K].double(), cos, sin) / s["k_scale"]
    v = x[:, H + K:].double() / s["v_scale"]
    at, slot = s["slots"] // s["page"], s["slots"] % s["page"]
    back = []
    for name, value in (("k", k), ("v", v)):
        s[name][at, :, slot], s[name + "_exp"][at, :, slot] = _encode(value)
        back.append((_decode_rows(s[name][at, :, slot], s[name + "_exp"][at, :, slot]) * s[name + "_scale"]).bfloat16())
    return out, back[0], back[1]


def _q4k_values(raw):
    """Q4_K super-blocks [..., blocks, 144] -> weights in 32 bits, [..., blocks * 256]."""
    d = raw[..., 0:2].contiguous().view(torch.float16).float()[..., 0]
    dmin = raw[..., 2:4].contiguous().view(torch.float16).float()[..., 0]
    sc, m, mix = raw[..., 4:8], raw[..., 8:12], raw[..., 12:16]
    scales = torch.cat((sc & 63, (mix & 15) | ((sc >> 6) << 4)), -1).float() * d[..., None]
    mins = torch.cat((m & 63, (mix >> 4) | ((m >> 6) << 4)), -1).float() * dmin[..., None]
    nibbles = raw[..., 16:].unflatten(-1, (4, 32))
    q = torch.stack((nibbles & 15, nibbles >> 4), -2).flatten(-3, -2).float()     # [..., blocks, 8, 32]
    return q.mul_(scales[..., None]).sub_(mins[..., None]).flatten(-3)


def _q8k_values(x):
    """What q8_K holds of x in 32 bits: 256 values share max|x| / 127."""
    blocks = x.unflatten(-1, (-1, 256))
    d = blocks.abs().amax(-1, keepdim=True) / 127
    return (torch.round(blocks / torch.where(d > 0, d, 1)) * d).flatten(-2)


def _plain_moe(s):
    T, E, U, K, F = s["tokens"], s["experts"], s["used"], s["hidden"], s["ffn"]
    logits = s["x"].float() @ s["router"].float().t()
    scores = torch.softmax(logits, -1) if s["score"] == "softmax" else torch.sigmoid(logits)
    order = scores if s["bias"] is None else scores + s["bias"]
    ids = torch.sort(order, dim=-1, descending=True, stable=True)[1][:, :U]           # ties go to the lowest index
    weights = scores.gather(-1, ids)
    weights = weights / weights.sum(-1, keepdim=True) * s["factor"]
    x = _q8k_values(s["x"].float())
    gate, up, down = s["gate"].view(E, F, -1, 144), s["up"].view(E, F, -1, 144), s["down"].view(E, K, -1, 144)
    if T * U <= E:                                                                # the chosen experts alone
        g = torch.matmul(_q4k_values(gate[ids]), x[:, None, :, None])[..., 0]
        u = torch.matmul(_q4k_values(up[ids]), x[:, None, :, None])[..., 0]
        h = _q8k_values(g * torch.sigmoid(g) * u)
        y = torch.matmul(_q4k_values(down[ids]), h[..., None])[..., 0]
    else:                                                                         # all of them, then the chosen
        g = (x @ _q4k_values(gate).view(E * F, K).t()).view(T, E, F)
        u = (x @ _q4k_values(up).view(E * F, K).t()).view(T, E, F)
        h = _q8k_values(g * torch.sigmoid(g) * u)
        y = torch.bmm(h.transpose(0, 1).contiguous(), _q4k_values(down).transpose(1, 2).contiguous()).transpose(0, 1)
        y = y.gather(1, ids[..., None].expand(-1, -1, K))
    y = (y * weights[..., None]).sum(1)
    return y.to(s["x"].dtype), ids.int(), weights


def run(state):
    if own:
        return _own(state)
    return {"decode": _plain_decode, "chunk": _plain_chunk, "append": _plain_append, "moe": _plain_moe}[
        state["op"]](state)


# ---------------------------------------------------------------- 64 bits, apart from the plain forms

def _rows64(s, name, b, where):
    """Tokens `where` of sequence b, [tokens, kv_heads, dim], by the codes' fields."""
    page = s["tables"][b].long()[where // s["page"]]
    byte = s[name][page, :, where % s["page"]]
    code = torch.empty(*byte.shape[:-1], s["dim"], dtype=torch.int64, device=DEV)
    code[..., 0::2] = byte & 15
    code[..., 1::2] = byte >> 4
    exponent, half = (code >> 1) & 3, (code & 1).double()
    size = torch.where(exponent == 0, half / 2, (1 + half / 2) * 2.0 ** (exponent - 1).double())
    power = s[name + "_exp"][page, :, where % s["page"]][..., :s["dim"] // 32].double() - 127
    sign = 1.0 - 2.0 * (code >> 3).double()
    return sign * size * torch.repeat_interleave(2.0 ** power, 32, -1) * s[name + "_scale"]


def _attend64(s, q, pos, b, hi):
    """q [rows, heads, dim] at positions pos of sequence b, whose first `hi` tokens are looked at."""
    lo = 0
    if s["window"]:
        lo = max(0, int(pos.min()) - s["window"] + 1)
    where = torch.arange(lo, hi, device=DEV)
    if lo:
        where = torch.cat((torch.arange(0, min(s["sinks"], lo), device=DEV), where))
    k, v = _rows64(s, "k", b, where), _rows64(s, "v", b, where)
    hidden = where[None] > pos[:, None]
    if s["window"]:
        hidden |= (where[None] + s["window"] <= pos[:, None]) & (where[None] >= s["sinks"])
    group, out = s["heads"] // s["kv_heads"], []
    for h in range(s["heads"]):
        e = torch.mm(q[:, h].double(), k[:, h // group].t().contiguous()) * s["scale"]
        e[hidden] = -math.inf
        out.append(torch.mm(torch.softmax(e, -1), v[:, h // group].contiguous()))
    return torch.stack(out, 1)


def _nearest64(x):
    """What 32 values hold of x, [..., 32]: the power by trial, each value the nearest of the eight."""
    sizes = torch.tensor(_VALUES, dtype=torch.float64, device=DEV)
    largest = x.abs().amax(-1, keepdim=True)
    power = torch.full_like(largest, 2.0 ** -23)
    for _ in range(36):                                                  # up to 2^13
        power = torch.where(largest >= 7 * power, 2 * power, power)
    u = (x.abs() / power).clamp(max=6.0)[..., None]
    gap = (u - sizes).abs()
    # of two equally near the one with an even index
    rank = torch.tensor([0, 1] * 4, dtype=torch.float64, device=DEV)
    near = gap <= gap.amin(-1, keepdim=True)
    pick = torch.where(near, rank, 2.0).argmin(-1)
    return torch.copysign(sizes[pick], x) * power


def _exact_append(case, s):
    half, turn = case["rot"] // 2, []
    for axis, count in enumerate(s["sections"]):
        i = len(turn)
        turn += [s["pos"][axis].double() * s["freq"][i + j] for j in range(count)]
    turn = torch.stack(turn, 1)
    turn = torch.complex(turn.cos(), turn.sin())

    def rotate(x):
        x = x.double().clone()
        even = torch.arange(half, device=DEV) * (2 if case["pairs"] == "adjacent" else 1)
        odd = even + (1 if case["pairs"] == "adjacent" else half)
        z = torch.complex(x[..., even], x[..., odd]) * turn[:, None]
        x[..., even], x[..., odd] = z.real, z.imag
        return x

    def held(x, scale):
        return torch.cat([_nearest64((y / scale).unflatten(-1, (-1, 32))).flatten(-2) * scale for y in x.split(256)])

    H, K = case["heads"], case["kv_heads"]
    k, v = rotate(s["qkv"][:, H:H + K]), s["qkv"][:, H + K:].double()
    return rotate(s["qkv"][:, :H]), held(k, s["k_scale"]), held(v, s["v_scale"])


def _q4k64(raw):
    """Q4_K super-blocks [rows, blocks, 144] -> [rows, blocks * 256], sub-block by sub-block."""
    d = raw[..., 0:2].contiguous().view(torch.float16).double()
    dmin = raw[..., 2:4].contiguous().view(torch.float16).double()
    b, parts = raw.long(), []
    for j in range(8):
        if j < 4:
            sc, m = b[..., 4 + j] % 64, b[..., 8 + j] % 64
        else:
            sc = b[..., 8 + j] % 16 + b[..., j] // 64 * 16
            m = b[..., 8 + j] // 16 + b[..., 4 + j] // 64 * 16
        group = b[..., 16 + 32 * (j // 2):48 + 32 * (j // 2)]
        q = group // 16 if j % 2 else group % 16
        parts.append(d * sc[..., None].double() * q.double() - dmin * m[..., None].double())
    return torch.cat(parts, -1).flatten(-2)


def _q8k64(x):
    """q8_K is defined in 32 bits: the scale one division, each code another."""
    out = []
    for block in x.float().split(256, -1):
        d = block.abs().amax(-1, keepdim=True) / 127
        code = torch.where(d > 0, torch.round(block / d), 0.0)
        out.append(code.double() * d.double())
    return torch.cat(out, -1)


def _exact_moe(case, s):
    T, E, U, K, F = case["tokens"], case["experts"], case["used"], case["hidden"], case["ffn"]
    logits = torch.stack([(s["router"].double() * x.double()).sum(-1) for x in s["x"]])
    if case["score"] == "softmax":
        scores = torch.exp(logits - torch.logsumexp(logits, -1, keepdim=True))
    else:
        scores = 1 / (1 + torch.exp(-logits))
    left = scores.clone() if s["bias"] is None else scores + s["bias"].double()
    ids = torch.empty(T, U, dtype=torch.int32, device=DEV)
    for k in range(U):
        best = torch.where(left == left.amax(-1, keepdim=True), torch.arange(E, device=DEV), E).amin(-1)
        ids[:, k] = best.int()
        left.scatter_(1, best[:, None], -math.inf)
    weights = scores.gather(1, ids.long())
    weights = weights / weights.sum(-1, keepdim=True) * s["factor"]
    x = _q8k64(s["x"])
    y = torch.zeros(T, K, dtype=torch.float64, device=DEV)
    chosen = ids.cpu().tolist()
    for e in sorted({e for row in chosen for e in row}):
        at = [(t, k) for t in range(T) for k in range(U) if chosen[t][k] == e]
        t, k = torch.tensor([p[0] for p in at], device=DEV), torch.tensor([p[1] for p in at], device=DEV)

        def product(name, rows, v):
            raw = s[name].view(E, rows, -1, 144)[e]
            return torch.cat([v @ _q4k64(part).t().contiguous() for part in raw.split(4096)], 1)

        g, u = product("gate", F, x[t]), product("up", F, x[t])
        d = product("down", K, _q8k64(g / (1 + torch.exp(-g)) * u))
        y.index_add_(0, t, d * weights[t, k][:, None])
    return y, None, weights


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "decode":
        return torch.cat([_attend64(s, s["q"][b:b + 1], s["lens"][b:b + 1].long() - 1, b, n)
                          for b, n in enumerate(s["host_lens"])])
    if case["op"] == "chunk":
        out = []
        for b, n in enumerate(s["host_lens"]):
            first, end = s["host_starts"][b:b + 2]
            for at in range(first, end, 1024):
                to = min(end, at + 1024)
                pos = torch.arange(n - end + at, n - end + to, device=DEV)
                out.append(_attend64(s, s["q"][at:to], pos, b, n - end + to))
        return torch.cat(out)
    if case["op"] == "append":
        return _exact_append(case, s)
    return _exact_moe(case, s)


# ---------------------------------------------------------------- work

def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if case["op"] == "moe":
        T, E, U, K, F = case["tokens"], case["experts"], case["used"], case["hidden"], case["ffn"]
        # experts that T tokens choose, on the average; each one's three matrices are read once
        distinct = E * (1 - (1 - U / E) ** T)
        return {"bytes": distinct * 3 * K * F // 256 * 144 + 2 * E * K + 2 * T * K * size[case["io"]] + 8 * T * U,
                "flops": 6 * T * U * K * F + 2 * T * E * K}
    H, K, D = case["heads"], case["kv_heads"], case["dim"]
    row = D // 2 + D // 32
    if case["op"] == "append":
        T = case["tokens"]
        # q, k and v in, q out, the rows written, read and given back as values
        return {"bytes": T * H * D * (size[case["src"]] + size[case["io"]]) + 8 * T + 4 * case["axes"] * T +
                         2 * T * K * (D * size[case["src"]] + 2 * row + 2 * D),
                "flops": 3 * T * (H + K) * case["rot"]}
    lens = _lengths(case["seqs"], case["longest"])
    w, sinks = case["window"], case["sinks"]

    def seen(pos):
        return pos + 1 if not w or pos < w else w + min(sinks, pos - w + 1)

    if case["op"] == "decode":
        touched = [seen(n - 1) for n in lens]
        rows, pairs = case["seqs"], sum(touched)
    else:
        chunks = _chunks(lens, case["chunk"])
        rows = sum(chunks)
        pairs = sum(seen(p) for n, m in zip(lens, chunks) for p in range(n - m, n))
        touched = [n if not w or n - m < w else min(n, m + w - 1 + min(sinks, n - m - w + 1))
                   for n, m in zip(lens, chunks)]
    return {"bytes": 2 * sum(touched) * K * row + 2 * rows * H * D * size[case["io"]], "flops": 4 * pairs * H * D}
