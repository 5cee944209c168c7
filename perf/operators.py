"""The operators of the paged key-value cache: what is measured, and their plain forms.

Four operators: attention of one new token per sequence over a paged cache (``decode``), attention of a chunk of
tokens with a sliding window and first tokens that stay visible (``prefill``), rotary positions with several axes,
fused with the write into the pages, and its gradient (``rope``), and the pages' management (``pages``).
"""

import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


def listed():
    return [
        # one user's chat, a few hundred tokens in: the call's latency
        dict(name="decode_one_short", op="decode", seqs=1, longest=517, heads=32, kv_heads=8, dim=128, page=16,
             cache="bf16", io="f32", order="hnd", window=0, sinks=0),
        # a ragged serving batch on the 4096-wide layer's heads
        dict(name="decode_batch_ragged", op="decode", seqs=32, longest=4099, heads=32, kv_heads=8, dim=128, page=16,
             cache="f16", io="f16", order="nhd", window=0, sinks=0),
        # two long documents: few rows, so the work has to be split over the length
        dict(name="decode_long", op="decode", seqs=2, longest=131072, heads=32, kv_heads=8, dim=128, page=64,
             cache="bf16", io="f32", order="hnd", window=0, sinks=0),
        # a full serving batch on an 8-bit cache, windowed layers with 4 first tokens kept
        dict(name="decode_window_8bit", op="decode", seqs=64, longest=16000, heads=64, kv_heads=8, dim=128, page=32,
             cache="e4m3", io="bf16", order="hnd", window=8192, sinks=4),
        # short turns appended to running chats, small heads, a short window
        dict(name="prefill_turns", op="prefill", seqs=7, chunk=300, longest=1500, heads=16, kv_heads=4, dim=64,
             page=16, cache="bf16", io="bf16", order="nhd", window=513, sinks=4),
        # one whole prompt, full causal attention
        dict(name="prefill_prompt", op="prefill", seqs=1, chunk=4096, longest=4096, heads=32, kv_heads=8, dim=128,
             page=64, cache="bf16", io="bf16", order="hnd", window=0, sinks=0),
        # a long prompt on a windowed layer
        dict(name="prefill_window", op="prefill", seqs=1, chunk=8192, longest=8192, heads=32, kv_heads=8, dim=128,
             page=64, cache="f16", io="f16", order="hnd", window=2048, sinks=16),
        # positions and append of one decode step of eight users, text positions
        dict(name="rope_decode_step", op="rope", tokens=8, heads=32, kv_heads=8, dim=128, rot=128, page=16, src="f32",
             io="f32", cache="bf16", order="hnd", axes=1, pairs="halves", back=False),
        # positions and append of an image-and-text prompt, three axes
        dict(name="rope_prompt_3axes", op="rope", tokens=8192, heads=32, kv_heads=8, dim=128, rot=128, page=16,
             src="f32", io="bf16", cache="bf16", order="nhd", axes=3, pairs="halves", back=False),
        # the gradient of video positions, adjacent pairs, part of each head rotated
        dict(name="rope_gradient", op="rope", tokens=4500, heads=24, kv_heads=8, dim=96, rot=64, page=16, src="bf16",
             io="bf16", cache="bf16", order="hnd", axes=3, pairs="adjacent", back=True),
        # a beam search's step: the losing beams are freed, the winners forked
        dict(name="pages_beams", op="pages", what="beams", layers=4, pages=4096, page=16, kv_heads=8, dim=128,
             cache="bf16", slots=128, longest=1000),
        # a fragmented pool is moved together
        dict(name="pages_compact", op="pages", what="compact", layers=8, pages=8192, page=16, kv_heads=8, dim=128,
             cache="bf16", slots=64, longest=2000),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "rope", "pages"])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8])
    dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
    order = rng.choice(["hnd", "nhd"])
    if op == "decode":
        cache = rng.choice(["bf16", "f16", "e4m3"])
        longest = _log(rng, 1, 32768)
        most = min(64, max(1, (1 << 30) // (longest * kv_heads * dim * 4)))
        windowed = rng.random() < 0.4
        return dict(op=op, seqs=_log(rng, 1, most), longest=longest, heads=kv_heads * group, kv_heads=kv_heads,
                    dim=dim, page=rng.choice([1, 8, 16, 24, 32, 64, 128]), cache=cache,
                    io=rng.choice(["f32", "bf16", "f16"]), order=order,
                    window=_log(rng, 1, 4096) if windowed else 0, sinks=rng.randint(0, 9) if windowed else 0)
    if op == "prefill":
        io = rng.choice(["bf16", "f16"])
        longest = _log(rng, 16, 2400)
        windowed = rng.random() < 0.6
        return dict(op=op, seqs=rng.randint(1, 3), chunk=_log(rng, 1, longest), longest=longest,
                    heads=kv_heads * min(group, 4), kv_heads=kv_heads, dim=dim, page=rng.choice([8, 16, 24, 64, 128]),
                    cache=rng.choice([io, io, "e4m3"]), io=io, order=order,
                    window=_log(rng, 1, 4096) if windowed else 0, sinks=rng.randint(0, 70) if windowed else 0)
    if op == "rope":
        back = rng.random() < 0.3
        return dict(op=op, tokens=_log(rng, 1, 4096), heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim // 2]), page=rng.choice([8, 16, 24, 64]),
                    src=rng.choice(["f32", "bf16", "f16"]), io=rng.choice(["f32", "bf16", "f16"]),
                    cache=rng.choice(["bf16", "f16", "e4m3"]), order=order, axes=rng.randint(1, 4),
                    pairs=rng.choice(["halves", "adjacent"]), back=back)
    return dict(op=op, what=rng.choice(["beams", "compact", "copy"]), layers=rng.randint(1, 4),
                pages=_log(rng, 512, 4096), page=rng.choice([8, 16, 24, 32]), kv_heads=kv_heads, dim=dim,
                cache=rng.choice(["bf16", "f16", "e4m3"]), slots=2 * _log(rng, 4, 48), longest=_log(rng, 8, 120))


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


def _pool(shape, order, kind, g):
    """A pool of pages [..., pages, kv_heads, page, dim]; "nhd" stores a page token by token."""
    *front, heads, page, dim = shape
    stored = (*front, heads, page, dim) if order == "hnd" else (*front, page, heads, dim)
    x = torch.empty(stored, dtype=TYPES[kind], device=DEV)
    flat = x.reshape(-1)
    for at in range(0, flat.numel(), 1 << 27):
        n = min(1 << 27, flat.numel() - at)
        flat[at:at + n] = torch.randn(n, device=DEV, generator=g).to(TYPES[kind])
    return x if order == "hnd" else x.transpose(-3, -2)


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
    shape = (pages, c["kv_heads"], c["page"], c["dim"])
    s = dict(c, k=_pool(shape, c["order"], c["cache"], g), v=_pool(shape, c["order"], c["cache"], g), tables=tables,
             lens=torch.tensor(lens, dtype=torch.int32, device=DEV), host_lens=lens, scale=c["dim"] ** -0.5)
    eight = c["cache"] == "e4m3"
    s["k_scale"], s["v_scale"] = (0.75, 1.25) if eight else (1.0, 1.0)
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
    q = torch.randn(rows, c["heads"], c["dim"], device=DEV, generator=g)
    s["q"] = q.to(TYPES[c["io"]])
    s["out"] = torch.empty_like(s["q"])
    return s


def _sections(rot, axes):
    base = rot // 2 // axes
    return [rot // 2 - base * (axes - 1)] + [base] * (axes - 1)


def _rope_state(c, seed):
    rng, g = random.Random(seed), _gen(seed)
    T, H, K, D = c["tokens"], c["heads"], c["kv_heads"], c["dim"]
    s = dict(c, sections=_sections(c["rot"], c["axes"]))
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device=DEV)
    s["freq"] = 500000.0 ** (-2.0 * i / c["rot"])
    # a text of T tokens somewhere in a long context; the other axes are grid places
    first = rng.randint(0, 200000)
    pos = torch.randint(0, 1000, (c["axes"], T), device=DEV, generator=g, dtype=torch.int32)
    pos[0] = first + torch.arange(T, device=DEV, dtype=torch.int32)
    s["pos"] = pos
    if c["back"]:
        s["x"] = torch.randn(T, H, D, device=DEV, generator=g).to(TYPES[c["src"]])
        s["out"] = torch.empty(T, H, D, dtype=TYPES[c["io"]], device=DEV)
        return s
    # one row of the qkv product's output per token; q, k and v are its slices
    s["qkv"] = torch.randn(T, H + 2 * K, D, device=DEV, generator=g).to(TYPES[c["src"]])
    pages = -(-T // c["page"]) + 2
    shape = (pages, K, c["page"], D)
    s["k"], s["v"] = _pool(shape, c["order"], c["cache"], g), _pool(shape, c["order"], c["cache"], g)
    order = list(range(pages))
    rng.shuffle(order)
    t = torch.arange(T)
    s["slots"] = (torch.tensor(order)[t // c["page"]] * c["page"] + t % c["page"]).to(DEV)
    s["k_scale"], s["v_scale"] = (0.05, 0.04) if c["cache"] == "e4m3" else (1.0, 1.0)
    s["out"] = torch.empty(T, H, D, dtype=TYPES[c["io"]], device=DEV)
    return s


def _filled(c):
    """The token counts of the rows that hold pages, a case's own, and how many pages they hold."""
    rng = random.Random(64 * c["longest"] + c["slots"])
    beams = c["what"] == "beams"
    rows = c["slots"] // 2 if beams else c["slots"]
    room = c["pages"] - rows if beams else c["pages"] * 3 // 5
    lens, used = [], 0
    for i in range(rows):
        n = min(_log(rng, max(1, c["longest"] // 4), c["longest"]),
                max(1, (room - used) * c["page"] // (c["slots"] - i)))
        lens.append(n)
        used += -(-n // c["page"])
    return lens, used


def _pages_state(c, seed):
    rng, g = random.Random(seed), _gen(seed)
    page, pages, slots = c["page"], c["pages"], c["slots"]
    shape = (c["layers"], pages, c["kv_heads"], page, c["dim"])
    s = dict(c, k=_pool(shape, "hnd", c["cache"], g), v=_pool(shape, "hnd", c["cache"], g))
    if c["what"] == "copy":
        ids = list(range(pages))
        rng.shuffle(ids)
        n = pages // 2
        s["src"] = torch.tensor(ids[:n], dtype=torch.int32, device=DEV)
        s["dst"] = torch.tensor(ids[n:2 * n], dtype=torch.int32, device=DEV)
        return s
    half = slots // 2
    lens, used = _filled(c)
    width = -(-c["longest"] // page) + 1
    ids = rng.sample(range(pages), used)
    tables, at = torch.full((slots, width), -1, dtype=torch.int32), 0
    refs = torch.zeros(pages, dtype=torch.int32)
    for i, n in enumerate(lens):
        k = -(-n // page)
        tables[i, :k] = torch.tensor(ids[at:at + k], dtype=torch.int32)
        at += k
    refs[torch.tensor(ids, dtype=torch.int64)] = 1
    lens += [0] * (slots - len(lens))
    s["refs"], s["tables"] = refs.to(DEV), tables.to(DEV)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["status"] = torch.zeros(2, dtype=torch.int32, device=DEV)
    if c["what"] == "beams":
        kids = list(range(half, slots))
        rng.shuffle(kids)
        s["children"] = torch.tensor(kids, dtype=torch.int32, device=DEV)
        s["parents"] = torch.tensor([rng.randrange(half) for _ in kids], dtype=torch.int32, device=DEV)
    else:
        s["refs0"], s["tables0"] = s["refs"].clone(), s["tables"].clone()
    return s


def prepare(case, seed):
    s = {"decode": _attention_state, "prefill": _attention_state, "rope": _rope_state,
         "pages": _pages_state}[case["op"]](case, seed)
    if own:
        import quantized_decode_mat_amd as xq
        if "k" in s:
            s["kv"] = xq.xq_kv_cache(s["k"], s["v"], s.get("k_scale", 1.0), s.get("v_scale", 1.0))
        if case["op"] == "rope":
            s["rope"] = xq.xq_rope_plan(s["freq"], s["sections"], s["pairs"] == "adjacent")
        need = 0
        if case["op"] == "decode":
            need = xq.xq_attn_decode_workspace_bytes(case["seqs"], case["heads"], s["kv"], case["longest"],
                                                     case["window"], case["sinks"])
        elif case["op"] == "pages" and case["what"] != "copy":
            need = xq.xq_cache_workspace_bytes(case["pages"], case["slots"])
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
    if op == "prefill":
        xq.xq_attn_prefill(s["out"], s["q"], s["kv"], s["tables"], s["lens"], s["starts"], s["most"], s["scale"],
                           window=s["window"], sinks=s["sinks"])
        return s["out"]
    if op == "rope":
        if s["back"]:
            xq.xq_rope(s["out"], s["x"], s["pos"], s["rope"], inverse=True)
            return s["out"]
        H, K = s["heads"], s["kv_heads"]
        x = s["qkv"]
        xq.xq_rope_append(s["out"], s["kv"], x[:, :H], x[:, H:H + K], x[:, H + K:], s["pos"], s["rope"], s["slots"])
        return s["out"], s["k"], s["v"]
    if s["what"] == "copy":
        xq.xq_cache_copy(s["kv"], s["src"], s["dst"])
        return s["k"], s["v"]
    if s["what"] == "beams":
        xq.xq_cache_free(s["kv"], s["refs"], s["tables"], s["lens"], s["children"])
        xq.xq_cache_fork(s["kv"], s["refs"], s["tables"], s["lens"], s["parents"], s["children"], s["status"],
                         workspace=s["ws"])
    else:
        s["refs"].copy_(s["refs0"])
        s["tables"].copy_(s["tables0"])
        xq.xq_cache_compact(s["kv"], s["refs"], s["tables"], s["status"], workspace=s["ws"])
    return s["k"], s["v"], s["refs"], s["tables"], s["lens"], s["status"]


# ---------------------------------------------------------------- plain forms

def _gathered(s, name):
    """[seqs, kv_heads, length, dim] in 32 bits through the table."""
    rows = s["tables"].long().clamp(min=0)
    x = s[name].view(torch.uint8) if s["cache"] == "e4m3" else s[name]
    x = x[rows]
    x = (x.view(TYPES["e4m3"]) if s["cache"] == "e4m3" else x).float()
    x = x.transpose(1, 2).reshape(len(rows), s["kv_heads"], -1, s["dim"])
    return x * s[name + "_scale"] if s["cache"] == "e4m3" else x


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


def _plain_prefill(s):
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


def _angles(s):
    axis = torch.repeat_interleave(torch.arange(s["axes"], device=DEV),
                                   torch.tensor(s["sections"], device=DEV), output_size=s["rot"] // 2)
    a = s["pos"].double()[axis].t() * s["freq"]                          # far positions need 64 bits
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _rotated(s, x, cos, sin):
    x, r = x.float(), s["rot"]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if s["pairs"] == "adjacent" else (x[..., :r // 2], x[..., r // 2:r])
    y, z = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((y, z), -1).flatten(-2) if s["pairs"] == "adjacent" else torch.cat((y, z), -1)
    return torch.cat((turned, x[..., r:]), -1)


def _stored(s, x, scale):
    if s["cache"] == "e4m3":
        return (x / scale).clamp(-448, 448).to(TYPES["e4m3"]).view(torch.uint8)
    return x.to(TYPES[s["cache"]])


def _plain_rope(s):
    cos, sin = _angles(s)
    if s["back"]:
        return _rotated(s, s["x"], cos, -sin).to(TYPES[s["io"]])
    H, K = s["heads"], s["kv_heads"]
    x = s["qkv"]
    out = _rotated(s, x[:, :H], cos, sin).to(TYPES[s["io"]])
    at, slot = s["slots"] // s["page"], s["slots"] % s["page"]
    k, v = (s["k"].view(torch.uint8), s["v"].view(torch.uint8)) if s["cache"] == "e4m3" else (s["k"], s["v"])
    k[at, :, slot] = _stored(s, _rotated(s, x[:, H:H + K], cos, sin), s["k_scale"])
    v[at, :, slot] = _stored(s, x[:, H + K:].float(), s["v_scale"])
    return out, s["k"], s["v"]


def _move(s, src, dst):
    for name in ("k", "v"):                                              # 8-bit values move as their bytes
        x = s[name].view(torch.uint8) if s["cache"] == "e4m3" else s[name]
        x[:, dst] = x[:, src]


def _plain_pages(s):
    if s["what"] == "copy":
        _move(s, s["src"].long(), s["dst"].long())
        return s["k"], s["v"]
    refs, tables, lens, page = s["refs"], s["tables"], s["lens"], s["page"]
    if s["what"] == "beams":
        kids, parents = s["children"].long(), s["parents"].long()
        old = tables[kids].flatten()
        refs.index_add_(0, old.clamp(min=0).long(), -(old >= 0).int())
        n = lens[parents]
        full, part = n // page, n % page > 0
        free = torch.argsort((refs != 0).int(), stable=True)
        new = free[(part.long().cumsum(0) - 1).clamp(min=0)]
        column = torch.arange(tables.shape[1], device=DEV)
        rows = tables[parents]
        last = rows.gather(1, full.long().clamp(max=tables.shape[1] - 1)[:, None])[:, 0].clamp(min=0).long()
        shared = column < full[:, None]
        tail = (column == full[:, None]) & part[:, None]
        refs.index_add_(0, rows.clamp(min=0).flatten().long(), shared.flatten().int())
        refs.index_add_(0, new, part.int())
        tables[kids] = torch.where(shared, rows, torch.where(tail, new[:, None].int(), -1))
        lens[kids] = n
        _move(s, last[part], new[part])                                 # a full last page is shared, not copied
        s["status"].zero_()
    else:
        refs.copy_(s["refs0"])
        tables.copy_(s["tables0"])
        live = refs > 0
        count = live.sum()
        i = torch.arange(s["pages"], device=DEV)
        src = torch.nonzero(live & (i >= count))[:, 0]
        dst = torch.nonzero(~live & (i < count))[:, 0]
        _move(s, src, dst)
        to = i.int()
        to[src] = dst.int()
        tables.copy_(torch.where(tables >= 0, to[tables.clamp(min=0).long()], tables))
        refs[dst] = refs[src]
        refs[src] = 0
        s["status"].copy_(torch.stack((torch.zeros_like(count), count)))
    return s["k"], s["v"], refs, tables, lens, s["status"]


def run(state):
    if own:
        return _own(state)
    return {"decode": _plain_decode, "prefill": _plain_prefill, "rope": _plain_rope, "pages": _plain_pages}[
        state["op"]](state)


# ---------------------------------------------------------------- 64 bits, apart from the plain forms

def _rows64(s, name, b, where):
    """Tokens `where` of sequence b, [tokens, kv_heads, dim]."""
    page = s["tables"][b].long()[where // s["page"]]
    x = s[name].double() if s[name].numel() < 1 << 26 else None
    if x is None:
        raw = s[name].view(torch.uint8) if s["cache"] == "e4m3" else s[name]
        got = raw[page, :, where % s["page"]]
        got = (got.contiguous().view(TYPES["e4m3"]) if s["cache"] == "e4m3" else got).double()
    else:
        got = x[page, :, where % s["page"]]
    return got * s[name + "_scale"]


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


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "decode":
        return torch.cat([_attend64(s, s["q"][b:b + 1], s["lens"][b:b + 1].long() - 1, b, n)
                          for b, n in enumerate(s["host_lens"])])
    if case["op"] == "prefill":
        out = []
        for b, n in enumerate(s["host_lens"]):
            first, end = s["host_starts"][b:b + 2]
            for at in range(first, end, 1024):
                to = min(end, at + 1024)
                pos = torch.arange(n - end + at, n - end + to, device=DEV)
                out.append(_attend64(s, s["q"][at:to], pos, b, n - end + to))
        return torch.cat(out)
    if case["op"] == "rope":
        half, turn = case["rot"] // 2, []
        for axis, count in enumerate(s["sections"]):
            i = len(turn)
            turn += [s["pos"][axis].double() * s["freq"][i + j] for j in range(count)]
        turn = torch.stack(turn, 1)
        turn = torch.complex(turn.cos(), turn.sin())
        if case["back"]:
            turn = turn.conj()

        def rotate(x):
            x = x.double().clone()
            even = torch.arange(half, device=DEV) * (2 if case["pairs"] == "adjacent" else 1)
            odd = even + (1 if case["pairs"] == "adjacent" else half)
            z = torch.complex(x[..., even], x[..., odd]) * turn[:, None]
            x[..., even], x[..., odd] = z.real, z.imag
            return x

        if case["back"]:
            return rotate(s["x"])
        H, K = case["heads"], case["kv_heads"]
        k, v = s["k"].double(), s["v"].double()
        page, slot = s["slots"] // case["page"], s["slots"] % case["page"]
        k[page, :, slot] = rotate(s["qkv"][:, H:H + K]) / s["k_scale"]
        v[page, :, slot] = s["qkv"][:, H + K:].double() / s["v_scale"]
        return rotate(s["qkv"][:, :H]), k, v
    return None                                                          # pages: nothing is computed, bytes move


# ---------------------------------------------------------------- work

def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
    if case["op"] in ("decode", "prefill"):
        lens = _lengths(case["seqs"], case["longest"])
        H, K, D, w, sinks = case["heads"], case["kv_heads"], case["dim"], case["window"], case["sinks"]

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
        return {"bytes": 2 * sum(touched) * K * D * size[case["cache"]] + 2 * rows * H * D * size[case["io"]],
                "flops": 4 * pairs * H * D}
    if case["op"] == "rope":
        T, H, K, D = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        n = T * H * D * (size[case["src"]] + size[case["io"]])
        if not case["back"]:
            n += 2 * T * K * D * (size[case["src"]] + size[case["cache"]]) + 8 * T
        return {"bytes": n + 4 * case["axes"] * T, "flops": 3 * T * (H + (0 if case["back"] else K)) * case["rot"]}
    one = 2 * case["layers"] * case["kv_heads"] * case["page"] * case["dim"] * size[case["cache"]]
    width = -(-case["longest"] // case["page"]) + 1
    meta = 4 * (case["pages"] + case["slots"] * width)
    if case["what"] == "copy":
        return {"bytes": 2 * (case["pages"] // 2) * one, "flops": 0}
    if case["what"] == "beams":
        return {"bytes": 2 * (case["slots"] // 2) * one + meta, "flops": 0}
    # of the live pages, as many lie above the live count as a shuffled pool has there
    used = _filled(case)[1]
    moved = used * (case["pages"] - used) / case["pages"]
    return {"bytes": 2 * moved * one + 2 * meta, "flops": 0}
