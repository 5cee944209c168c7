"""The 4-bit cache's format in 64 bits, written from include/xq.h without the library."""
import torch

import kv_reference as ref

SIZES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def exp_row(dim):
    return 4 if dim <= 128 else 8


def encode(x):
    """[..., dim] in 64 bits -> codes [..., dim / 2], powers [..., dim / 32] as bytes."""
    b = x.unflatten(-1, (-1, 32))
    nan = b.isnan().any(-1)
    top = b.abs().amax(-1).nan_to_num(nan=0.0, posinf=1e300)
    e, power = torch.full_like(top, -23.0), torch.full_like(top, 2.0 ** -23)  # (doubled: pow is not exact)
    for _ in range(36):
        up = top >= 7 * power
        e, power = torch.where(up, e + 1, e), torch.where(up, 2 * power, power)
    u = b.abs().nan_to_num(nan=0.0, posinf=1e300) / power[..., None]
    sizes = torch.tensor(SIZES, dtype=torch.float64, device=x.device)
    middle = (sizes[1:] + sizes[:-1]) / 2
    code = torch.bucketize(u, middle)                       # a middle itself goes to the lower code
    on = (u == middle[code.clamp(max=6)]) & (code < 7) & (code % 2 == 1)
    code = code + on.long()                                 # ... and to the upper one where that is even
    code = (code + 8 * torch.signbit(b).long()).flatten(-2).to(torch.uint8)
    power = torch.where(nan, 255.0, e + 127).to(torch.uint8)
    return code[..., 0::2] + 16 * code[..., 1::2], power, nan


def values(codes, powers):
    """codes [..., dim / 2], powers [..., >= dim / 32] -> [..., dim] in 64 bits."""
    c = torch.stack((codes % 16, codes // 16), -1).flatten(-2).long()
    sizes = torch.tensor(SIZES, dtype=torch.float64, device=codes.device)
    x = sizes[c % 8] * torch.where(c >= 8, -1.0, 1.0)
    n = x.shape[-1] // 32
    p = powers[..., :n]
    powers_of_two = torch.tensor([2.0 ** (i - 127) for i in range(255)] + [torch.nan], dtype=torch.float64, device=codes.device)
    scale = powers_of_two[p.long()]
    return (x.unflatten(-1, (n, 32)) * scale[..., None]).flatten(-2)


def pool(pages, heads, page, dim, order, g, dev, layers=()):
    """Random rows as the append would store them: codes, powers (uint8), [*layers, pages, heads, page, .]."""
    front = (heads, page) if order == "hnd" else (page, heads)
    x = torch.randn(*layers, pages, *front, dim, device=dev, generator=g, dtype=torch.float64)
    codes, powers, _ = encode(x)
    exps = torch.randint(0, 256, (*powers.shape[:-1], exp_row(dim)), device=dev, generator=g, dtype=torch.int32).to(torch.uint8)
    exps[..., :powers.shape[-1]] = powers                   # what is behind a row's powers means nothing
    return (codes.transpose(-3, -2), exps.transpose(-3, -2)) if order == "nhd" else (codes, exps)


def cache(xq, k, k_exp, v, v_exp, scales):
    four, eight = torch.float4_e2m1fn_x2, torch.float8_e8m0fnu
    return xq.xq_kv_cache(k.view(four), v.view(four), *scales, k_exp=k_exp.view(eight), v_exp=v_exp.view(eight))


def rows_of(codes, exps, table, n, page):
    """Tokens 0..n-1 of one sequence, [n, heads, dim] in 64 bits, and which of them are there."""
    j = torch.arange(n, device=codes.device)
    p = table.long()[j // page]
    there = (p >= 0) & (p < codes.shape[0])
    at = p.clamp(0, codes.shape[0] - 1)
    return values(codes[at, :, j % page], exps[at, :, j % page]), there


def attend(s, rows, b, pos, n, window, sinks):
    k, there = rows_of(s["k"], s["k_exp"], s["table"][b], n, s["page"])
    v, _ = rows_of(s["v"], s["v_exp"], s["table"][b], n, s["page"])
    return ref.attend(s["q"][rows], k * s["scales"][0], v * s["scales"][1], there, pos, s["scale"], window, sinks)
