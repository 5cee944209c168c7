"""The paged cache's operators in 64 bits, and the tests' inputs. Written from
the formulas in include/xq.h, without the library."""
import math

import torch

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


def half_step(kind: str) -> float:
    """Largest relative error of one rounding to the type."""
    return {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11, "e4m3": 2.0 ** -4}[kind]


def smallest(kind: str) -> float:
    """Half the type's smallest positive value: a rounding's absolute error next to zero."""
    return {"f32": 2.0 ** -150, "bf16": 2.0 ** -134, "f16": 2.0 ** -25, "e4m3": 2.0 ** -10}[kind]


def pool(pages, heads, page, dim, kind, order, g, dev, layers=None):
    shape = (pages, page, heads, dim) if order == "nhd" else (pages, heads, page, dim)
    if layers:
        shape = (layers, *shape)
    x = torch.randn(shape, device=dev, generator=g).to(TYPES[kind])
    return x.transpose(-3, -2) if order == "nhd" else x


def as_f64(x):
    if x.dtype == torch.float8_e4m3fn:
        x = x.to(torch.float32)
    return x.double()


def rows_of(cache, table, n, page):
    """Tokens 0..n-1 of one sequence, [n, heads, dim] in 64 bits, and which of them are there."""
    pages = cache.shape[0]
    j = torch.arange(n, device=cache.device)
    p = table.long()[j // page]
    there = (p >= 0) & (p < pages)
    raw = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
    x = raw[p.clamp(0, pages - 1), :, j % page]
    if cache.dtype == torch.float8_e4m3fn:
        x = x.contiguous().view(torch.float8_e4m3fn)
    return as_f64(x), there


def attend(q, k, v, there, pos, scale, window, sinks):
    """q [rows, heads, dim] at positions pos over tokens k, v [n, kv_heads, dim] (64 bits, scales in).
    Returns the outputs, the sum of their terms' magnitudes, and the error that a row's scores may
    have relative to f32's half step (dim + 4 roundings of terms of that magnitude)."""
    rows, heads, dim = q.shape
    n, kv_heads = k.shape[:2]
    out = torch.zeros(rows, heads, dim, dtype=torch.float64, device=q.device)
    mag, slack = out.clone(), torch.zeros(rows, heads, 1, dtype=torch.float64, device=q.device)
    if n == 0:
        return out, mag, slack
    j = torch.arange(n, device=q.device)
    sees = there[None] & (j[None] <= pos[:, None])
    if window:
        sees &= (j[None] > pos[:, None] - window) | (j[None] < sinks)
    for h in range(heads):
        kh, vh = k[:, h // (heads // kv_heads)].contiguous(), v[:, h // (heads // kv_heads)].contiguous()
        qh = q[:, h].double()
        s = (torch.mm(qh, kh.t().contiguous()) * scale).masked_fill(~sees, -math.inf)
        top = s.amax(1, keepdim=True)
        p = torch.exp(s - torch.where(top > -math.inf, top, torch.zeros_like(top)))
        p = p.masked_fill(~sees, 0.0)
        p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
        clean = torch.where(sees.any(0)[:, None], vh, torch.zeros_like(vh))
        out[:, h] = torch.mm(p, clean)
        mag[:, h] = torch.mm(p, clean.abs())
        seen = torch.where(sees.any(0)[:, None], kh, torch.zeros_like(kh)).abs()
        worst = (torch.mm(qh.abs(), seen.t().contiguous()) * abs(scale)).masked_fill(~sees, 0.0).amax(1)
        slack[:, h, 0] = worst * (dim + 4)
    return out, mag, slack


def attend_tolerance(out, mag, slack, kind, weight_error, n):
    """One rounding of the result; the weights' error (their rounding, and exp of the scores' error,
    twice: numerator and sum); a chain of n/16 partial sums with their rescalings, in f32."""
    f = 2.0 ** -24
    return (half_step(kind) * out.abs() + smallest(kind)
            + mag * 1.01 * (weight_error + 2 * f * slack + (n / 8 + 64) * f))


def rotate(x, pos, freq, sections, adjacent, inverse):
    """x [tokens, heads, dim] in 64 bits."""
    half = freq.numel()
    axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections)).to(pos.device)
    angle = pos.double()[axis].t() * freq
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    if inverse:
        s = -s
    y = x.double().clone()
    if adjacent:
        a, b = x[..., 0:2 * half:2].double(), x[..., 1:2 * half:2].double()
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., :half].double(), x[..., half:2 * half].double()
        y[..., :half], y[..., half:2 * half] = a * c - b * s, a * s + b * c
    return y


def rotate_tolerance(x, y, kind, dim_half, adjacent, angle_max):
    """One rounding to the type; sine and cosine to 3 half steps of 1 (two roundings and the reduced
    angle's), two products and a sum (3 half steps), each of |a| + |b|; the angle's own rounding in
    64 bits."""
    z = x.double().abs()
    pair = z.clone()
    if adjacent:
        both = z[..., 0:2 * dim_half:2] + z[..., 1:2 * dim_half:2]
        pair[..., 0:2 * dim_half:2] = both
        pair[..., 1:2 * dim_half:2] = both
    else:
        both = z[..., :dim_half] + z[..., dim_half:2 * dim_half]
        pair[..., :dim_half] = both
        pair[..., dim_half:2 * dim_half] = both
    return half_step(kind) * y.abs() + smallest(kind) + 1.01 * pair * (6 * 2.0 ** -24 + angle_max * 2.0 ** -52)


class Pages:
    """The pages' bookkeeping, one step at a time on the host."""

    def __init__(self, refs, tables, lens, page):
        self.refs, self.tables, self.lens, self.page = list(refs), [list(r) for r in tables], list(lens), page
        self.copies = []

    def free(self, rows):
        for r in rows:
            if not 0 <= r < len(self.lens):
                continue
            for p in self.tables[r]:
                if 0 <= p < len(self.refs):
                    self.refs[p] -= 1
            self.tables[r] = [-1] * len(self.tables[r])
            self.lens[r] = 0

    def fork(self, parents, children):
        slots, width, pages = len(self.lens), len(self.tables[0]), len(self.refs)
        old_t, old_l = [list(r) for r in self.tables], list(self.lens)
        free = [p for p in range(pages) if self.refs[p] == 0]
        refused, lacking, named = 0, 0, set()
        for p, c in zip(parents, children):
            ok = 0 <= c < slots and c not in named
            if 0 <= c < slots:
                named.add(c)
            ok = ok and 0 <= p < slots and old_l[c] == 0 and old_l[p] >= 0
            need = -(-old_l[p] // self.page) if ok else 0
            if not ok or need > width or any(not 0 <= x < pages for x in old_t[p][:need]):
                refused += 1
                continue
            n, full = old_l[p], old_l[p] // self.page
            row = old_t[p][:full]
            if n % self.page:
                if not free:
                    refused += 1
                    lacking += 1
                    continue
                new = free.pop(0)
                self.refs[new] = 1
                self.copies.append((old_t[p][full], new))
                row = row + [new]
            for x in row[:full]:
                self.refs[x] += 1
            self.tables[c] = row + [-1] * (width - len(row))
            self.lens[c] = n
        return [refused, lacking]

    def compact(self):
        pages = len(self.refs)
        live = sum(r > 0 for r in self.refs)
        src = [p for p in range(live, pages) if self.refs[p] > 0]
        dst = [p for p in range(live) if self.refs[p] <= 0]
        to = {s: d for s, d in zip(src, dst)}
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
            self.copies.append((s, d))
        self.tables = [[to.get(p, p) for p in r] for r in self.tables]
        return [0, live]
