"""Edges of the paged cache's calls: what lies beside a row, scales of zero,
small weights, starts that do not fit, sizes past a launch's."""
import pytest
import torch

import kv_reference as ref
import quantized_decode_mat_amd as xq
import workloads as wl
from test_gpu_kv_attention import _device, check_decode, check_prefill, compare, decode, expect, prefill, setup  # noqa: F401
from test_gpu_kv_prefill_large import copies
from test_gpu_kv_rope_pages import check_rope, freqs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def beside(s, fill):
    """The same cache as slices of rows of 256, with `fill` in what is beside them."""
    kv = []
    for x in (s["k"], s["v"]):
        wide = torch.full((*x.shape[:3], 256), fill, device=DEV).to(x.dtype)
        wide[..., :x.shape[3]] = x
        kv.append(wide[..., :x.shape[3]])
    return dict(s, k=kv[0], v=kv[1], kv=xq.xq_kv_cache(*kv, *s["scales"]))


@pytest.mark.parametrize("cache,io", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "f16")])
@pytest.mark.parametrize("dim", [176, 192])
def test_what_lies_beside_a_row_has_no_influence(cache, io, dim):
    lens = [517, 90, 3]
    s = setup(lens, 6, 2, dim, 16, cache, io, "hnd", poison=False)
    results = []
    for fill in (0.0, float("nan")):
        t = beside(s, fill)
        decode(t, 0, 0, 517)
        check_decode(t, lens, 0, 0, "decode")
        results.append(t["out"].clone())
        prefill(t, [1, 1, 1], 0, 0)
        check_prefill(t, lens, [1, 1, 1], [0, 1, 2, 3], 0, 0, "single rows")
        results.append(t["out"].clone())
    assert torch.equal(results[0], results[2]) and torch.equal(results[1], results[3])


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("cache,io,scale,k_scale", [("bf16", "bf16", 0.0, 1.0), ("f16", "f16", 0.0, 1.0),
                                                   ("e4m3", "bf16", 0.0, 0.75), ("e4m3", "f16", 1e-30, 1e-20),
                                                   ("bf16", "bf16", 1e-39, 1.0), ("f16", "f16", -1e-39, 1.0)])
def test_scale_of_zero(cache, io, scale, k_scale, many):
    """Every visible token weighs the same."""
    n = copies([64, 129], 4, 2) if many else 1
    lens, chunks = [300, 129] * n, [64, 129] * n
    s = setup(lens, 4, 2, 80, 16, cache, io, "hnd", rows=193 * n)
    s["scale"], s["scales"] = scale, (k_scale, s["scales"][1])
    s["kv"] = xq.xq_kv_cache(s["k"], s["v"], *s["scales"])
    starts = prefill(s, chunks, 50, 2)
    check_prefill(s, lens, chunks, starts, 50, 2, "scale of zero")


def test_rope_of_more_tokens_than_a_launch_has_threads():
    tokens, plan = (1 << 26) + 5, xq.xq_rope_plan(freqs(8), [4])
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(1 << 20, 1, 8, device=DEV, generator=g).to(torch.bfloat16).repeat(65, 1, 1)[:tokens]
    pos = torch.arange(tokens, dtype=torch.int32, device=DEV)
    out = torch.zeros_like(x)
    xq.xq_rope(out, x, pos, plan)
    torch.cuda.synchronize()
    for at in (0, 1 << 22, 1 << 24, 1 << 25, tokens - 40):
        part = slice(at, at + 40)
        check_rope(out[part], x[part], pos[None, part], plan, [4], False, False, "bf16")
    assert (out.view(-1, 8) != 0).any(-1).all()


def test_append_of_more_tokens_than_a_launch_has_workgroups():
    """One row of q, k and v for all tokens; each has its own position and slot."""
    tokens, heads, dim, page = (1 << 24) + 5, 4, 256, 64
    plan = xq.xq_rope_plan(freqs(32), [16])
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(1, heads + 2, dim, device=DEV, generator=g).expand(tokens, -1, -1)
    pages = -(-tokens // page)
    k, v = (torch.zeros(pages, 1, page, dim, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2))
    pos = torch.arange(tokens, dtype=torch.int32, device=DEV)
    slots = torch.arange(tokens - 1, -1, -1, device=DEV)
    out = torch.zeros(tokens, heads, dim, dtype=torch.bfloat16, device=DEV)
    xq.xq_rope_append(out, xq.xq_kv_cache(k, v, 0.05, 0.04), x[:, :heads], x[:, heads:heads + 1], x[:, heads + 1:], pos,
                      plan, slots)
    torch.cuda.synchronize()
    for at in (0, (1 << 23) - 20, 1 << 23, tokens - 40):
        part = slice(at, at + 40)
        check_rope(out[part], x[part, :heads], pos[None, part], plan, [16], False, False, "bf16")
        page_of, place = slots[part] // page, slots[part] % page
        check_rope(k.view(torch.uint8)[page_of, :, place].view(k.dtype), x[part, heads:heads + 1], pos[None, part], plan,
                   [16], False, False, "e4m3", 0.05)
        want = (x[part, heads + 1:] / 0.04).to(k.dtype)
        assert torch.equal(v.view(torch.uint8)[page_of, :, place], want.view(torch.uint8))


@pytest.mark.parametrize("N", [196608, 200704, 1 << 19])
@pytest.mark.parametrize("between", ["decode", "fork"])
def test_one_workspace_for_calls_with_counters(between, N):
    """Counters past 96 KiB would meet the other calls' lists and partial results."""
    K = 256
    w = torch.from_numpy(wl.q4k_weights(N, K, wl.rng(1)).reshape(-1)).to(DEV)
    x = torch.empty(xq.xq_q8k_bytes(1, K), dtype=torch.uint8, device=DEV)
    xq.xq_quantize_q8k(x, torch.randn(1, K, device=DEV), 1, K)
    s = setup([3000], 8, 2, 128, 16, "bf16", "f32", "hnd")
    refs, status = torch.zeros(s["k"].shape[0], dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    tables, lens = torch.full((30000, 4), -1, dtype=torch.int32, device=DEV), torch.zeros(30000, dtype=torch.int32, device=DEV)
    ids = torch.arange(10000, dtype=torch.int32, device=DEV)
    need = max(xq.xq_gemv_q4k_q8k_workspace_bytes(N), xq.xq_attn_decode_workspace_bytes(1, 8, s["kv"], 3000),
               xq.xq_cache_workspace_bytes(s["k"].shape[0], 30000))
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    y, yq = torch.empty(N, device=DEV), torch.empty(xq.xq_q8k_bytes(1, N), dtype=torch.uint8, device=DEV)
    want = torch.empty_like(yq)
    for _ in range(3):
        yq.fill_(0xa5)
        xq.xq_gemv_q4k_q8k(y, yq, w, x, N, K, workspace=ws)
        xq.xq_quantize_q8k(want, y, 1, N)
        torch.cuda.synchronize()
        assert torch.equal(yq.view(-1, 320)[:, :292], want.view(-1, 320)[:, :292])
        if between == "decode":
            decode(s, 0, 0, 3000, ws)
            check_decode(s, [3000], 0, 0, "decode")
        else:
            xq.xq_cache_fork(s["kv"], refs, tables, lens, ids, ids + 10000, status, workspace=ws)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("starts,most,window", [([3, 63], 25, 0), ([3, 63], 25, 20), ([-5, 40], 100, 0), ([20, 2000], 100, 0),
                                                ([20, 2 ** 31 - 1], 100, 30), ([-2 ** 31, 2 ** 31 - 1], 100, 30), ([90, 115], 100, 6)])
def test_rows_that_are_left_out_move_no_others(starts, most, window, many):
    """Row i of a chunk of c has position n - c + i whatever part of the chunk is done."""
    rows, n, seqs = 100, 90, 1 if not many else 300
    s = setup([n] * seqs, 4, 2, 64, 16, "bf16", "bf16", "hnd", rows=rows)
    # the sequences of the larger call have no rows but for the first
    s["starts"] = torch.tensor(starts + [starts[1]] * (seqs - 1), dtype=torch.int32, device=DEV)
    xq.xq_attn_prefill(s["out"], s["q"], s["kv"], s["table"], s["lens"], s["starts"], most, s["scale"], window=window, sinks=2)
    torch.cuda.synchronize()
    first = max(starts[0], 0)
    done = torch.arange(first, max(first, min(starts[1], rows, first + most)), device=DEV)
    pos = n - starts[1] + done
    assert len(done) and ((s["full"] != 7.0).any(-1).any(-1).nonzero()[:, 0] == done).all()
    want, mag, slack = expect(s, 0, slice(int(done[0]), int(done[-1]) + 1), pos, n, window, 2)
    compare(s, s["out"][done], want, mag, slack, ref.half_step("bf16"), n, "part of a chunk")


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("io", ["bf16", "f16"])
@pytest.mark.parametrize("strong", [5, 2000])
def test_many_small_weights(io, many, strong):
    """2047 tokens of 2^-26 the weight of one whose v is 0."""
    n = copies([64], 4, 2) if many else 1
    lens, chunks = [2048] * n, [64] * n
    s = setup(lens, 4, 2, 64, 16, io, io, "hnd", rows=64 * n, poison=False)
    s["q"].zero_(), s["k"].zero_()
    s["v"].copy_(s["v"].float().abs())
    s["q"][..., 0], s["scale"] = 1.0, 1.0
    page = s["table"][:, strong // 16].long()
    s["k"][page, :, strong % 16, 0], s["v"][page, :, strong % 16] = 18.0, 0.0
    starts = prefill(s, chunks, 0, 0)
    check_prefill(s, lens, chunks, starts, 0, 0, "small weights")


def test_tables_with_room_for_more_than_the_longest_length():
    """max_len, left out, is the tables' room; 2^30 tokens are the most a call takes."""
    s = setup([2000, 70], 4, 2, 64, 1024, "bf16", "f32", "hnd")
    wide = torch.full((2, (1 << 20) + 3), -1, dtype=torch.int32, device=DEV)
    wide[:, :s["table"].shape[1]] = s["table"]
    ws = torch.zeros(xq.xq_attn_decode_workspace_bytes(2, 4, s["kv"], 1 << 30), dtype=torch.uint8, device=DEV)
    xq.xq_attn_decode(s["out"], s["q"], s["kv"], wide, s["lens"], s["scale"], workspace=ws)
    check_decode(s, [2000, 70], 0, 0, "wide tables")
