"""Single-token attention of many sequences: more than a wave adds up at once
in the shared plan, and more units than that plan takes."""
import random

import pytest
import torch

import quantized_decode_mat_amd as xq
from test_gpu_kv_attention import _device, check_decode, decode, setup  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs,heads,kv_heads,dim,cache,io,window,sinks,longest,shared", [
    (130, 6, 2, 64, "bf16", "f32", 0, 0, 1500, True),
    (65, 4, 1, 128, "e4m3", "bf16", 700, 5, 1500, True),
    (64, 8, 4, 128, "f16", "f16", 0, 0, 900, True),
    (200, 1, 1, 256, "f16", "f32", 0, 0, 700, True),
    # 3 units for each of 256 workgroups (512 for 64 dims) end the sharing, and so do three steps (a window of 300)
    (400, 4, 2, 64, "bf16", "bf16", 0, 0, 800, True),
    (800, 1, 1, 128, "e4m3", "f16", 300, 2, 700, False),
    (400, 4, 2, 128, "bf16", "bf16", 0, 0, 800, False),
    (768, 1, 1, 256, "e4m3", "f16", 300, 2, 700, False),
])
def test_decode(seqs, heads, kv_heads, dim, cache, io, window, sinks, longest, shared):
    rng = random.Random(seqs)
    lens = [rng.choice([0, 1, 127, 128, 129, rng.randint(2, longest), longest // 8]) for _ in range(seqs)]
    lens[seqs // 2] = longest
    s = setup(lens, heads, kv_heads, dim, 16, cache, io, "hnd")
    need = xq.xq_attn_decode_workspace_bytes(seqs, heads, s["kv"], longest, window, sinks)
    assert (need > 0) == shared
    ws = decode(s, window, sinks, longest)
    check_decode(s, lens, window, sinks, "decode")
    if ws is not None:
        assert not ws[:96 * 1024].any(), "arrival counters left standing"
    first = s["out"].clone()
    decode(s, window, sinks, longest, ws)
    assert torch.equal(s["out"], first), "the same call gave other bits"


def test_no_tokens_at_all():
    s = setup([0] * 70, 4, 2, 64, 16, "bf16", "f32", "hnd")
    decode(s, 0, 0, 4096)
    torch.cuda.synchronize()
    assert (s["out"] == 0).all()
