"""The workspace that single-token attention over 4 bits asks for, to the byte, on the host: 96 KiB of counters, and for
each workgroup two partial results of its heads, a padded row of values and four floats each. A workgroup's step is 256
tokens; calls of up to three steps, and of units enough, share nothing and need none."""
import ctypes

import pytest

import quantized_decode_mat_amd as xq
from test_kv_four_gates import four

PAD = {32: 64, 64: 64, 96: 128, 128: 128, 160: 192, 192: 192, 224: 256, 256: 256}


def want(seqs, heads, kv_heads, dim, max_len, window, sinks):
    group, padded = heads // kv_heads, PAD[dim]
    units = kv_heads * -(-group // 16)                       # of a sequence
    seen = min(max_len, window + sinks) if window else max_len
    steps = -(-seen // 256)
    room = 256 * (2 if padded <= 128 else 1)                 # workgroups on the card at once
    if steps <= 3 or seqs * units >= 3 * room or units > room:
        return 0
    ranges = min(room // units, seqs * steps)
    return 96 * 1024 + units * ranges * 2 * min(16, group) * (padded + 4) * 4


@pytest.mark.parametrize("dim", sorted(PAD))
@pytest.mark.parametrize("heads,kv_heads", [(32, 8), (8, 8), (33, 1), (40, 2), (600, 600)])
@pytest.mark.parametrize("max_len,window,sinks", [(1, 0, 0), (700, 0, 0), (768, 0, 0), (769, 0, 0), (131072, 0, 0),
                                                  (131072, 700, 68), (131072, 700, 69), (300, 131072, 4)])
def test_workspace_to_the_byte(dim, heads, kv_heads, max_len, window, sinks):
    kv = four(dict(dim=dim, kv_heads=kv_heads))
    for seqs in (1, 2, 3, 47, 48, 95, 96, 191, 192, 500):
        got = xq.lib().xq_attn_decode_workspace_bytes(seqs, heads, ctypes.byref(kv), max_len, window, sinks)
        assert got == want(seqs, heads, kv_heads, dim, max_len, window, sinks), seqs
