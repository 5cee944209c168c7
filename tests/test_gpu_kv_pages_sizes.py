"""The pages' lists on either side of the sizes up to which one launch keeps
them on the chip: 1024 forks of 4096 rows, 8192 pages."""
import random

import pytest
import torch

import kv_reference as ref
import quantized_decode_mat_amd as xq
from test_gpu_kv_rope_pages import DEV, Device, _device, cache, filled, raw  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages,slots,forks", [(8192, 2048, 1024), (8193, 2050, 1025), (20000, 4096, 1000),
                                               (20000, 4097, 1000), (9000, 64, 30), (1, 2, 1), (8191, 3000, 700)])
def test_fork_and_compact(pages, slots, forks):
    rng = random.Random(pages + slots)
    kv, k, v = cache(1, pages, 1, 2, 16, "bf16", "hnd")
    rows = slots - forks
    refs, tables, lens = filled(rng, pages, 2, slots, 5, rows)
    d, m = Device(refs, tables, lens), ref.Pages(refs, tables, lens, 2)
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    pairs = [(x, raw(x).clone()) for x in (k, v)]
    kids = list(range(rows, slots))
    rng.shuffle(kids)
    parents = [rng.randrange(rows) for _ in kids]
    want = m.fork(parents, kids)
    xq.xq_cache_fork(kv, d.refs, d.tables, d.lens, t(parents), t(kids), d.status, workspace=d.ws)
    d.check(m, pairs)
    assert d.status.tolist() == want
    gone = rng.sample(range(slots), slots // 2)
    m.free(gone)
    xq.xq_cache_free(kv, d.refs, d.tables, d.lens, t(gone))
    pairs, m.copies = [(x, raw(x).clone()) for x in (k, v)], []
    want = m.compact()
    xq.xq_cache_compact(kv, d.refs, d.tables, d.status, workspace=d.ws)
    d.check(m, pairs)
    assert d.status.tolist() == want


@pytest.mark.parametrize("pages", [8192, 8193])
def test_compact_every_page_in_use_or_none(pages):
    kv, k, v = cache(1, pages, 1, 1, 16, "bf16", "hnd")
    for used in (0, pages, pages // 2):
        # the last `used` pages, one row each of up to four
        refs = [0] * (pages - used) + [1] * used
        tables = [[pages - 1 - 4 * r - i if 4 * r + i < used else -1 for i in range(4)] for r in range(pages // 4 + 1)]
        lens = [sum(p >= 0 for p in row) for row in tables]
        d, m = Device(refs, tables, lens), ref.Pages(refs, tables, lens, 1)
        pairs = [(x, raw(x).clone()) for x in (k, v)]
        want = m.compact()
        xq.xq_cache_compact(kv, d.refs, d.tables, d.status, workspace=d.ws)
        d.check(m, pairs)
        assert d.status.tolist() == want == [0, used]
