"""The example's attention layer: what its calls leave in the cache and in the
outputs is attention of the layer's own queries, keys and values, through
prompts, single tokens, forks and a compaction."""
import importlib.util
import os

import pytest
import torch

import kv_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_layer.py")
    spec = importlib.util.spec_from_file_location("attention_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _check(layer, out, q, rows, io):
    """out and q [tokens, heads, dim]; rows: (slot, position) of each token."""
    tables, lens = layer.tables.clone(), layer.lens.tolist()
    for t, (slot, pos) in enumerate(rows):
        n = lens[slot]
        k, there = ref.rows_of(layer.kv.k, tables[slot], n, layer.page)
        v, _ = ref.rows_of(layer.kv.v, tables[slot], n, layer.page)
        want, mag, slack = ref.attend(q[t:t + 1], k, v, there, torch.tensor([pos], device=DEV), layer.scale,
                                      layer.window, layer.sinks)
        weight = 2.0 ** -8 if io == "bf16" else 2.0 ** -24
        tol = ref.attend_tolerance(want, mag, slack, io, weight, n)
        assert ((out[t:t + 1].double() - want).abs() <= tol).all(), (slot, pos)


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
def test_layer(window, sinks):
    layer = _example().Layer(window=window, sinks=sinks)
    g = torch.Generator(device=DEV).manual_seed(3)
    draw = lambda n: torch.randn(n, layer.hidden, device=DEV, generator=g)
    y, out, q = layer.prompt(draw(103), [(0, 70), (1, 33)])
    _check(layer, out, q, [(0, p) for p in range(70)] + [(1, p) for p in range(33)], "bf16")
    for _ in range(2):
        y, out, q = layer.step(draw(2), [0, 1])
        _check(layer, out, q, [(0, layer.lens[0].item() - 1), (1, layer.lens[1].item() - 1)], "f32")
    layer.fork([0, 0], [2, 3])
    assert layer.status.tolist() == [0, 0] and layer.lens.tolist() == [72, 35, 72, 72]
    y, out, q = layer.step(draw(4), [0, 1, 2, 3])
    _check(layer, out, q, [(s, layer.lens[s].item() - 1) for s in range(4)], "f32")
    layer.fork([3], [1])
    layer.compact()
    live = layer.status.tolist()[1]
    assert layer.refs[:live].min() > 0 and (layer.refs[live:] == 0).all()
    y, out, q = layer.step(draw(4), [0, 1, 2, 3])
    _check(layer, out, q, [(s, layer.lens[s].item() - 1) for s in range(4)], "f32")
    assert y.isfinite().all()
