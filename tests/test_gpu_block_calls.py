"""Ways to call the linear layers and the residual norm that other tests do not take: counts given once for all
ranks, one buffer for several inputs, ranks whose empty buffers have no address, a group's first call while a
graph is captured, and calls from several host threads."""
from __future__ import annotations

import threading

import pytest
import torch

from gpu_util import group
from test_gpu_linear import WHICH, Layer, like, workspace
from test_gpu_residual_norm import EPS, Rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dt():
    from same_device_collective_gb300 import dt as mod
    assert torch.cuda.is_available()
    return mod


def flat(v):
    return [t for u in v for t in flat(u)] if isinstance(v, (list, tuple)) else [v] if v is not None else []


def same(a, b):
    a, b = flat(a), flat(b)
    assert len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


def both(a, g, act):
    """Both passes of a layer."""
    if a.which == "gather_linear":
        return [a.forward(g, act), a.backward(g, act)]
    return [a.forward(g), a.backward(g)]


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("rows,dim,features", [(1, 512, 256), (20, 100, 33), (300, 520, 136)])
def test_layers_of_equal_pieces(dt, which, rows, dim, features):
    P = 3
    a = Layer(dt, which, [rows] * P, dim, [features] * P, seed=1)
    query, fwd, bwd = (getattr(dt, f"dt_{which}{s}") for s in ("_workspace", "", "_backward"))
    with group(P) as g:
        want = both(a, g, "silu")
        size = [query(g, None, rows, dim, None, features, "bf16", back) for back in (False, True)]
        assert size == [query(g, a.rows, 0, dim, a.features, 0, "bf16", back) for back in (False, True)]
        ws = torch.empty(max(size), dtype=torch.uint8, device="cuda")
        counts, dx, dw = (None, rows, dim, None, features, "bf16"), like(a.x), like(a.w)
        if which == "gather_linear":
            y, db = like(a.pre), like(a.b)
            pre = like(y)
            fwd(g, a.x, a.w, a.b, pre, y, *counts, "silu", ws)
            bwd(g, a.x, a.w, a.pre, a.dy, dx, dw, db, *counts, "silu", ws)
            same([(y, pre), (dx, dw, db)], want)
        else:
            y, db = like(a.res), torch.empty_like(a.b)
            fwd(g, a.x, a.w, a.b, a.res, y, *counts, ws)
            bwd(g, a.x, a.w, a.dy, dx, dw, db, *counts, ws)
            same([y, (dx, dw, db)], want)


@pytest.mark.parametrize("rows", [2, 200])
def test_norm_of_equal_pieces(dt, rows):
    a = Rows(dt, [rows] * 3, 264, "bf16", "f32", seed=1)
    with group(3) as g:
        want = [a.forward(g), a.backward(g)]
        y, z, dx, do = (a.like(a.x) for _ in range(4))
        r1, r2 = a.like(a.r1), a.like(a.r2)
        w = [torch.empty(264, device="cuda") for _ in range(3)]
        ws = torch.empty(dt.dt_residual_norm_workspace(g, 264), dtype=torch.uint8, device="cuda")
        dt.dt_residual_norm(g, a.x, a.branch, a.post, a.gate, a.pre, a.scale, y, z, r1, r2, None, rows, 264, EPS, "bf16", "f32")
        dt.dt_residual_norm_backward(g, a.branch, a.y, a.dy, a.dz, a.post, a.gate, a.pre, a.scale, a.r1, a.r2, dx, do, *w, None,
                                     rows, 264, "bf16", "f32", "sum", ws)
        same([(y, z, r1, r2), (dx, do, w)], want)


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("rows,dim,features", [(1, 512, 256), (16, 104, 40), (24, 512, 264), (300, 520, 136)])
def test_one_buffer_for_every_rank(dt, which, rows, dim, features):
    """Inputs may overlap: all ranks' tokens, weights and gradients are the first's.  (Against the definition:
    where ranks' rows follow one another in memory, as those of copies may, the sums' order is another.)"""
    a = Layer(dt, which, [rows] * 3, dim, [features] * 3, seed=2)
    for name in ("x", "w", "dy", "pre" if which == "gather_linear" else "res"):
        setattr(a, name, [getattr(a, name)[0]] * 3)
    with group(3) as g:
        forward, backward = both(a, g, "gelu")
        a.check_forward(forward, "gelu")
        a.check_backward(backward, "gelu")
        assert dt.dt_group_check(g) == dt.DT_OK


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("scale", [1, 40])
def test_empty_buffers_without_an_address(dt, which, scale):
    a = Layer(dt, which, [0, 3 * scale, 4 * scale, 0], 64, [24 * scale, 0, 16 * scale, 0], seed=3)
    with group(4) as g:
        want = both(a, g, "relu")
        fill = lambda ts: [t if t.numel() else None for t in ts]
        counts = (a.rows, 0, 64, a.features, 0, "bf16")
        ws = [workspace(dt, which, g, a.rows, 64, a.features, back) for back in (False, True)]
        dx, dw = fill(like(a.x)), fill(like(a.w))
        kept = lambda ts: [t for t in ts if t.numel()]
        if which == "gather_linear":
            y, pre, db = fill(like(a.pre)), fill(like(a.pre)), fill(like(a.b))
            dt.dt_gather_linear(g, fill(a.x), fill(a.w), fill(a.b), pre, y, *counts, "relu", ws[0])
            dt.dt_gather_linear_backward(g, fill(a.x), fill(a.w), fill(a.pre), fill(a.dy), dx, dw, db, *counts, "relu", ws[1])
            same([y, pre, dx, dw, db], kept(flat(want)))
        else:
            y, db = fill(like(a.res)), torch.empty_like(a.b)
            dt.dt_linear_reduce(g, fill(a.x), fill(a.w), a.b, fill(a.res), y, *counts, ws[0])
            dt.dt_linear_reduce_backward(g, fill(a.x), fill(a.w), fill(a.dy), dx, dw, db, *counts, ws[1])
            same([y, dx, dw, db], kept(flat(want)))


@pytest.mark.parametrize("rows", [[1, 2], [150, 90]])
def test_first_calls_of_a_group_in_a_capture(dt, rows):
    layers = [Layer(dt, which, rows, 136, [96, 200], seed=4) for which in WHICH]
    norm = Rows(dt, rows, 136, seed=4)
    calls = lambda g: [both(a, g, "gelu") for a in layers] + [norm.forward(g), norm.backward(g)]
    with group(2) as g:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = calls(g)
        graph.replay()
        torch.cuda.synchronize()
        same(got, calls(g))
        assert dt.dt_group_check(g) == dt.DT_OK


def test_calls_from_several_threads(dt):
    """Threads with a group and a stream each, and threads that share a group."""
    sizes = [([3, 2], 72, [40, 24]), ([70, 50], 200, [64, 24]), ([300, 212], 520, [600, 136]), ([9, 0], 1024, [300, 700])]
    results, errors = {}, []
    with group(2) as shared:
        layers = [[Layer(dt, which, *size, seed=5) for which in WHICH] for size in sizes]
        want = [[both(a, shared, "gelu") for a in pair] for pair in layers]
        torch.cuda.synchronize()

        def work(k, g):
            try:
                own = g or dt.dt_group_create(2, 0)
                with torch.cuda.stream(torch.cuda.Stream()):
                    for _ in range(5):
                        results[k, bool(g)] = [both(a, own, "gelu") for a in layers[k]]
                    torch.cuda.current_stream().synchronize()
                if not g:
                    dt.dt_group_destroy(own)
            except Exception as e:   # noqa: BLE001
                errors.append(e)
        for g in (None, shared):
            threads = [threading.Thread(target=work, args=(k, g)) for k in range(len(sizes))]
            for t in threads:
                t.start()
            for t in threads:
                t.join()
        torch.cuda.synchronize()
        assert not errors and dt.dt_group_check(shared) == dt.DT_OK
    for (k, _), got in results.items():
        same(got, want[k])
