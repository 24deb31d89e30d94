"""The linear layers and the residual norm write their outputs and nothing else: every output and workspace
stands between guard bytes, and no input changes.  Sizes reach every kernel of each call: few tokens, small
products, and the tensor cores' tiles with splits and with rows laid out again."""
from __future__ import annotations

import pytest
import torch

from gpu_util import TORCH_DTYPE, group
from test_gpu_guards import Guarded, guarded_like, snapshot, unchanged, values

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def dt():
    from same_device_collective_gb300 import dt as mod
    return mod


SIZES = [([1, 0, 2], 64, [40, 0, 100]), ([9, 4, 1], 333, [100, 31, 7]), ([30, 0, 47], 500, [100, 301, 250]),
         ([200, 50, 60], 96, [64, 128, 33]), ([40, 20, 30], 2050, [3000, 1001, 700]), ([700, 300, 61], 1021, [1500, 601, 800]),
         ([600, 20, 400], 64, [2000, 0, 1096]), ([256, 256, 256], 1024, [2048, 1024, 1024])]


@pytest.mark.parametrize("rows,dim,features", SIZES)
@pytest.mark.parametrize("shift", [0, 2])
def test_linear_layers_write_only_their_outputs(dt, rows, dim, features, shift):
    n, P = sum(rows), len(rows)
    v = lambda *s, seed: values(*s, seed=seed, dtype=BF16, std=0.5)
    tokens = lambda seed: [v(k, dim, seed=seed + r) for r, k in enumerate(rows)]
    inner = lambda seed: [v(n, f, seed=seed + r) for r, f in enumerate(features)]
    out_tokens = lambda: [guarded_like(k * dim, "bf16", shift) for k in rows]
    out_inner = lambda: [guarded_like(n * f, "bf16", shift) for f in features]
    out_w = lambda: [guarded_like(f * dim, "bf16", shift) for f in features]
    view = lambda out: [t for _, t in out]
    x, h, w1, w2 = tokens(1), inner(20), [v(f, dim, seed=40 + r) for r, f in enumerate(features)], [v(dim, f, seed=60 + r) for r, f in enumerate(features)]
    b1, b2 = [v(f, seed=80 + r) for r, f in enumerate(features)], v(dim, seed=99)
    inputs = [*x, *h, *w1, *w2, *b1, b2]
    snap = snapshot(inputs)
    y, pre, dxr, dx, dw1, dw2 = out_inner(), out_inner(), out_inner(), out_tokens(), out_w(), out_w()
    z, db1, db2 = out_tokens(), [guarded_like(f, "bf16", shift) for f in features], guarded_like(dim, "bf16", shift)
    args = (rows, 0, dim, features, 0, "bf16")
    with group(P) as g:
        ws = [Guarded(query(g, *args, back)) for query in (dt.dt_gather_linear_workspace, dt.dt_linear_reduce_workspace)
              for back in (False, True)]
        w = [t.view(torch.uint8) for t in ws]
        dt.dt_gather_linear(g, x, w1, b1, view(pre), view(y), *args, "gelu", w[0])
        dt.dt_gather_linear_backward(g, x, w1, h, h, view(dx), view(dw1), view(db1), *args, "gelu", w[1])
        dt.dt_linear_reduce(g, h, w2, b2, x, view(z), *args, w[2])
        dt.dt_linear_reduce_backward(g, h, w2, x, view(dxr), view(dw2), db2[1], *args, w[3])
        torch.cuda.synchronize()
        assert dt.dt_group_check(g) == dt.DT_OK
    assert unchanged(inputs, snap)
    for what, outs in (("y", y), ("pre", pre), ("dx", dx), ("dw1", dw1), ("db1", db1), ("z", z), ("dxr", dxr), ("dw2", dw2),
                       ("db2", [db2])):
        for r, (guard, t) in enumerate(outs):
            assert guard.intact(), (what, r)
            assert torch.isfinite(t).all(), (what, r)
    assert all(t.intact() for t in ws)


@pytest.mark.parametrize("rows,cols,dtype,wdtype", [([3, 0, 5], 7, "bf16", "bf16"), ([400, 1, 30], 1024, "bf16", "f32"),
                                                    ([40, 33, 0], 1021, "f32", "f32"), ([9, 300, 4], 64, "bf16", "f32"),
                                                    ([350, 2, 3], 33, "f32", "bf16"), ([5, 3, 1], 9000, "f32", "f32"),
                                                    ([3, 2, 1], 20001, "bf16", "bf16"), ([700, 80, 9], 4096, "f32", "f32")])
@pytest.mark.parametrize("shift", [0, 4])
def test_residual_norm_writes_only_its_outputs(dt, rows, cols, dtype, wdtype, shift):
    t = TORCH_DTYPE[dtype]
    x, branch, dy, dz = ([values(k, cols, seed=s + r, dtype=t) for r, k in enumerate(rows)] for s in (1, 100, 200, 300))
    w = [values(cols, seed=s, dtype=TORCH_DTYPE[wdtype]) for s in (5, 6, 7)]
    inputs = [*x, *branch, *dy, *dz, *w]
    snap = snapshot(inputs)
    y, z, dx, do = ([guarded_like(k * cols, dtype, shift) for k in rows] for _ in range(4))
    r1, r2 = ([guarded_like(k, "f32", shift) for k in rows] for _ in range(2))
    dw = [guarded_like(cols, wdtype, shift) for _ in range(3)]
    view = lambda out: [v for _, v in out]
    with group(len(rows)) as g:
        ws = Guarded(dt.dt_residual_norm_workspace(g, cols))
        dt.dt_residual_norm(g, x, branch, *w, 0.5, view(y), view(z), view(r1), view(r2), rows, 0, cols, 1e-6, dtype, wdtype)
        dt.dt_residual_norm_backward(g, branch, view(y), dy, dz, *w, 0.5, view(r1), view(r2), view(dx), view(do), *view(dw), rows,
                                     0, cols, dtype, wdtype, "sum", ws.view(torch.uint8))
        torch.cuda.synchronize()
        assert dt.dt_group_check(g) == dt.DT_OK
    assert unchanged(inputs, snap)
    for what, outs in (("y", y), ("z", z), ("rstd post", r1), ("rstd pre", r2), ("dx", dx), ("dbranch", do), ("weights", dw)):
        for r, (guard, v) in enumerate(outs):
            assert guard.intact(), (what, r)
            assert torch.isfinite(v).all(), (what, r)
    assert ws.intact()
