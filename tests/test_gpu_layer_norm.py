"""Layer norm of P ranks' rows against its definition in 64 bits.

Tolerances, with u = 2^-24.  A row's sum is at most 64 dependent fp32 additions
(up to 32 elements of a thread, two shuffle trees, the last division), so a
mean is off by at most 64 u times the mean magnitude, and what is made of it
by a few roundings more: 2^-17 = 128 u times the magnitudes that enter covers
each result before it is rounded, and the store rounds by half an ulp (2^-8 of
the value in bf16, 2^-24 in f32, where twice that is allowed).  A column sum over R rows adds at most R
values in a row: (R + 8) u times the sum of magnitudes.
"""
from __future__ import annotations

import pytest
import torch

from gpu_util import TORCH_DTYPE, group

pytestmark = pytest.mark.gpu

E32 = 2.0 ** -17
HALF_ULP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -23}


@pytest.fixture(scope="module")
def dt():
    from same_device_collective_gb300 import dt as mod
    assert torch.cuda.is_available()
    return mod


def make(rows, cols, dtype, wdtype, seed, offset=0, mean=0.5):
    """x, dy per rank (views `offset` elements into an allocation), weight, bias."""
    gen = torch.Generator("cuda").manual_seed(seed)

    def view(n, dt_, std, m):
        base = torch.empty(n * cols + offset, dtype=dt_, device="cuda")
        t = base[offset:].view(n, cols)
        t.copy_(torch.randn(n, cols, generator=gen, device="cuda") * std + m)
        return t

    x = [view(n, TORCH_DTYPE[dtype], 2.0, mean) for n in rows]
    dy = [view(n, TORCH_DTYPE[dtype], 0.3, 0.0) for n in rows]
    w = (torch.randn(cols, generator=gen, device="cuda") * 0.2 + 1).to(TORCH_DTYPE[wdtype])
    b = (torch.randn(cols, generator=gen, device="cuda") * 0.2).to(TORCH_DTYPE[wdtype])
    return x, dy, w, b


def forward(dt, g, x, w, b, rows, cols, dtype, wdtype, eps=1e-5, y=None, offset=0):
    if y is None:
        y = [torch.full((t.numel() + offset,), 7.0, dtype=t.dtype, device="cuda")[offset:].view(t.shape) for t in x]
    mean, rstd = ([torch.full((n,), 9.0, device="cuda") for n in rows] for _ in range(2))
    dt.dt_layer_norm(g, x, w, b, y, mean, rstd, rows, 0, cols, eps, dtype, wdtype)
    return y, mean, rstd


def backward(dt, g, x, dy, w, mean, rstd, rows, cols, dtype, wdtype, op="sum", dx=None, offset=0):
    if dx is None:
        dx = [torch.full((t.numel() + offset,), 7.0, dtype=t.dtype, device="cuda")[offset:].view(t.shape) for t in x]
    dw, db = (torch.full((cols,), 7.0, dtype=TORCH_DTYPE[wdtype], device="cuda") for _ in range(2))
    ws = torch.empty(dt.dt_layer_norm_workspace(g, cols), dtype=torch.uint8, device="cuda")
    dt.dt_layer_norm_backward(g, x, dy, w, mean, rstd, dx, dw, db, rows, 0, cols, dtype, wdtype, op, ws)
    return dx, dw, db


def check_forward(x, w, b, y, mean, rstd, dtype, eps=1e-5):
    for r in range(len(x)):
        xd = x[r].double()
        m = xd.mean(1, keepdim=True)
        i = 1 / torch.sqrt((xd - m).square().mean(1, keepdim=True) + eps)
        h = (xd - m) * i
        wd = torch.ones_like(h[:1]) if w is None else w.double()
        bd = torch.zeros_like(h[:1]) if b is None else b.double()
        want = h * wd + bd
        big = xd.abs().amax(1, keepdim=True) if xd.numel() else xd
        tol = E32 * (wd.abs() * (h.abs() + i * big) + bd.abs()) + HALF_ULP[dtype] * want.abs()
        assert ((y[r].double() - want).abs() <= tol).all(), r
        assert ((mean[r].double() - m[:, 0]).abs() <= E32 * xd.abs().mean(1)).all()
        # the variance adds the mean's error squared and roundings of x - mean
        loose = E32 * (1 + (i * big)[:, 0]) ** 2
        assert ((rstd[r].double() - i[:, 0]).abs() <= loose * i[:, 0]).all()


def expected_backward(x, dy, w, mean, rstd):
    """dx per rank with its tolerance before the store; dweight and dbias with the sums of magnitudes."""
    out, sums = [], [0.0, 0.0, 0.0, 0.0]
    for r in range(len(x)):
        xd, g = x[r].double(), dy[r].double()
        i = rstd[r].double()[:, None]
        h = (xd - mean[r].double()[:, None]) * i
        q = g if w is None else g * w.double()
        mq, mqh = q.mean(1, keepdim=True), (q * h).mean(1, keepdim=True)
        dx = i * (q - mq - h * mqh)
        out.append((dx, E32 * i * (q.abs() + q.abs().mean(1, keepdim=True) + h.abs() * (q * h).abs().mean(1, keepdim=True))))
        for k, v in enumerate(((g * h).sum(0), g.sum(0), (g * h).abs().sum(0), g.abs().sum(0))):
            sums[k] = sums[k] + v
    return out, sums


def check_backward(x, dy, w, mean, rstd, dx, dw, db, dtype, wdtype, div=1):
    out, (sw, sb, aw, ab) = expected_backward(x, dy, w, mean, rstd)
    for r, (want, tol) in enumerate(out):
        assert ((dx[r].double() - want).abs() <= tol + HALF_ULP[dtype] * want.abs()).all(), r
    R = sum(t.shape[0] for t in x)
    for got, want, mag in ((dw, sw / div, aw / div), (db, sb / div, ab / div)):
        tol = (R + 8) * 2.0 ** -24 * mag + HALF_ULP[wdtype] * want.abs()
        assert ((got.double() - want).abs() <= tol).all()


CASES = [
    # rows per rank, cols, dtype, weight dtype, element offset
    ([1], 1, "f32", "f32", 0), ([3, 0, 2], 1, "bf16", "f32", 0), ([1, 1], 7, "bf16", "bf16", 0),
    ([5, 9], 8, "bf16", "bf16", 0), ([4, 4], 31, "f32", "bf16", 0), ([2, 3, 4, 5], 64, "bf16", "f32", 0),
    ([33, 1], 255, "bf16", "f32", 0), ([16] * 16, 256, "f32", "f32", 0), ([7, 300], 500, "bf16", "bf16", 0),
    ([700, 0, 1], 777, "f32", "f32", 0), ([64, 65], 1024, "bf16", "bf16", 1), ([64, 65], 1024, "f32", "f32", 3),
    ([200, 1000], 1021, "f32", "f32", 0), ([500] * 4, 2048, "f32", "bf16", 0), ([1] * 8, 4096, "bf16", "bf16", 0),
    ([1500, 900], 4096, "bf16", "f32", 0), ([40, 2], 4097, "bf16", "f32", 0), ([40, 2], 4096, "f32", "f32", 0),
    ([9, 4], 8192, "f32", "f32", 0), ([9, 4], 8192, "bf16", "f32", 0), ([9, 4], 8191, "bf16", "f32", 0),
    ([5], 16384, "bf16", "bf16", 0), ([5, 6], 16392, "bf16", "f32", 0), ([5], 30000, "f32", "f32", 0),
    ([2, 40], 33001, "bf16", "f32", 0), ([3], 70000, "bf16", "f32", 0),
]


@pytest.mark.parametrize("rows,cols,dtype,wdtype,offset", CASES)
def test_both_passes(dt, rows, cols, dtype, wdtype, offset):
    x, dy, w, b = make(rows, cols, dtype, wdtype, seed=cols * 31 + len(rows), offset=offset)
    with group(len(rows)) as g:
        y, mean, rstd = forward(dt, g, x, w, b, rows, cols, dtype, wdtype, offset=offset)
        check_forward(x, w, b, y, mean, rstd, dtype)
        dx, dw, db = backward(dt, g, x, dy, w, mean, rstd, rows, cols, dtype, wdtype, offset=offset)
        check_backward(x, dy, w, mean, rstd, dx, dw, db, dtype, wdtype)
        again = backward(dt, g, x, dy, w, mean, rstd, rows, cols, dtype, wdtype, offset=offset)
        assert torch.equal(dw, again[1]) and torch.equal(db, again[2])
        assert dt.dt_group_check(g) == dt.DT_OK


@pytest.mark.parametrize("dtype,cols", [("bf16", 512), ("f32", 300), ("bf16", 20000), ("f32", 40000)])
def test_in_place_equal_rows_no_weights_and_avg(dt, dtype, cols):
    P, n = 3, 17
    rows = [n] * P
    x, dy, w, _ = make(rows, cols, dtype, "f32", seed=5)
    with group(P) as g:
        y, mean, rstd = forward(dt, g, x, None, None, rows, cols, dtype, "f32")
        check_forward(x, None, None, y, mean, rstd, dtype)
        z = [t.clone() for t in x]
        dt.dt_layer_norm(g, z, None, None, z, None, [None] * P, None, n, cols, 1e-5, dtype, "f32")
        assert all(torch.equal(a, b_) for a, b_ in zip(z, y))
        dx, dw, db = backward(dt, g, x, dy, w, mean, rstd, rows, cols, dtype, "f32", op="avg")
        check_backward(x, dy, w, mean, rstd, dx, dw, db, dtype, "f32", div=P)
        # dx over dy; one gradient only; none, without a workspace
        d2 = [t.clone() for t in dy]
        ws = torch.empty(dt.dt_layer_norm_workspace(g, cols), dtype=torch.uint8, device="cuda")
        only = torch.empty(cols, device="cuda")
        dt.dt_layer_norm_backward(g, x, d2, w, mean, rstd, d2, only, None, None, n, cols, dtype, "f32", "avg", ws)
        assert all(torch.equal(a, b_) for a, b_ in zip(d2, dx)) and torch.equal(only, dw)
        d3 = [torch.empty_like(t) for t in dy]
        dt.dt_layer_norm_backward(g, x, dy, w, mean, rstd, d3, None, None, None, n, cols, dtype, "f32", "sum", None)
        assert all(torch.equal(a, b_) for a, b_ in zip(d3, dx))


def test_no_rows_gives_zero_gradients(dt):
    with group(2) as g:
        empty = [torch.empty(0, 64, device="cuda") for _ in range(2)]
        w = torch.ones(64, device="cuda")
        nothing = [torch.empty(0, device="cuda")] * 2
        dx, dw, db = backward(dt, g, empty, empty, w, nothing, nothing, [0, 0], 64, "f32", "f32", dx=empty)
        assert not dw.any() and not db.any()
        dt.dt_layer_norm(g, empty, w, w, empty, None, None, [0, 0], 0, 64, 1e-5, "f32", "f32")


@pytest.mark.parametrize("cols", [4096, 1021])
def test_mean_far_from_zero_and_constant_rows(dt, cols):
    # rows whose mean is 1000 times their spread, and rows without any spread
    with group(1) as g:
        x, _, w, b = make([64], cols, "f32", "f32", seed=3, mean=2000.0)
        x[0][1] = 3.25
        y, mean, rstd = forward(dt, g, x, w, b, [64], cols, "f32", "f32")
        check_forward(x, w, b, y, mean, rstd, "f32")
        assert torch.equal(y[0][1], b) and abs(float(rstd[0][1]) - 1e-5 ** -0.5) < 1e-2


def test_not_finite_rows_stay_in_their_rows(dt):
    with group(2) as g:
        x, dy, w, b = make([8, 8], 512, "bf16", "f32", seed=9)
        clean = forward(dt, g, x, w, b, [8, 8], 512, "bf16", "f32")
        x[0][2, 5] = float("nan")
        x[1][7, 0] = float("inf")
        y, mean, rstd = forward(dt, g, x, w, b, [8, 8], 512, "bf16", "f32")
        for r, bad in ((0, 2), (1, 7)):
            keep = torch.arange(8) != bad
            assert torch.isnan(y[r][bad]).all()
            assert torch.equal(y[r][keep], clean[0][r][keep])


# Rows that share a warp, four to 32 lanes each, and widths that are taken in 4,
# 5 and 6 vectors a thread; the last warps have fewer rows than they could.
@pytest.mark.parametrize("cols", [3, 8, 24, 33, 64, 65, 72, 128, 136, 200, 256, 264, 400, 512, 520, 640, 1280, 2056, 3000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows_of_few_columns_and_between_powers_of_two(dt, dtype, cols):
    rows = [403, 0, 1, 350]
    x, dy, w, b = make(rows, cols, dtype, "f32", seed=cols)
    with group(len(rows)) as g:
        y, mean, rstd = forward(dt, g, x, w, b, rows, cols, dtype, "f32")
        check_forward(x, w, b, y, mean, rstd, dtype)
        dx, dw, db = backward(dt, g, x, dy, w, mean, rstd, rows, cols, dtype, "f32")
        check_backward(x, dy, w, mean, rstd, dx, dw, db, dtype, "f32")
        again = backward(dt, g, x, dy, w, mean, rstd, rows, cols, dtype, "f32")
        assert torch.equal(dw, again[1]) and torch.equal(db, again[2])
        assert dt.dt_group_check(g) == dt.DT_OK


@pytest.mark.parametrize("dtype,cols", [("bf16", 64), ("bf16", 40), ("f32", 32), ("f32", 17)])
def test_not_finite_rows_leave_the_rows_of_their_warp_alone(dt, dtype, cols):
    rows = [310, 9]
    x, dy, w, b = make(rows, cols, dtype, "f32", seed=cols)
    clean = [t.clone() for t in x]
    with group(2) as g:
        y0, mean0, rstd0 = forward(dt, g, clean, w, b, rows, cols, dtype, "f32")
        dx0 = backward(dt, g, clean, dy, w, mean0, rstd0, rows, cols, dtype, "f32")[0]
        x[0][5, 0], x[0][6, cols - 1], x[0][309, 1], x[1][8, 2] = float("nan"), float("inf"), -float("inf"), float("nan")
        y, mean, rstd = forward(dt, g, x, w, b, rows, cols, dtype, "f32")
        dx = backward(dt, g, x, dy, w, mean, rstd, rows, cols, dtype, "f32")[0]
        for r, bad in ((0, [5, 6, 309]), (1, [8])):
            keep = [k for k in range(rows[r]) if k not in bad]
            assert torch.equal(y[r][keep], y0[r][keep]) and torch.equal(dx[r][keep], dx0[r][keep])
            assert not torch.isfinite(mean[r][bad]).any()


@pytest.mark.parametrize("dtype,cols", [("f32", 96), ("f32", 1021), ("bf16", 256)])
def test_gradients_against_differences(dt, dtype, cols):
    # sum(dy * y) along random directions of x, weight and bias, by central
    # differences of the definition in 64 bits
    rows = [6, 3]
    x, dy, w, b = make(rows, cols, dtype, "f32", seed=21)
    with group(2) as g:
        _, mean, rstd = forward(dt, g, x, w, b, rows, cols, dtype, "f32")
        dx, dw, db = backward(dt, g, x, dy, w, mean, rstd, rows, cols, dtype, "f32")
    X, G = torch.cat(x).double(), torch.cat(dy).double()

    def value(X, w, b):
        m = X.mean(1, keepdim=True)
        return float((G * ((X - m) / torch.sqrt((X - m).square().mean(1, keepdim=True) + 1e-5) * w + b)).sum())

    gen = torch.Generator("cuda").manual_seed(1)
    at = (X, w.double(), b.double())
    for k, grad in enumerate((torch.cat(dx), dw, db)):
        d = torch.randn(at[k].shape, generator=gen, device="cuda", dtype=torch.float64)
        lo, hi = ([v + s * 1e-4 * d if i == k else v for i, v in enumerate(at)] for s in (-1, 1))
        diff = (value(*hi) - value(*lo)) / 2e-4
        got = float((grad.double() * d).sum())
        # each element is rounded once and off by E32 of the terms it is made of: at most a few times its own size on average
        tol = float((grad.double().abs() * d.abs()).sum()) * (HALF_ULP[dtype if k == 0 else "f32"] + 8 * E32) + 1e-5
        assert abs(got - diff) <= tol, (k, got, diff, tol)


def test_another_stream_and_graph_replay(dt):
    rows, cols = [130, 70], 1024
    x, dy, w, b = make(rows, cols, "bf16", "f32", seed=2)
    with group(2) as g:
        want = forward(dt, g, x, w, b, rows, cols, "bf16", "f32")
        grads = backward(dt, g, x, dy, w, want[1], want[2], rows, cols, "bf16", "f32")
        torch.cuda.synchronize()
        y = [torch.zeros_like(t) for t in x]
        mean, rstd = ([torch.zeros(n, device="cuda") for n in rows] for _ in range(2))
        dx = [torch.zeros_like(t) for t in x]
        dw, db = torch.zeros(cols, device="cuda"), torch.zeros(cols, device="cuda")
        ws = torch.empty(dt.dt_layer_norm_workspace(g, cols), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()

        def both(stream):
            dt.dt_layer_norm(g, x, w, b, y, mean, rstd, rows, 0, cols, 1e-5, "bf16", "f32", stream)
            dt.dt_layer_norm_backward(g, x, dy, w, mean, rstd, dx, dw, db, rows, 0, cols, "bf16", "f32", "sum", ws,
                                      stream)

        side = torch.cuda.Stream()
        both(side)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            both(side)
        for t in (*y, *dx, dw, db):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b_) for a, b_ in zip(y, want[0]))
        assert all(torch.equal(a, b_) for a, b_ in zip(dx, grads[0]))
        assert torch.equal(dw, grads[1]) and torch.equal(db, grads[2])


def test_refusals(dt):
    rows, cols = [4, 4], 64
    x, dy, w, b = make(rows, cols, "f32", "f32", seed=2)
    y = [torch.zeros_like(t) for t in x]
    m = [torch.zeros(4, device="cuda") for _ in range(2)]
    s = [torch.zeros(4, device="cuda") for _ in range(2)]
    with group(2) as g:
        ws = torch.empty(dt.dt_layer_norm_workspace(g, cols), dtype=torch.uint8, device="cuda")

        def norm(status, x=x, w=w, b=b, y=y, mean=m, rstd=s, rows=rows, cols=cols, eps=1e-5, dtype="f32", wdtype="f32"):
            with pytest.raises(dt.DtError) as e:
                dt.dt_layer_norm(g, x, w, b, y, mean, rstd, rows, 0, cols, eps, dtype, wdtype)
            assert e.value.status == status

        def back(status, x=x, dy=dy, mean=m, rstd=s, dx=y, dw=torch.zeros_like(w), db=torch.zeros_like(b), ws=ws,
                 op="sum", dtype="f32"):
            with pytest.raises(dt.DtError) as e:
                dt.dt_layer_norm_backward(g, x, dy, w, mean, rstd, dx, dw, db, rows, 0, cols, dtype, "f32", op, ws)
            assert e.value.status == status

        bad, no = dt.DT_ERR_INVALID, dt.DT_ERR_UNSUPPORTED
        norm(bad, cols=0)
        norm(bad, cols=(1 << 24) + 1)
        norm(bad, eps=-1.0)
        norm(bad, eps=float("nan"))
        norm(bad, eps=float("inf"))
        norm(no, dtype="i32")
        norm(no, wdtype="i32")
        norm(bad, dtype=9)
        norm(bad, x=[x[0], 0])
        norm(bad, y=[y[0], 0])
        norm(bad, x=[x[0], x[1].data_ptr() + 2])              # not a multiple of the element
        norm(bad, w=w.data_ptr() + 1)
        norm(bad, y=[y[0], y[0]])                             # two outputs in one place
        norm(bad, y=[x[1], y[1]])                             # another rank's input
        norm(bad, y=[x[0].data_ptr() + 16, y[1]])             # not the same buffer
        norm(bad, mean=[m[0], m[0]])
        norm(bad, rows=[1 << 62, 4])
        back(no, op="max")
        back(bad, op=77)
        back(bad, ws=None)
        back(bad, ws=ws[:-16])
        back(bad, ws=(ws.data_ptr() + 4, ws.numel()))
        back(bad, dy=[dy[0], 0])
        back(bad, mean=[m[0], 0])
        back(bad, dx=[x[0], y[1]])                            # dx over x
        back(no, dtype="i32")
        with pytest.raises(ValueError):
            dt.dt_layer_norm(g, [t.t() for t in x], w, b, y, m, s, rows, 0, cols, 1e-5, "f32", "f32")
        assert dt.dt_layer_norm_workspace(g, 0) == 0
        torch.cuda.synchronize()
        assert not any(t.any() for t in y) and dt.dt_group_check(g) == dt.DT_OK


# Rows too long for registers have 32 shares of the weights' gradients, whatever
# the number of SMs; no share lies outside the workspace that was asked for.
@pytest.mark.parametrize("cols,dtype", [(16384, "bf16"), (16384, "f32"), (16385, "bf16"), (16388, "f32"), (1 << 20, "f32")])
def test_workspace_of_long_rows(dt, cols, dtype):
    rows = [37, 3]
    x, dy, w, b = make(rows, cols, dtype, "f32", seed=cols)
    with group(2) as g:
        assert dt.dt_layer_norm_workspace(g, 1 << 24) == 32 * 2 * 4 << 24
        size = dt.dt_layer_norm_workspace(g, cols)
        assert size >= 32 * 2 * 4 * cols and (cols <= 16384 or size == 32 * 2 * 4 * cols)
        _, mean, rstd = forward(dt, g, x, w, b, rows, cols, dtype, "f32")
        dx, dw, db = [torch.empty_like(t) for t in x], torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        base = torch.full((size + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        dt.dt_layer_norm_backward(g, x, dy, w, mean, rstd, dx, dw, db, rows, 0, cols, dtype, "f32", "sum",
                                  base[4096:4096 + size])
        check_backward(x, dy, w, mean, rstd, dx, dw, db, dtype, "f32")
        assert (base[:4096] == 0xA5).all() and (base[4096 + size:] == 0xA5).all()
        with pytest.raises(dt.DtError):
            dt.dt_layer_norm_backward(g, x, dy, w, mean, rstd, dx, dw, db, rows, 0, cols, dtype, "f32", "sum",
                                      base[4096:4096 + size - 16])


# One row of blocks for all ranks where their rows are uneven, a row to a rank
# where they are not: every rank has its own rows' results either way.
@pytest.mark.parametrize("rows", [[900] + [0] * 15, [0] * 15 + [900], [1] * 7 + [700] + [2] * 8, [0, 0, 1000], [500, 0, 500],
                                  [400, 300, 350], [3, 900, 0, 0, 40]])
@pytest.mark.parametrize("dtype,cols", [("bf16", 64), ("bf16", 1024), ("f32", 640), ("f32", 31), ("bf16", 4096)])
def test_rows_of_uneven_ranks(dt, rows, dtype, cols):
    x, dy, w, b = make(rows, cols, dtype, "f32", seed=cols + len(rows))
    with group(len(rows)) as g, group(1) as one:
        y, mean, rstd = forward(dt, g, x, w, b, rows, cols, dtype, "f32")
        check_forward(x, w, b, y, mean, rstd, dtype)
        # the same rows as those of a single rank, bit for bit
        ya, ma, ra = forward(dt, one, [torch.cat(x)], w, b, [sum(rows)], cols, dtype, "f32")
        assert torch.equal(torch.cat(y), ya[0]) and torch.equal(torch.cat(mean), ma[0]) and torch.equal(torch.cat(rstd), ra[0])
        assert dt.dt_group_check(g) == dt.DT_OK


def test_a_rank_with_all_rows_costs_no_more_than_one_rank(dt):
    cols, n = 64, 1 << 19
    x = torch.randn(n, cols, device="cuda").bfloat16()
    y, w = torch.empty_like(x), torch.ones(cols, device="cuda")
    none = torch.empty(0, cols, dtype=torch.bfloat16, device="cuda")

    def best(P):
        rest = [none] * (P - 1)
        with group(P) as g:
            call = dt.prepare(dt.dt_layer_norm, g, [x, *rest], w, w, [y, *rest], None, None, [n] + [0] * (P - 1), 0, cols,
                              1e-5, "bf16", "f32")
            took = []
            for _ in range(8):
                a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
                torch.cuda._sleep(200_000)
                a.record()
                for _ in range(4):
                    call()
                b.record()
                torch.cuda.synchronize()
                took.append(a.elapsed_time(b))
            return min(took)

    one, many = best(1), best(16)
    assert many <= 2 * one, (one, many)


# Rows of a few bytes: a stage of them has as many means and reciprocals, which
# take more room than the rows, and all groups' stages have to fit an SM.
@pytest.mark.parametrize("rows,cols,dtype", [([5_100_000, 7], 1, "bf16"), ([1_300_000, 1_400_000], 2, "bf16"),
                                             ([2_600_000], 1, "f32"), ([0, 1_800_000], 3, "bf16")])
def test_millions_of_very_short_rows(dt, rows, cols, dtype):
    x, dy, w, b = make(rows, cols, dtype, "f32", seed=cols)
    with group(len(rows)) as g:
        y, mean, rstd = forward(dt, g, x, w, b, rows, cols, dtype, "f32")
        check_forward(x, w, b, y, mean, rstd, dtype)
        dx, dw, db = backward(dt, g, x, dy, w, mean, rstd, rows, cols, dtype, "f32")
        check_backward(x, dy, w, mean, rstd, dx, dw, db, dtype, "f32")
        assert dt.dt_group_check(g) == dt.DT_OK


# A kernel may have 48 KB of shared memory without asking, its static part
# included: calls whose rings come near that, each the first of its kernel in a
# process (once a larger call has asked, they all may).
NEAR_48_KB = r"""
import sys
sys.path[:0] = [ROOT, TESTS]
import torch
import test_gpu_layer_norm as T
from same_device_collective_gb300 import dt
from gpu_util import group
for rows, cols, dtype, offset in (([1], 6144, "bf16", 0), ([6, 7], 6112, "f32", 0), ([13], 6144, "bf16", 1), ([0, 13], 6104, "f32", 3),
                                  ([13], 12256, "f32", 0), ([300], 12224, "bf16", 0), ([5000], 592, "bf16", 1),
                                  ([2000], 592, "f32", 1), ([1000], 864, "bf16", 0), ([500], 1480, "f32", 0),
                                  ([1000], 1465, "bf16", 1), ([500], 1465, "f32", 1), ([500], 6102, "bf16", 3)):
    x, dy, w, b = T.make(rows, cols, dtype, "f32", seed=cols, offset=offset)
    with group(len(rows)) as g:
        y, mean, rstd = T.forward(dt, g, x, w, b, rows, cols, dtype, "f32", offset=offset)
        T.check_forward(x, w, b, y, mean, rstd, dtype)
        dx, dw, db = T.backward(dt, g, x, dy, w, mean, rstd, rows, cols, dtype, "f32", offset=offset)
        T.check_backward(x, dy, w, mean, rstd, dx, dw, db, dtype, "f32")
print("all right")
"""


def test_first_calls_that_need_nearly_48_kb(dt):
    import os
    import subprocess
    import sys
    tests = os.path.dirname(os.path.abspath(__file__))
    code = NEAR_48_KB.replace("ROOT", repr(os.path.dirname(tests))).replace("TESTS", repr(tests))
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "all right" in out.stdout, out.stderr[-3000:]
