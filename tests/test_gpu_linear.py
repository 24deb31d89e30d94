"""The linear layers over the ranks against their definitions in 64 bits.

Tolerances, with u = 2^-23 (the tensor cores' fp32 sums may truncate).  A sum over K products is made
in steps of 16, each rounded once, with at most a step more for each rank's piece and a few additions
where splits are joined and bias and residual added: (K / 16 + 32 + P) u times the sum of magnitudes.
An activation is steep by at most 1.13 and off by 2^-16 of its result (its exponential's argument, up
to 100, is off by u of itself; the tail's fit by 3e-6), its derivative by 2^-16.  A result is rounded
to bf16 once: 2^-8 of itself.  The gradient before the activation is rounded as the products' operand
as well: 2^-8 of each term.  1e-37 is for what is flushed to zero.
"""
from __future__ import annotations

import math

import pytest
import torch

from gpu_util import group

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
R = 2.0 ** -8
ACTS = ["none", "relu", "gelu", "silu"]
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def dt():
    from same_device_collective_gb300 import dt as mod
    assert torch.cuda.is_available()
    return mod


def made(gen, *shape, std=1.0, offset=0):
    """bf16 values of a dense tensor that starts `offset` elements into its allocation."""
    n = math.prod(shape)
    t = torch.empty(n + offset, dtype=BF16, device="cuda")[offset:].view(*shape)
    return t.copy_(torch.randn(*shape, generator=gen, device="cuda") * std)


def like(ts, offset=0):
    return [torch.full((t.numel() + offset,), 7.0, dtype=BF16, device="cuda")[offset:].view(t.shape) for t in ts]


def workspace(dt, which, g, rows, dim, features, backward):
    n = getattr(dt, f"dt_{which}_workspace")(g, rows, 0, dim, features, 0, "bf16", backward)
    assert n > 0
    return torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")


def act64(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "gelu":
        return v * 0.5 * torch.erfc(v * -math.sqrt(0.5))
    if act == "silu":
        return v * torch.sigmoid(v)
    return v


def slope64(v, act):
    if act == "relu":
        return (v > 0).double()
    if act == "gelu":
        return 0.5 * torch.erfc(v * -math.sqrt(0.5)) + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    if act == "silu":
        p = torch.sigmoid(v)
        return p * (1 + v * (1 - p))
    return torch.ones_like(v)


def sum_error(k, P):
    return (k / 16 + 32 + P) * U


def check(got, want, tol, what):
    got = got.double()
    bad = ~((got - want).abs() <= tol + R * want.abs() + 1e-37)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], want[bad][:4], tol.expand_as(want)[bad][:4])


class Layer:
    """Inputs of a gathering or a reducing layer, and its calls."""

    def __init__(self, dt, which, rows, dim, features, seed=0, offset=0, bias=True, residual=True):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.dt, self.which, self.rows, self.dim, self.features, self.P = dt, which, rows, dim, features, len(rows)
        self.n, self.offset = sum(rows), offset
        F = sum(features)
        if which == "gather_linear":
            self.x = [made(gen, k, dim, offset=offset) for k in rows]
            self.w = [made(gen, f, dim, std=1.5 * dim ** -0.5, offset=offset) for f in features]
            self.b = [made(gen, f, offset=offset) for f in features] if bias else None
            self.pre = [made(gen, self.n, f, std=1.5, offset=offset) for f in features]
            self.dy = [made(gen, self.n, f, offset=offset) for f in features]
        else:
            self.x = [made(gen, self.n, f, offset=offset) for f in features]
            self.w = [made(gen, dim, f, std=F ** -0.5, offset=offset) for f in features]
            self.b = made(gen, dim, offset=offset) if bias else None
            self.res = [made(gen, k, dim, offset=offset) for k in rows] if residual else None
            self.dy = [made(gen, k, dim, offset=offset) for k in rows]

    def forward(self, g, act="none", keep=True, stream=None, y=None):
        dt, ws = self.dt, workspace(self.dt, self.which, g, self.rows, self.dim, self.features, False)
        if self.which == "gather_linear":
            y = like([torch.empty(self.n, f) for f in self.features], self.offset)
            pre = like(y, self.offset) if keep else None
            dt.dt_gather_linear(g, self.x, self.w, self.b, pre, y, self.rows, 0, self.dim, self.features, 0, "bf16", act,
                                ws, stream)
            return y, pre
        y = y or like([torch.empty(k, self.dim) for k in self.rows], self.offset)
        dt.dt_linear_reduce(g, self.x, self.w, self.b, self.res, y, self.rows, 0, self.dim, self.features, 0, "bf16", ws,
                            stream)
        return y

    def backward(self, g, act="none", stream=None):
        dt, ws = self.dt, workspace(self.dt, self.which, g, self.rows, self.dim, self.features, True)
        dx, dw = like(self.x, self.offset), like(self.w, self.offset)
        if self.which == "gather_linear":
            db = like(self.b, self.offset) if self.b else None
            dt.dt_gather_linear_backward(g, self.x, self.w, self.pre if act != "none" else None, self.dy, dx, dw, db,
                                         self.rows, 0, self.dim, self.features, 0, "bf16", act, ws, stream)
        else:
            db = like([self.b], self.offset)[0] if self.b is not None else None
            dt.dt_linear_reduce_backward(g, self.x, self.w, self.dy, dx, dw, db, self.rows, 0, self.dim, self.features, 0,
                                         "bf16", ws, stream)
        return dx, dw, db

    def check_forward(self, out, act="none"):
        if self.which == "gather_linear":
            y, pre = out
            X = torch.cat(self.x).double()
            for r, w in enumerate(self.w):
                w = w.double()
                v, tol = X @ w.t(), sum_error(self.dim, self.P) * (X.abs() @ w.abs().t())
                if self.b:
                    v = v + self.b[r].double()
                tol = tol + 4 * U * v.abs()
                if pre:
                    check(pre[r], v, tol, f"pre {r}")
                a = act64(v, act)
                check(y[r], a, 1.13 * tol + 2.0 ** -16 * a.abs(), f"y {r}")
            return
        X, W = torch.cat(self.x, 1).double(), torch.cat(self.w, 1).double()
        v, tol = X @ W.t(), sum_error(X.shape[1], self.P) * (X.abs() @ W.abs().t())
        for extra in (self.b, torch.cat(self.res) if self.res else None):
            if extra is not None:
                v, tol = v + extra.double(), tol + 4 * U * (v.abs() + extra.double().abs())
        check(torch.cat(out), v, tol, "y")

    def check_backward(self, out, act="none"):
        dx, dw, db = out
        if self.which == "gather_linear":
            X, dX, size = torch.cat(self.x).double(), 0.0, 0.0
            for r in range(self.P):
                dy = self.dy[r].double()
                gr = dy * slope64(self.pre[r].double(), act)
                off = 0 * gr if act in ("none", "relu") else R * gr.abs() + 2.0 ** -16 * dy.abs()
                w = self.w[r].double()
                dX = dX + gr @ w
                size = size + (off + sum_error(sum(self.features), self.P) * gr.abs()) @ w.abs()
                tol = (off + sum_error(self.n, self.P) * gr.abs()).t() @ X.abs()
                check(dw[r], gr.t() @ X, tol, f"dw {r}")
                if db:
                    check(db[r], gr.sum(0), (2.0 ** -16 * dy.abs() + (self.n + 32) * U * gr.abs()).sum(0), f"db {r}")
            check(torch.cat(dx), dX, size, "dx")
            return
        Y = torch.cat(self.dy).double()
        for r in range(self.P):
            x, w = self.x[r].double(), self.w[r].double()
            check(dx[r], Y @ w, sum_error(self.dim, self.P) * (Y.abs() @ w.abs()), f"dx {r}")
            check(dw[r], Y.t() @ x, sum_error(self.n, self.P) * (Y.abs().t() @ x.abs()), f"dw {r}")
        if db is not None:
            check(db, Y.sum(0), (self.n + 32) * U * Y.abs().sum(0), "db")


# tokens of each rank, columns, features of each rank: single tokens, tile edges (128, 256), ranks without tokens or
# features, widths that TMA cannot address, pieces that end inside a tile or a step of 16
SHAPES = [
    ([1], 8, [8]),
    ([1], 1, [1]),
    ([1, 0, 2], 64, [5, 0, 300]),
    ([1, 1, 1, 1], 512, [256, 256, 256, 256]),
    ([5], 1024, [1000]),
    ([16], 136, [72]),
    ([17, 3], 200, [64, 129]),
    ([40, 30, 7], 333, [100, 1, 20]),
    ([64, 64], 256, [128, 384]),
    ([128], 130, [258]),
    ([129], 128, [257]),
    ([0, 255, 2], 96, [0, 31, 500]),
    ([256, 256], 320, [256, 128]),
    ([256, 16, 240], 264, [640, 8]),
    ([300, 200, 100, 9], 127, [33, 65, 90, 2]),
    ([512, 512], 2048, [40, 56]),
    ([1100], 72, [1500]),
    ([700, 333], 1000, [513, 511]),
]
WHICH = ["gather_linear", "linear_reduce"]


def padded(shape, P):
    rows, dim, features = shape
    return rows + [0] * (P - len(rows)), dim, features + [0] * (P - len(features))


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(dt, which, shape):
    rows, dim, features = padded(shape, max(len(shape[0]), len(shape[2])))
    a = Layer(dt, which, rows, dim, features, seed=dim)
    with group(a.P) as g:
        act = ACTS[sum(rows) % 4] if which == "gather_linear" else "none"
        out = a.forward(g, act) if which == "gather_linear" else a.forward(g)
        assert dt.dt_group_check(g) == dt.DT_OK
        a.check_forward(out, act)


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(dt, which, shape):
    rows, dim, features = padded(shape, max(len(shape[0]), len(shape[2])))
    a = Layer(dt, which, rows, dim, features, seed=dim + 1)
    with group(a.P) as g:
        act = ACTS[(sum(rows) + 2) % 4] if which == "gather_linear" else "none"
        out = a.backward(g, act)
        assert dt.dt_group_check(g) == dt.DT_OK
        a.check_backward(out, act)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("keep,bias", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("rows", [[3, 2], [70, 130]])
def test_activations(dt, act, keep, bias, rows):
    a = Layer(dt, "gather_linear", rows, 144, [72, 56], seed=3, bias=bias)
    a.w = [w.mul_(6) for w in a.w]   # far into both of an activation's tails
    with group(2) as g:
        a.check_forward(a.forward(g, act, keep), act)
        a.pre = [p.mul_(4) for p in a.pre]
        a.check_backward(a.backward(g, act), act)


@pytest.mark.parametrize("bias,residual", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("rows", [[2, 2], [100, 50]])
def test_reduce_without(dt, bias, residual, rows):
    a = Layer(dt, "linear_reduce", rows, 96, [64, 33], seed=4, bias=bias, residual=residual)
    with group(2) as g:
        a.check_forward(a.forward(g))
        a.check_backward(a.backward(g))


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("offset", [1, 2, 4])
@pytest.mark.parametrize("rows,dim,features", [([2, 1], 64, [96, 32]), ([150, 50], 64, [128, 72])])
def test_buffers_off_a_vector_boundary(dt, which, offset, rows, dim, features):
    a = Layer(dt, which, rows, dim, features, seed=offset, offset=offset)
    with group(a.P) as g:
        a.check_forward(a.forward(g))
        a.check_backward(a.backward(g))


@pytest.mark.parametrize("which", WHICH)
def test_many_ranks(dt, which):
    rows = [0, 1, 17, 40, 3, 0, 64, 5, 9, 16, 2, 2, 7, 31, 33, 1]
    a = Layer(dt, which, rows, 160, [16 * (r % 5) for r in range(16)], seed=9)
    with group(16) as g:
        a.check_forward(a.forward(g, "silu") if which == "gather_linear" else a.forward(g), "silu")
        a.check_backward(a.backward(g))


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("tokens,dim,features", [(384, 8192, [24, 40]), (64, 72, [9000, 3000]), (600, 64, [64, 64]),
                                                  (20, 16384, [64, 8])])
def test_few_tiles_of_a_long_inner_axis(dt, which, tokens, dim, features):
    """Few outputs, so that the inner axis is split over the SMs."""
    a = Layer(dt, which, [tokens // 2, tokens - tokens // 2], dim, features, seed=tokens)
    with group(2) as g:
        a.check_forward(a.forward(g, "gelu") if which == "gather_linear" else a.forward(g), "gelu")
        a.check_backward(a.backward(g, "gelu") if which == "gather_linear" else a.backward(g), "gelu")


@pytest.mark.parametrize("which", WHICH)
def test_ranks_whose_tokens_follow_one_another(dt, which):
    """One tensor cut between the ranks at no tile's edge is read in place."""
    a = Layer(dt, which, [100, 37, 200], 128, [64, 64, 64], seed=6)
    if which == "gather_linear":
        a.x = list(torch.cat(a.x).split(a.rows))
    else:
        a.dy = list(torch.cat(a.dy).split(a.rows))
    with group(3) as g:
        a.check_forward(a.forward(g))
        a.check_backward(a.backward(g))


def test_residual_in_place(dt):
    a = Layer(dt, "linear_reduce", [90, 200], 200, [128, 136], seed=8)
    before = [t.clone() for t in a.res]
    with group(2) as g:
        want = a.forward(g)
        a.forward(g, y=a.res)
        for got, w in zip(a.res, want):
            assert torch.equal(got, w)
        a.res = before
        a.check_forward(want)


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("rows", [[3, 1], [48, 80, 16], [300, 212]])
def test_a_bad_token_stays_alone(dt, which, rows):
    """Infinities and NaN of one token reach no other token's results."""
    features = [64] * len(rows)
    a = Layer(dt, which, rows, 128, features, seed=11)
    with group(a.P) as g:
        clean = a.forward(g)
        clean = torch.cat(clean[0], 1) if which == "gather_linear" else torch.cat(clean)
        dx = a.backward(g)[0]
        dx = torch.cat(dx) if which == "gather_linear" else torch.cat(dx, 1)
        bad = rows[0]   # the second rank's first token
        if which == "gather_linear":
            a.x[1][0, 3] = float("inf")
            a.dy[0][bad, 5] = float("nan")
        else:
            a.x[0][bad, 3] = float("nan")
            a.dy[1][0, 5] = float("inf")
        y = a.forward(g)
        y = torch.cat(y[0], 1) if which == "gather_linear" else torch.cat(y)
        keep = torch.arange(sum(rows), device="cuda") != bad
        assert torch.equal(y[keep], clean[keep]) and not torch.isfinite(y[bad].float()).all()
        d, dw, db = a.backward(g)
        d = torch.cat(d) if which == "gather_linear" else torch.cat(d, 1)
        assert torch.equal(d[keep], dx[keep]) and not torch.isfinite(d[bad].float()).all()
        # a weight's gradient is bad where the bad token's value enters it, and only there
        for r in range(a.P):
            w = torch.isfinite(dw[r].float())
            if which == "gather_linear":
                assert w[:5 if r == 0 else None, :3].all() and not w[:, 3].any() and (r or not w[5].any())
            else:
                assert (w[:5, :3] if r == 0 else w[:5]).all() and not w[5].any() and (r or not w[:, 3].any())


@pytest.mark.parametrize("which", WHICH)
def test_no_tokens(dt, which):
    a = Layer(dt, which, [0, 0], 24, [16, 40], seed=1)
    with group(2) as g:
        a.forward(g)
        dx, dw, db = a.backward(g)
        assert all((t == 0).all() for t in dw)
        assert all((t == 0).all() for t in (db if isinstance(db, list) else [db]))


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("rows", [[2, 2], [90, 70]])
def test_the_same_bits_again_and_on_another_stream(dt, which, rows):
    a = Layer(dt, which, rows, 1000, [96, 2000], seed=2)
    flat = lambda out: [t for v in out if v is not None for t in (v if isinstance(v, (list, tuple)) else [v])]
    with group(2) as g:
        first = flat([a.forward(g)[0] if which == "gather_linear" else a.forward(g), *a.backward(g)])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            again = flat([a.forward(g)[0] if which == "gather_linear" else a.forward(g), *a.backward(g)])
        s.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(first, again))


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("rows", [[1, 1], [90, 71]])
def test_captured_and_replayed(dt, which, rows):
    """A graph of both passes, replayed on new inputs, gives what the calls give."""
    a = Layer(dt, which, rows, 152, [96, 200], seed=12)
    b = Layer(dt, which, rows, 152, [96, 200], seed=13)
    with group(2) as g:
        want = [b.forward(g), b.backward(g)]
        a.forward(g), a.backward(g)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = [a.forward(g), a.backward(g)]
        for name in ("x", "w", "dy"):
            for t, v in zip(getattr(a, name), getattr(b, name)):
                t.copy_(v)
        if which == "gather_linear":
            for t, v in zip(a.b, b.b):
                t.copy_(v)
        else:
            a.b.copy_(b.b)
            for t, v in zip(a.res, b.res):
                t.copy_(v)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()

        def flat(v):
            return [t for u in v for t in flat(u)] if isinstance(v, (list, tuple)) else [v] if v is not None else []
        assert all(torch.equal(x, y) for x, y in zip(flat(got), flat(want)))


@pytest.mark.parametrize("which", WHICH)
def test_refusals(dt, which):
    a = Layer(dt, which, [4, 2], 16, [8, 24], seed=1)
    fwd, bwd = getattr(dt, f"dt_{which}"), getattr(dt, f"dt_{which}_backward")
    with group(2) as g:
        def call(fn=fwd, status=dt.DT_ERR_INVALID, **change):
            back = fn is bwd
            args = dict(g=g, x=a.x, weight=a.w, rows=a.rows, rows_equal=0, dim=16, features=a.features, features_equal=0,
                        dtype="bf16", workspace=workspace(dt, which, g, a.rows, 16, a.features, back))
            if which == "gather_linear":
                y = like([torch.empty(6, f) for f in a.features])
                args["act"] = "gelu"
                args.update(dict(dy=a.dy, dx=like(a.x), dweight=like(a.w), dbias=like(a.b), pre=a.pre) if back
                            else dict(bias=a.b, pre=like(y), y=y))
            else:
                args.update(dict(dy=a.dy, dx=like(a.x), dweight=like(a.w), dbias=like([a.b])[0]) if back
                            else dict(bias=a.b, residual=a.res, y=like(a.res)))
            args.update({k: v(args) if callable(v) else v for k, v in change.items()})
            if status == dt.DT_OK:
                return fn(**args)
            with pytest.raises(dt.DtError) as e:
                fn(**args)
            assert e.value.status == status

        for fn in (fwd, bwd):
            call(fn, dt.DT_OK)
            call(fn, dim=0)
            call(fn, features=[0, 0])
            call(fn, workspace=None)
            call(fn, workspace=lambda k: k["workspace"][256:])          # too small
            call(fn, workspace=lambda k: (k["workspace"].data_ptr() + 64, k["workspace"].numel()))
            call(fn, rows=[1 << 40, 2])
            call(fn, x=[None, a.x[1]])
            call(fn, weight=[a.w[0], None])
        call(fwd, y=lambda k: [None, k["y"][1]])
        call(fwd, y=lambda k: [k["y"][0], k["y"][0].view(-1)[:k["y"][1].numel()]] if k["y"][1].numel() < k["y"][0].numel()
             else [k["y"][1].view(-1)[:k["y"][0].numel()], k["y"][1]])   # outputs that overlap
        call(fwd, y=lambda k: [k["x"][0] if which == "linear_reduce" else k["weight"][0], k["y"][1]])
        call(bwd, dweight=lambda k: k["weight"])
        call(bwd, dx=lambda k: k["x"])
        call(bwd, dx=lambda k: [None, k["dx"][1]])
        call(bwd, dy=lambda k: [None, k["dy"][1]])
        if which == "gather_linear":
            for fn in (fwd, bwd):
                call(fn, act=4)
                call(fn, act=-1)
            call(bwd, pre=None)
            call(bwd, dt.DT_OK, pre=None, act="none")
        f32 = [t.float() for t in a.x]
        with pytest.raises(ValueError):
            call(fwd, x=f32)
        with pytest.raises(ValueError):
            call(fwd, x=[t.t() for t in a.x])
        with pytest.raises(ValueError):
            call(fwd, weight=a.w[:1])
        query = getattr(dt, f"dt_{which}_workspace")
        assert query(g, a.rows, 0, 16, a.features, 0, "f32", False) == 0
        assert query(g, a.rows, 0, 0, a.features, 0, "bf16", False) == 0
        assert query(g, a.rows, 0, 16, [0, 0], 0, "bf16", True) == 0
        assert dt.dt_group_check(g) == dt.DT_OK


def test_f32_is_unsupported(dt):
    f = lambda *s: torch.zeros(*s, device="cuda")
    with group(1) as g:
        ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
        with pytest.raises(dt.DtError) as e:
            dt.dt_gather_linear(g, [f(4, 8)], [f(8, 8)], None, None, [f(4, 8)], [4], 0, 8, [8], 0, "f32", "none", ws)
        assert e.value.status == dt.DT_ERR_UNSUPPORTED
        with pytest.raises(dt.DtError) as e:
            dt.dt_linear_reduce(g, [f(4, 8)], [f(8, 8)], None, None, [f(4, 8)], [4], 0, 8, [8], 0, "f32", ws)
        assert e.value.status == dt.DT_ERR_UNSUPPORTED


# sizes that the tensor cores' tiles take: one CTA and pairs, widths that TMA cannot address, ranks' pieces that are read
# in place, as one, or laid out again, tiles that end inside a rank, and inner axes that are split over the SMs
LARGE = [
    ([100], 2048, [4000]),
    ([60, 0, 61], 1999, [3001, 0, 2001]),
    ([128], 4096, [512]),
    ([256, 128, 384], 1024, [1024, 512, 640]),
    ([700, 521], 1021, [2003, 1000]),
    ([300, 900, 100, 260], 1500, [515, 700, 1030, 129]),
    ([1, 1300, 0, 11], 1024, [1500, 8, 0, 800]),
    ([2000, 2100], 136, [3000, 1000]),
    ([9000, 7000], 72, [100, 30]),
    ([20000], 64, [64]),
    ([512], 6000, [100, 100]),
    ([160, 96], 64, [9000, 7000]),
    ([500, 12], 2000, [600, 400]),
    ([300, 0, 33], 1000, [1400, 700, 8]),
]


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("offset", [0, 3])
@pytest.mark.parametrize("shape", LARGE, ids=str)
def test_large_products(dt, which, shape, offset):
    rows, dim, features = padded(shape, max(len(shape[0]), len(shape[2])))
    a = Layer(dt, which, rows, dim, features, seed=dim + 2, offset=offset)
    with group(a.P) as g:
        act = ACTS[(sum(rows) + dim) % 4] if which == "gather_linear" else "none"
        a.check_forward(a.forward(g, act) if which == "gather_linear" else a.forward(g), act)
        a.check_backward(a.backward(g, act), act)
        assert dt.dt_group_check(g) == dt.DT_OK


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("shape", [([7, 5], 4096, [5000, 4600]), ([2, 1], 8192, [16000, 400])], ids=str)
def test_few_tokens_of_large_weights(dt, which, shape):
    a = Layer(dt, which, *shape, seed=21)
    with group(2) as g:
        a.check_forward(a.forward(g, "gelu") if which == "gather_linear" else a.forward(g),
                        "gelu" if which == "gather_linear" else "none")
        assert dt.dt_group_check(g) == dt.DT_OK


@pytest.mark.parametrize("rows,dim,features", [([3, 2], 72, [40, 24]), ([40, 30], 200, [64, 24]),
                                               ([300, 84], 64, [4096, 4096]), ([700, 324], 2048, [512, 512])])
def test_residual_in_place_of_every_size(dt, rows, dim, features):
    """y in the residual's place: few tokens, small products, splits of the inner axis, and large ones."""
    a = Layer(dt, "linear_reduce", rows, dim, features, seed=9)
    with group(2) as g:
        want = a.forward(g)
        a.check_forward(want)
        a.forward(g, y=a.res)
        assert all(torch.equal(got, w) for got, w in zip(a.res, want))


@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
@pytest.mark.parametrize("rows,dim,features", [([1, 0], 424, [192, 100]), ([3, 2], 70, [33, 500]), ([60, 40], 200, [96, 24])])
def test_small_gradients_are_as_near_as_their_rounding(dt, act, rows, dim, features):
    """The gradient before the activation enters small products as its rounding and what that left: off by
    2^-17 of itself, and by what the derivative is off, 2^-16."""
    a = Layer(dt, "gather_linear", rows, dim, features, seed=17)
    with group(2) as g:
        dx, dw, _ = a.backward(g, act)
    G = torch.cat([d.double() * slope64(v.double(), act) for d, v in zip(a.dy, a.pre)], 1)
    M = torch.cat([d.double().abs() * 1.2 for d in a.dy], 1)   # a derivative is 1.13 at most
    X, W = torch.cat(a.x).double(), torch.cat(a.w).double()
    near = lambda k: 2.0 ** -16 + 2.0 ** -17 + sum_error(2 * k, 2)
    check(torch.cat(dx), G @ W, near(sum(features)) * (M @ W.abs()), "dx")
    check(torch.cat(dw), G.t() @ X, near(sum(rows)) * (M.t() @ X.abs()), "dw")


@pytest.mark.parametrize("which", WHICH)
def test_two_calls_at_once(dt, which):
    """Calls on two streams, each with its own workspace and outputs, as a group's calls may run."""
    layers = [Layer(dt, which, [300, 212], 520, [600, 136], seed=s) for s in (31, 32)]
    with group(2) as g:
        streams = [torch.cuda.Stream() for _ in layers]
        torch.cuda.synchronize()
        outs = []
        for _ in range(3):
            for a, s in zip(layers, streams):
                with torch.cuda.stream(s):
                    outs.append((a, a.forward(g), a.backward(g)))
        torch.cuda.synchronize()
        for a, fwd, bwd in outs:
            a.check_forward(fwd)
            a.check_backward(bwd)
        assert dt.dt_group_check(g) == dt.DT_OK


def test_many_tokens_of_few_features_and_a_long_inner_axis(dt):
    """More rows than a grid has in its second dimension, where splits of the inner axis would pay."""
    rows, dim, features = [60001, 5999], 16384, [200, 0]
    layer = Layer(dt, "gather_linear", rows, dim, features, bias=False)
    with group(2) as g:
        pre, y = layer.forward(g)
    x = torch.cat(layer.x)
    some = torch.cat([torch.arange(0, 80), torch.arange(32700, 32800), torch.arange(59990, 60010),
                      torch.arange(65500, 66000)]).cuda()
    want = x[some].double() @ layer.w[0].double().T
    tol = sum_error(dim, 2) * (x[some].double().abs() @ layer.w[0].double().abs().T)
    check(y[0][some], want, tol, "y")
    check(pre[0][some], want, tol, "pre")


def test_ends_of_the_activations(dt):
    """Zeros, infinities and NaN before each activation: relu and gelu of infinities are their limits (gelu
    of minus infinity 0), a NaN stays one, and silu of minus infinity is no number, as its formula says."""
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([0.0, -0.0, inf, -inf, nan, 300.0, -300.0, 1e-30], device="cuda").to(BF16)
    for n in (8, 40, 20000):   # tokens of one column: a kernel each
        with group(1) as g:
            for act in ACTS:
                X = x[torch.arange(n, device="cuda") % 8][:, None].contiguous()
                y = torch.empty(n, 8, dtype=BF16, device="cuda")
                ws = workspace(dt, "gather_linear", g, [n], 1, [8], False)
                dt.dt_gather_linear(g, [X], [torch.ones(8, 1, dtype=BF16, device="cuda")], None, None, [y], [n], 0, 1, [8], 0,
                                    "bf16", act, ws)
                want = act64(X.double(), act).repeat(1, 8)
                if act == "gelu":
                    want[X[:, 0] == -inf] = 0.0
                assert torch.equal(y.isnan(), want.isnan())
                ok = ~want.isnan()
                assert torch.equal(y.double().isinf()[ok], want.isinf()[ok])
                fin = ok & ~want.isinf()
                assert ((y.double() - want).abs()[fin] <= (2 * R * want.abs() + 1e-37)[fin]).all()


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("rows", [[1], [2, 0, 3], [7, 5], [16]])
@pytest.mark.parametrize("long,short", [(4096, 64), (9001, 33), (33000, 40), (20000, 1000)])
def test_few_tokens_of_a_long_inner_axis(dt, which, rows, long, short):
    """Single tokens whose inner axis is shared by the CTAs of a cluster."""
    P = len(rows)
    cut = lambda n: [n * (r + 1) // P - n * r // P for r in range(P)]
    dim, features = (long, cut(short)) if which == "gather_linear" else (short, cut(long))
    a = Layer(dt, which, rows, dim, features, seed=long)
    with group(P) as g:
        a.check_forward(a.forward(g, "relu") if which == "gather_linear" else a.forward(g), "relu")
        assert dt.dt_group_check(g) == dt.DT_OK
