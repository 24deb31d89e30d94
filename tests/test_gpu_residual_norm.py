"""The residual norm and its gradient against their definitions in 64 bits.

Tolerances, with u = 2^-24.  A row's sum is made of chains of at most 16 additions a thread (rows too
long for registers: cols / 512) and a tree: M = 64 + cols / 256 roundings at most, each relative to
the sum of magnitudes.  From there errors are carried through the formulas to first order, with a few
roundings for the operations of each (the reciprocal square root is off by 2 ulp).  A column's sum over
n rows is at most n + 64 roundings.  A result is rounded to its type once: half an ulp, eps / 2 of it.
"""
from __future__ import annotations

import pytest
import torch

from gpu_util import group

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def dt():
    from same_device_collective_gb300 import dt as mod
    assert torch.cuda.is_available()
    return mod


def made(gen, shape, dtype, offset, std=1.0, mean=0.0):
    n = shape if isinstance(shape, int) else shape[0] * shape[1]
    t = torch.empty(n + offset, dtype=TYPES[dtype], device="cuda")[offset:].view(shape)
    return t.copy_(torch.randn(shape, generator=gen, device="cuda") * std + mean)


def check(got, want, tol, what):
    half = torch.finfo(got.dtype).eps / 2
    bad = ~((got.double() - want).abs() <= tol * 1.01 + half * want.abs() + 1e-37)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], want[bad][:4], tol.expand_as(want)[bad][:4])


class Rows:
    def __init__(self, dt, rows, cols, dtype="bf16", wdtype="f32", seed=0, offset=0, scale=0.75, weights="abc", dy=True):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.dt, self.rows, self.cols, self.dtype, self.wdtype, self.scale, self.offset = dt, rows, cols, dtype, wdtype, scale, offset
        m = lambda std, mean=0.0: [made(gen, (k, cols), dtype, offset, std, mean) for k in rows]
        self.x, self.branch, self.dy, self.dz = m(1.5, 0.3), m(0.3), m(1.0) if dy else None, m(0.7)
        w = lambda c, std, mean: made(gen, cols, wdtype, offset, std, mean) if c in weights else None
        self.post, self.gate, self.pre = w("a", 0.2, 1.0), w("b", 0.4, 0.5), w("c", 0.2, 1.0)
        self.y = m(1.2)
        for y, x in zip(self.y, self.x):
            y.add_(x * 0.5)
        self.r1 = [torch.rsqrt(b.double().square().mean(1) + EPS).float() for b in self.branch]
        self.r2 = [torch.rsqrt(b.double().square().mean(1) + EPS).float() for b in self.y]

    def like(self, ts):
        return [torch.full((t.numel() + self.offset,), 7.0, dtype=t.dtype, device="cuda")[self.offset:].view(t.shape) for t in ts]

    def forward(self, g, y=None, z=None, stats=True, stream=None):
        y, z = y or self.like(self.x), z or self.like(self.x)
        r1, r2 = ([torch.full((k,), 7.0, device="cuda") for k in self.rows] if stats else None for _ in range(2))
        self.dt.dt_residual_norm(g, self.x, self.branch, self.post, self.gate, self.pre, self.scale, y, z, r1, r2, self.rows, 0,
                                 self.cols, EPS, self.dtype, self.wdtype, stream)
        return y, z, r1, r2

    def backward(self, g, dx=None, do=None, op="sum", stream=None, want="abc"):
        dx, do = dx or self.like(self.y), do or self.like(self.y)
        w = [torch.full((self.cols + self.offset,), 7.0, dtype=TYPES[self.wdtype], device="cuda")[self.offset:] if c in want else None
             for c in "abc"]
        ws = torch.full((self.dt.dt_residual_norm_workspace(g, self.cols),), 0xA5, dtype=torch.uint8, device="cuda") if want else None
        self.dt.dt_residual_norm_backward(g, self.branch, self.y, self.dy, self.dz, self.post, self.gate, self.pre, self.scale,
                                          self.r1, self.r2, dx, do, *w, self.rows, 0, self.cols, self.dtype, self.wdtype, op, ws,
                                          stream)
        return dx, do, w

    def weights64(self):
        one = torch.ones(self.cols, dtype=torch.float64, device="cuda")
        return [one if w is None else w.double() for w in (self.post, self.gate, self.pre)]

    def check_forward(self, out, x=None, branch=None):
        y, z, r1, r2 = out
        post, gate, pre = self.weights64()
        x, o = torch.cat(x or self.x).double(), torch.cat(branch or self.branch).double()
        M = 64 + self.cols / 256
        w1 = 1 / torch.sqrt(o.square().mean(1, keepdim=True) + EPS)
        e1 = (M / 2 + 4) * U
        gh = gate * post * o * w1
        wy = self.scale * x + gh
        ty = gh.abs() * (e1 + 4 * U) + 3 * U * ((self.scale * x).abs() + wy.abs())
        w2 = 1 / torch.sqrt(wy.square().mean(1, keepdim=True) + EPS)
        e2 = (M / 2 + 4) * U + ty.norm(dim=1, keepdim=True) / wy.norm(dim=1, keepdim=True).clamp(min=1e-30)
        wz = wy * w2 * pre
        check(torch.cat(y), wy, ty, "y")
        check(torch.cat(z), wz, (pre * w2).abs() * ty + wz.abs() * (e2 + 4 * U), "z")
        if r1:
            check(torch.cat(r1), w1[:, 0], w1[:, 0] * e1, "rstd post")
            check(torch.cat(r2), w2[:, 0], w2[:, 0] * e2[:, 0], "rstd pre")

    def check_backward(self, out, op="sum", dy=None, dz=None):
        dx, do, (dpost, dgate, dpre) = out
        post, gate, pre = self.weights64()
        o, y = torch.cat(self.branch).double(), torch.cat(self.y).double()
        z = torch.cat(dz or self.dz).double()
        dy = dy or self.dy
        dyv = torch.cat(dy).double() if dy else torch.zeros_like(z)
        r1, r2 = torch.cat(self.r1).double()[:, None], torch.cat(self.r2).double()[:, None]
        M, n = 64 + self.cols / 256, y.shape[0]
        mean = lambda v: v.mean(1, keepdim=True)
        q, g = z * pre, gate * post * o
        m2, tm2 = r2 * mean(q * y), (M + 4) * U * r2 * mean((q * y).abs())
        d = dyv + r2 * q - y * r2 ** 2 * m2
        td = 5 * U * (dyv.abs() + (r2 * q).abs() + (y * r2 ** 2 * m2).abs()) + (y * r2 ** 2).abs() * tm2
        c = d * gate * post
        ch = r1 * mean(c * o)
        tch = (M + 8) * U * r1 * mean((g * dyv).abs() + (r2 * g * q).abs() + (r2 ** 2 * m2 * g * y).abs()) \
            + r1 * r2 ** 2 * tm2 * mean((g * y).abs())
        check(torch.cat(dx), self.scale * d, abs(self.scale) * td + 2 * U * (self.scale * d).abs(), "dx")
        wo = r1 * c - o * r1 ** 2 * ch
        check(torch.cat(do), wo, r1 * (gate * post).abs() * td + o.abs() * r1 ** 2 * tch
              + 6 * U * ((r1 * c).abs() + (o * r1 ** 2 * ch).abs()), "dbranch")
        h, nn = o * r1, y * r2
        by = len(self.rows) if op == "avg" else 1
        G, tG = (d * h).sum(0) / by, ((h.abs() * td + (n + 64) * U * (d * h).abs()).sum(0)) / by
        if dpost is not None:
            check(dpost, G * gate, tG * gate.abs() + 4 * U * (G * gate).abs(), "dpost")
        if dgate is not None:
            check(dgate, G * post, tG * post.abs() + 4 * U * (G * post).abs(), "dgate")
        if dpre is not None:
            check(dpre, (z * nn).sum(0) / by, (n + 64) * U * (z * nn).abs().sum(0) / by, "dpre")


# single rows, ranks without rows, a column, odd widths, widths of few lanes, of a warp, of several, past 4096 and 8192
SHAPES = [([1], 1), ([1, 1], 8), ([2, 0, 1], 3), ([1, 1, 1, 1], 4096), ([5, 300], 64), ([700, 1], 128), ([40], 100),
          ([33, 0, 90], 257), ([200, 77], 512), ([600, 600, 600], 777), ([64], 1024), ([31, 2], 2048), ([1, 1000], 2056),
          ([17], 4095), ([150, 9], 4096), ([5], 4104), ([12, 3], 8192), ([7], 8000), ([3, 2], 8193), ([2], 20000), ([160], 16384)]


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows,cols", SHAPES, ids=str)
def test_both_passes(dt, rows, cols, dtype, wdtype):
    a = Rows(dt, rows, cols, dtype, wdtype, seed=cols)
    with group(len(rows)) as g:
        a.check_forward(a.forward(g))
        a.check_backward(a.backward(g))
        assert dt.dt_group_check(g) == dt.DT_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offset", [1, 2, 4])
@pytest.mark.parametrize("cols", [8, 64, 1000, 4096])
def test_rows_off_a_vector_boundary(dt, dtype, offset, cols):
    a = Rows(dt, [3, 50], cols, dtype, dtype, seed=offset, offset=offset)
    with group(2) as g:
        a.check_forward(a.forward(g))
        a.check_backward(a.backward(g))


@pytest.mark.parametrize("weights", ["", "a", "b", "c", "bc"])
@pytest.mark.parametrize("dy", [True, False])
def test_without_weights_or_a_later_gradient(dt, weights, dy):
    a = Rows(dt, [9, 20], 320, "bf16", "f32", seed=5, weights=weights, dy=dy, scale=1.0)
    with group(2) as g:
        a.check_forward(a.forward(g, stats=False))
        a.check_backward(a.backward(g, op="avg"), op="avg")
        a.check_backward(a.backward(g, want="b"))
        a.check_backward(a.backward(g, want=""))


@pytest.mark.parametrize("scale", [0.0, -2.0])
def test_scale(dt, scale):
    a = Rows(dt, [9], 96, "f32", "f32", seed=6, scale=scale)
    with group(1) as g:
        a.check_forward(a.forward(g))
        a.check_backward(a.backward(g))


@pytest.mark.parametrize("cols", [64, 777, 4096, 9000])
def test_in_place(dt, cols):
    a = Rows(dt, [40, 3], cols, "bf16", "bf16", seed=7)
    x, branch, dy, dz = ([t.clone() for t in v] for v in (a.x, a.branch, a.dy, a.dz))
    with group(2) as g:
        want = a.forward(g)
        got = a.forward(g, y=a.x, z=a.branch)
        for p, q in zip(got, want):
            assert all(torch.equal(s, t) for s, t in zip(p, q))
        a.branch = branch
        want = a.backward(g)
        got = a.backward(g, dx=a.dy, do=a.dz)
        for p, q in zip(got, want):
            assert all(torch.equal(s, t) for s, t in zip(p, q))
        a.check_backward(got, dy=dy, dz=dz)


@pytest.mark.parametrize("cols", [8, 96, 777, 4096, 9000])
def test_a_bad_row_stays_alone(dt, cols):
    a = Rows(dt, [30, 11], cols, "bf16", "f32", seed=8)
    with group(2) as g:
        clean = [torch.cat(t) for t in a.forward(g)[:2]]
        cd = [torch.cat(t) for t in a.backward(g)[:2]]
        a.x[0][4, cols // 2] = float("nan")
        a.branch[1][3, 0] = float("inf")
        a.dz[0][7, cols - 1] = float("nan")
        keep = torch.ones(41, dtype=torch.bool, device="cuda")
        keep[[4, 33]] = False
        for got, want in zip(a.forward(g)[:2], clean):
            got = torch.cat(got)
            assert torch.equal(got[keep], want[keep])
        y, z, _, _ = a.forward(g)
        assert z[0][4].isnan().all() and z[1][3].isnan().all()
        a.branch[1][3, 0] = 0.5
        dx, do, _ = a.backward(g)
        keep = torch.ones(41, dtype=torch.bool, device="cuda")
        keep[[7, 33]] = False
        for got, want in zip((dx, do), cd):
            assert torch.equal(torch.cat(got)[keep], want[keep])
        assert dx[0][7].isnan().all() and do[0][7].isnan().all()


def test_a_row_of_zeros(dt):
    a = Rows(dt, [6], 200, "bf16", "f32", seed=9)
    a.branch[0][2] = 0
    a.x[0][3] = 0
    with group(1) as g:
        a.check_forward(a.forward(g))


def test_no_rows(dt):
    a = Rows(dt, [0, 0], 64, seed=1)
    with group(2) as g:
        a.forward(g)
        for w in a.backward(g)[2]:
            assert (w == 0).all()


@pytest.mark.parametrize("rows,cols", [([1, 1], 4096), ([300, 20], 1000)])
def test_captured_replayed_and_on_another_stream(dt, rows, cols):
    a, b = Rows(dt, rows, cols, seed=1), Rows(dt, rows, cols, seed=2)
    with group(2) as g:
        want = [b.forward(g), b.backward(g)]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            again = [b.forward(g), b.backward(g)]
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = [a.forward(g), a.backward(g)]
        for name in ("x", "branch", "dy", "dz", "y", "r1", "r2"):
            for t, v in zip(getattr(a, name), getattr(b, name)):
                t.copy_(v)
        for name in ("post", "gate", "pre"):
            getattr(a, name).copy_(getattr(b, name))
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()

        def flat(v):
            return [t for u in v for t in flat(u)] if isinstance(v, (list, tuple)) else [v]
        for other in (got, again):
            assert all(torch.equal(p, q) for p, q in zip(flat(other), flat(want)))


def test_gradients_against_differences(dt):
    """f32 throughout: the loss' change over a step along each input's own gradient.  The difference of
    the two losses is off by the third derivative's part, (step / size)^2 of the change, and by the
    losses' own roundings, 2^-20 of a loss' terms over the step."""
    a = Rows(dt, [5, 3], 48, "f32", "f32", seed=3)
    with group(2) as g:
        def loss():
            y, z, r1, r2 = a.forward(g)
            a.y, a.r1, a.r2 = y, r1, r2
            return sum(float((t.double() * w.double()).sum()) for t, w in zip(y + z, a.dy + a.dz))
        loss()
        dx, do, dw = a.backward(g)
        for at, grad in ((a.x, dx), (a.branch, do), ([a.post], [dw[0]]), ([a.gate], [dw[1]]), ([a.pre], [dw[2]])):
            size = float(torch.cat([t.double().reshape(-1) for t in grad]).norm())
            keep = [t.clone() for t in at]
            ends = []
            for sign in (1, -1):
                for t, k, d in zip(at, keep, grad):
                    t.copy_(k.double() + sign * 1e-2 * d.double() / size)
                ends.append(loss())
            for t, k in zip(at, keep):
                t.copy_(k)
            assert abs((ends[0] - ends[1]) / 2e-2 - size) <= 0.01 * size


def test_refusals(dt):
    a = Rows(dt, [4, 2], 16, "bf16", "f32", seed=1)
    with group(2) as g:
        def call(back=False, status=dt.DT_ERR_INVALID, **change):
            args = dict(g=g, branch=a.branch, post_weight=a.post, gate=a.gate, pre_weight=a.pre, residual_scale=1.0,
                        rstd_post=a.r1, rstd_pre=a.r2, rows=a.rows, rows_equal=0, cols=16, dtype="bf16", weight_dtype="f32")
            if back:
                args.update(y=a.y, dy=a.dy, dz=a.dz, dx=a.like(a.y), dbranch=a.like(a.y), dpost_weight=torch.empty(16, device="cuda"),
                            dgate=torch.empty(16, device="cuda"), dpre_weight=torch.empty(16, device="cuda"), op="sum",
                            workspace=torch.empty(dt.dt_residual_norm_workspace(g, 16), dtype=torch.uint8, device="cuda"))
            else:
                args.update(x=a.x, y=a.like(a.x), z=a.like(a.x), eps=EPS, rstd_post=None, rstd_pre=None)
            args.update({k: v(args) if callable(v) else v for k, v in change.items()})
            fn = dt.dt_residual_norm_backward if back else dt.dt_residual_norm
            if status == dt.DT_OK:
                return fn(**args)
            with pytest.raises(dt.DtError) as e:
                fn(**args)
            assert e.value.status == status

        for back in (False, True):
            call(back, dt.DT_OK)
            call(back, cols=0)
            call(back, cols=(1 << 24) + 1)
            call(back, residual_scale=float("nan"))
            call(back, residual_scale=float("inf"))
            call(back, rows=[1 << 62, 2])
            call(back, branch=[None, a.branch[1]])
        for eps in (-1.0, float("nan"), float("inf")):
            call(eps=eps)
        call(z=lambda k: k["y"])
        call(y=lambda k: k["branch"])
        call(z=lambda k: k["x"])
        call(y=lambda k: [k["y"][0], k["y"][0][1:3]])
        call(False, dt.DT_OK, rstd_post=[a.like(a.r1)[0], None])   # a rank whose reciprocals are not wanted
        call(True, workspace=None)
        call(True, workspace=lambda k: k["workspace"][16:])
        call(True, workspace=lambda k: (k["workspace"].data_ptr() + 4, 1 << 30))
        call(True, dx=lambda k: k["dz"])
        call(True, dbranch=lambda k: k["branch"])
        call(True, dgate=lambda k: k["dpre_weight"])
        call(True, dz=[None, a.dz[1]])
        call(True, rstd_pre=[None, a.r2[1]])
        call(True, dt.DT_ERR_UNSUPPORTED, op="max")
        call(True, op=9)
        call(True, dt.DT_OK, dpost_weight=None, dgate=None, dpre_weight=None, workspace=None)
        with pytest.raises(ValueError):
            call(x=[t.float() for t in a.x])
        with pytest.raises(ValueError):
            call(gate=a.gate.bfloat16())
        with pytest.raises(ValueError):
            call(x=a.x[:1])
        assert dt.dt_residual_norm_workspace(g, 0) == 0
        assert dt.dt_group_check(g) == dt.DT_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [([500, 1, 200], 8192), ([700], 4104), ([400, 9], 5001), ([1000], 101), ([3, 400], 8191),
                                       ([20000], 8), ([5000, 3000], 24), ([160, 200], 20000)])
def test_many_rows_of_other_widths(dt, rows, cols, dtype):
    a = Rows(dt, rows, cols, dtype, "f32", seed=cols)
    with group(len(rows)) as g:
        a.check_forward(a.forward(g))
        a.check_backward(a.backward(g))
        assert dt.dt_group_check(g) == dt.DT_OK
