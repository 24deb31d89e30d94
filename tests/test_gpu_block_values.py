"""What the header says of values at the ends: NaN, infinities and squares past fp32's range in the residual
norm's rows, for each of its kernels (few rows, rings of vectors and of single elements, rows too long for
registers), and what the tensor cores cut off of the linear layers' sums."""
from __future__ import annotations

import pytest
import torch

from gpu_util import group
from test_gpu_linear import workspace
from test_gpu_residual_norm import EPS, Rows

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
# a case to a row: the input, the value
CASES = [("x", INF), ("x", -INF), ("x", NAN), ("branch", INF), ("branch", -INF), ("branch", NAN)]


@pytest.fixture(scope="module")
def dt():
    from same_device_collective_gb300 import dt as mod
    assert torch.cuda.is_available()
    return mod


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [8, 96, 777, 4096, 9000])
@pytest.mark.parametrize("rows", [[5, 6], [700, 5]], ids=str)
def test_a_value_that_is_not_finite(dt, rows, cols, dtype):
    a = Rows(dt, rows, cols, dtype, "f32", seed=3)
    j = cols // 3
    with group(2) as g:
        clean = [torch.cat(t) for t in a.forward(g)]
        n = rows[0]
        at = [(0, 1), (0, n - 1), (1, 0), (1, 1), (1, 3), (1, 4)]
        for (name, v), (r, i) in zip(CASES, at):
            getattr(a, name)[r][i, j] = v
        y, z, r1, r2 = (torch.cat(t) for t in a.forward(g))
        assert dt.dt_group_check(g) == dt.DT_OK
    rest = torch.ones(sum(rows), dtype=torch.bool, device="cuda")
    other = torch.arange(cols, device="cuda") != j
    scaled = a.scale * torch.cat(a.x).double()
    half = torch.finfo(y.dtype).eps / 2
    for (name, v), (r, i) in zip(CASES, at):
        k = i + r * n
        rest[k] = False
        if name == "x":
            assert torch.equal(y[k][other], clean[0][k][other]) and r1[k] == clean[2][k]
            if v != v:
                assert y[k, j].isnan() and z[k].isnan().all() and r2[k].isnan()
            else:
                assert y[k, j] == v and z[k, j].isnan() and (z[k][other] == 0).all() and r2[k] == 0
        elif v != v:
            assert y[k].isnan().all() and z[k].isnan().all() and r1[k].isnan() and r2[k].isnan()
        else:
            # (scale x is rounded to fp32 and to the rows' type)
            off = (y[k].double() - scaled[k]).abs()[other]
            assert r1[k] == 0 and y[k, j].isnan() and (off <= (half + 2.0 ** -23) * scaled[k].abs()[other]).all()
            assert z[k].isnan().all() and r2[k].isnan()
    for got, want in zip((y, z, r1, r2), clean):
        assert torch.equal(got[rest], want[rest])


@pytest.mark.parametrize("cols", [8, 777, 4096, 9000])
@pytest.mark.parametrize("rows", [3, 400])
def test_squares_past_the_range(dt, rows, cols):
    """Rows of 1e20, and with an eps of 0 rows of zeros and of 1e-30."""
    a = Rows(dt, [rows], cols, "f32", "f32", seed=4)
    with group(1) as g:
        clean = a.forward(g)
        a.branch[0][0], a.x[0][1] = 1e20, 1e20
        y, z, r1, r2 = (t[0] for t in a.forward(g))
        assert r1[0] == 0 and r2[1] == 0 and (z[1] == 0).all() and y.isfinite().all()
        assert ((y[0].double() - a.scale * a.x[0][0].double()).abs() <= 2.0 ** -23 * a.scale * a.x[0][0].abs()).all()
        for got, want in zip((y, z, r1, r2), clean):
            assert torch.equal(got[2:], want[0][2:])
        a.branch[0][0], a.branch[0][1] = 0, 1e-30
        y, z, r1, r2 = (torch.empty_like(t) for t in (y, z, r1, r2))
        dt.dt_residual_norm(g, a.x, a.branch, a.post, a.gate, a.pre, a.scale, [y], [z], [r1], [r2], [rows], 0, cols, 0.0,
                            "f32", "f32")
        assert (r1[:2] == INF).all() and y[0].isnan().all() and y[1].isinf().all()
        # other rows, with the least eps that matters nowhere
        o, x = a.branch[0][2:].double(), a.x[0][2:].double()
        want = a.scale * x + a.gate.double() * a.post.double() * o / o.square().mean(1, keepdim=True).sqrt()
        if rows > 2:
            tol = 2.0 ** -24 * (64 + cols / 256 + 16)   # (a row's sum, and a few operations)
            assert ((y[2:].double() - want).abs() <= tol * (want.abs() + (a.scale * x).abs() + (want - a.scale * x).abs())).all()


@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [8, 777, 4096, 9000])
def test_backward_of_a_value_that_is_not_finite(dt, cols, dtype, value):
    """It reaches its own row's dx and dbranch only, and the weights' gradients."""
    a = Rows(dt, [40, 9], cols, dtype, "f32", seed=5)
    with group(2) as g:
        clean = [torch.cat(t) for t in a.backward(g)[:2]]
        rest = torch.ones(49, dtype=torch.bool, device="cuda")
        for k, name in enumerate(("branch", "y", "dy", "dz")):
            getattr(a, name)[k % 2][3 + k, cols - 1] = value
            rest[3 + k + 40 * (k % 2)] = False
        dx, do = (torch.cat(t) for t in a.backward(g)[:2])
    for got, want in zip((dx, do), clean):
        assert torch.equal(got[rest], want[rest])
    finite = lambda t: t.isfinite()
    assert torch.equal(dx[3], clean[0][3]) and not finite(do[3]).any()              # branch
    assert not finite(dx[44]).any() and not finite(do[44]).any()                    # y
    assert torch.equal(dx[5][:-1], clean[0][5][:-1]) and not finite(dx[5, -1]) and not finite(do[5]).any()   # dy
    assert not finite(dx[46]).any() and not finite(do[46]).any()                    # dz


@pytest.mark.parametrize("terms", ["uniform", "small"])
@pytest.mark.parametrize("n,features,dim", [(2048, 4096, 16384), (300, 200, 65536), (64, 64, 2048), (4, 4096, 16384)])
def test_sums_of_one_sign(dt, n, features, dim, terms):
    """Sums that a bias takes off again, so that the result shows their error: terms of one size, and terms
    of one to two quarters of the last place of the 1 that they follow.  A term loses 2^-25 of the
    largest part sum at most, here the sum; a sum's splits, the bias and the conversions take 64 roundings
    of 2^-23 of it, and the result is rounded to bf16."""
    gen = torch.Generator("cuda").manual_seed(dim)
    x, w = (torch.rand(k, dim, generator=gen, device="cuda") for k in (n, features))
    if terms == "small":
        x, w = torch.ones_like(x), (1 + w) * 2.0 ** -25
        w[:, 0] = 1
    x, w = x.bfloat16(), w.bfloat16()
    exact = x[:8].double() @ w.double().t()
    bias = (-exact[0]).bfloat16()
    y = torch.empty(n, features, dtype=torch.bfloat16, device="cuda")
    with group(1) as g:
        ws = workspace(dt, "gather_linear", g, [n], dim, [features], False)
        dt.dt_gather_linear(g, [x], [w], [bias], None, [y], [n], 0, dim, [features], 0, "bf16", "none", ws)
        assert dt.dt_group_check(g) == dt.DT_OK
    want = exact + bias.double()
    off = (y[:8].double() - want).abs()
    assert (off <= (dim * 2.0 ** -25 + 64 * 2.0 ** -23) * exact + 2.0 ** -8 * want.abs()).all()
    if terms == "uniform":   # what the header calls usual, with half of it to spare
        assert (off <= (dim * 7.5e-9 + 64 * 2.0 ** -23) * exact + 2.0 ** -8 * want.abs()).all()


@pytest.mark.parametrize("act,least", [("gelu", 1.2e-38), ("silu", 1.1e-36)])
@pytest.mark.parametrize("n", [4, 70, 3000])
def test_far_below_zero(dt, n, act, least):
    """Every bf16 value from -120 to -2: an activation's exponential is off by 2^-16 of itself, its result is
    rounded to bf16, and what lies below `least` may be 0."""
    v = torch.arange(-2 ** 15, 0, device="cuda").to(torch.int16).view(torch.bfloat16)
    v = v[(v >= -120) & (v <= -2)]
    x = torch.ones(n, 1, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(n, len(v), dtype=torch.bfloat16, device="cuda")
    with group(1) as g:
        ws = workspace(dt, "gather_linear", g, [n], 1, [len(v)], False)
        dt.dt_gather_linear(g, [x], [v[:, None].contiguous()], None, None, [y], [n], 0, 1, [len(v)], 0, "bf16", act, ws)
    d = v.double()
    want = d * torch.exp(torch.special.log_ndtr(d)) if act == "gelu" else d * torch.sigmoid(d)
    assert ((y.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -15) * want.abs() + least).all() and (y <= 0).all()
