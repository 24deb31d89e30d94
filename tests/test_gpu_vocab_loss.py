"""Vocabulary-parallel softmax cross entropy against its definition in 64 bits.

Tolerances, with u = 2^-23 (the tensor cores' fp32 sums may truncate).  A sum
over K products is made in steps of 16, each rounded once: (K / 16 + 16) u times
the sum of magnitudes.  That is the error of a logit (`dl`).  A sum of
exponentials adds at most 256 columns one by one, then at most 64 + 32 partial
sums: 2^-15 covers it, relatively, so absolutely in its logarithm.  A
probability is off by its logit's error and by 2^-18 (the scaled exponent's and
the power's roundings at logits up to 32); p - [target] is then rounded to
bf16 (half an ulp of 8 significant bits: 2^-8 of itself), and the gradients add
the products' summation error and one more such rounding.
"""
from __future__ import annotations

import pytest
import torch

from gpu_util import group

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
IGNORE = -100


@pytest.fixture(scope="module")
def dt():
    from same_device_collective_gb300 import dt as mod
    assert torch.cuda.is_available()
    return mod


def rows_at(n, dim, offset, gen, std):
    """[n, dim] bf16 that starts `offset` elements into its allocation."""
    base = torch.empty(n * dim + offset, dtype=torch.bfloat16, device="cuda")
    t = base[offset:].view(n, dim)
    t.copy_(torch.randn(n, dim, generator=gen, device="cuda") * std)
    return t


def make(tokens, vocab, dim, seed, offset=0, std=None, drop=0.2):
    gen = torch.Generator("cuda").manual_seed(seed)
    h = rows_at(tokens, dim, offset, gen, 1.0)
    w = [rows_at(v, dim, offset, gen, std or 2.0 / dim ** 0.5) for v in vocab]
    t = torch.randint(0, sum(vocab), (tokens,), generator=gen, device="cuda", dtype=torch.int32)
    t[torch.rand(tokens, generator=gen, device="cuda") < drop] = IGNORE
    return h, w, t


def forward(dt, g, h, w, t, op="avg", ignore=IGNORE, stream=None, vocab=None, equal=0):
    n, dim = h.shape
    vocab = [x.shape[0] for x in w] if vocab is None and not equal else vocab
    losses, lse = (torch.full((n,), 9.0, device="cuda") for _ in range(2))
    loss = torch.full((1,), 9.0, device="cuda")
    ws = torch.empty(dt.dt_vocab_loss_workspace(g, vocab, equal, n, dim, "bf16", False), dtype=torch.uint8, device="cuda")
    ws.fill_(0xA5)
    dt.dt_vocab_loss(g, h, w, vocab, equal, t, n, dim, "bf16", op, ignore, losses, lse, loss, ws, stream)
    return losses, lse, loss


def backward(dt, g, h, w, t, lse, grad=None, op="avg", ignore=IGNORE, stream=None, offset=0):
    n, dim = h.shape
    vocab = [x.shape[0] for x in w]

    def like(x):
        return torch.full((x.numel() + offset,), 7.0, dtype=x.dtype, device="cuda")[offset:].view(x.shape)

    dh, dw = like(h), [like(x) for x in w]
    ws = torch.empty(dt.dt_vocab_loss_workspace(g, vocab, 0, n, dim, "bf16", True), dtype=torch.uint8, device="cuda")
    ws.fill_(0xA5)
    dt.dt_vocab_loss_backward(g, h, w, vocab, 0, t, lse, grad, n, dim, "bf16", op, ignore, dh, dw, ws, stream)
    return dh, dw


def sum_error(k):
    return (k / 16 + 16) * U


def logits(h, w):
    """Logits in 64 bits, and how far they may be off."""
    h, w = h.double(), torch.cat(w).double()
    return h @ w.t(), sum_error(h.shape[1]) * (h.abs() @ w.abs().t())


def check_forward(h, w, t, losses, lse, loss, op="avg", ignore=IGNORE):
    l, dl = logits(h, w)
    want = torch.logsumexp(l, 1)
    tol = dl.amax(1) + 2.0 ** -15 + 8 * U * want.abs()
    assert ((lse.double() - want).abs() <= tol).all()
    keep = t != ignore
    at = l.gather(1, torch.where(keep, t, 0).long()[:, None])[:, 0]
    each = torch.where(keep, want - at, 0.0)
    tol = torch.where(keep, 2 * tol + 8 * U * at.abs(), 0.0)
    assert ((losses.double() - each).abs() <= tol).all()
    div = max(1, int(keep.sum())) if op == "avg" else 1
    assert abs(float(loss) - float(each.sum()) / div) <= float(tol.sum()) / div + 4 * U * abs(float(each.sum())) / div


def check_backward(h, w, t, lse, dh, dw, grad=1.0, op="avg", ignore=IGNORE):
    l, dl = logits(h, w)
    keep = (t != ignore)[:, None]
    p = torch.exp(l - lse.double()[:, None])
    g = p.clone()
    rows = torch.arange(len(t), device="cuda")
    g[rows, torch.where(keep[:, 0], t, 0).long()] -= 1
    g *= keep
    off = (2.0 ** -8 * g.abs() + p * (dl + 2.0 ** -18) * 1.01) * keep
    c = grad / max(1, int(keep.sum())) if op == "avg" else grad
    wd, hd = torch.cat(w).double(), h.double()
    want = c * (g @ wd)
    tol = abs(c) * (off @ wd.abs() + sum_error(len(wd)) * (g.abs() @ wd.abs())) + 2.0 ** -8 * want.abs()
    assert ((dh.double() - want).abs() <= tol).all()
    want = c * (g.t() @ hd)
    tol = abs(c) * (off.t() @ hd.abs() + sum_error(len(t)) * (g.abs().t() @ hd.abs())) + 2.0 ** -8 * want.abs()
    assert ((torch.cat(dw).double() - want).abs() <= tol).all()


CASES = [
    # tokens, vocabulary rows per rank, dim, element offset
    (1, [1], 1, 0), (1, [7], 8, 0), (3, [2, 0, 5], 5, 0), (1, [300, 300], 64, 0), (64, [256], 64, 0),
    (65, [257, 1], 72, 0), (128, [512, 512], 128, 0), (129, [100, 900, 0, 24], 200, 0), (77, [1000, 3000, 6007], 500, 0),
    (300, [2048] * 4, 256, 0), (300, [2048] * 4, 256, 1), (200, [1111, 2222], 333, 0), (40, [64] * 16, 1000, 3),
    (1000, [6000, 6001], 128, 0), (1, [40000], 1024, 0), (17, [20000, 12000], 768, 0), (513, [4096] * 8, 1024, 0),
    (2500, [3000], 96, 0), (256, [700, 800], 256, 0), (257, [700, 800], 264, 0), (192, [50, 3000], 129, 0),
    # the vocabulary in several pieces: by p - [target]'s size, and by that of rows laid out again
    (2048, [70000, 70001], 64, 0), (300, [9000, 11000], 4100, 0),
]


@pytest.mark.parametrize("tokens,vocab,dim,offset", CASES)
def test_both_passes(dt, tokens, vocab, dim, offset):
    h, w, t = make(tokens, vocab, dim, seed=tokens + dim, offset=offset)
    grad = torch.tensor([1.75], device="cuda")
    with group(len(vocab)) as g:
        losses, lse, loss = forward(dt, g, h, w, t)
        check_forward(h, w, t, losses, lse, loss)
        dh, dw = backward(dt, g, h, w, t, lse, grad, offset=offset)
        check_backward(h, w, t, lse, dh, dw, 1.75)
        again = backward(dt, g, h, w, t, lse, grad, offset=offset)
        assert torch.equal(dh, again[0]) and all(torch.equal(a, b) for a, b in zip(dw, again[1]))
        more = forward(dt, g, h, w, t)
        assert torch.equal(lse, more[1]) and torch.equal(losses, more[0]) and torch.equal(loss, more[2])
        torch.cuda.synchronize()
        assert dt.dt_group_check(g) == dt.DT_OK


def test_sum_equal_pieces_and_optional_outputs(dt):
    h, w, t = make(70, [640] * 3, 128, seed=4)
    with group(3) as g:
        losses, lse, loss = forward(dt, g, h, w, t, op="sum", equal=640)
        check_forward(h, w, t, losses, lse, loss, op="sum")
        dh, dw = backward(dt, g, h, w, t, lse, op="sum")
        check_backward(h, w, t, lse, dh, dw, op="sum")
        only = torch.zeros(70, device="cuda")
        ws = torch.empty(dt.dt_vocab_loss_workspace(g, None, 640, 70, 128, "bf16", False), dtype=torch.uint8, device="cuda")
        dt.dt_vocab_loss(g, h, w, None, 640, t, 70, 128, "bf16", "sum", IGNORE, None, only, None, ws)
        assert torch.equal(only, lse)


def test_every_token_ignored_and_no_tokens(dt):
    h, w, t = make(33, [400, 300], 64, seed=4)
    t[:] = 5
    with group(2) as g:
        losses, lse, loss = forward(dt, g, h, w, t, ignore=5)
        check_forward(h, w, t, losses, lse, loss, ignore=5)
        assert not losses.any() and float(loss) == 0.0
        dh, dw = backward(dt, g, h, w, t, lse, ignore=5)
        assert not dh.any() and not any(x.any() for x in dw)
        none = h[:0]
        _, _, loss = forward(dt, g, none, w, t[:0])
        assert float(loss) == 0.0
        dh, dw = backward(dt, g, none, w, t[:0], lse[:0])
        assert not any(x.any() for x in dw)


def test_ignore_index_may_be_a_vocabulary_index_or_zero(dt):
    h, w, t = make(100, [90, 38], 64, seed=6, drop=0.0)
    t[::3] = 0
    with group(2) as g:
        losses, lse, loss = forward(dt, g, h, w, t, ignore=0)
        check_forward(h, w, t, losses, lse, loss, ignore=0)
        dh, dw = backward(dt, g, h, w, t, lse, ignore=0)
        check_backward(h, w, t, lse, dh, dw, ignore=0)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("bad", [-1, 128, 2 ** 31 - 1, -2 ** 31])
def test_a_target_outside_the_vocabulary_is_recorded_and_ignored(dt, back, bad):
    h, w, t = make(40, [100, 28], 64, seed=8)
    with group(2) as g:
        lse = forward(dt, g, h, w, t)[1]
        kept = t.clone()
        kept[7] = IGNORE
        t[7] = bad
        if back:
            dh, dw = backward(dt, g, h, w, t, lse)
            check_backward(h, w, kept, lse, dh, dw)
        else:
            check_forward(h, w, kept, *forward(dt, g, h, w, t))
        torch.cuda.synchronize()
        code, rank, token, value = dt.dt_group_error_detail(g)
        assert (code, rank, token, value) == (dt.DT_ERR_INVALID, -1, 7, bad)
        with pytest.raises(dt.DtError):
            forward(dt, g, h, w, t)
        dt.dt_group_reset(g)
        t[7] = 0
        forward(dt, g, h, w, t)


@pytest.mark.parametrize("std", [0.0, 4.0])
def test_flat_and_peaked_distributions(dt, std):
    # weights of zero: every logit equal; large weights: logits past 100, one word takes all
    h, w, t = make(130, [500, 600], 256, seed=3, std=std or 1e-30)
    if not std:
        for x in w:
            x.zero_()
    with group(2) as g:
        losses, lse, loss = forward(dt, g, h, w, t)
        check_forward(h, w, t, losses, lse, loss)
        if not std:
            dh, dw = backward(dt, g, h, w, t, lse)
            check_backward(h, w, t, lse, dh, dw)


def test_not_finite_tokens_stay_in_their_rows(dt):
    h, w, t = make(140, [300, 500], 128, seed=3, drop=0.0)
    with group(2) as g:
        clean = forward(dt, g, h, w, t)
        h[5, 3] = float("nan")
        h[131, 0] = float("inf")
        losses, lse, loss = forward(dt, g, h, w, t)
        bad = torch.zeros(140, dtype=torch.bool, device="cuda")
        bad[[5, 131]] = True
        assert torch.isnan(losses[bad]).all() and torch.isnan(loss)
        assert torch.equal(losses[~bad], clean[0][~bad]) and torch.equal(lse[~bad], clean[1][~bad])


@pytest.mark.parametrize("tokens,vocab,dim", [(40, [300, 500], 64), (300, [700, 1000], 200)])
def test_what_ignored_tokens_hold_reaches_no_other_token(dt, tokens, vocab, dim):
    h, w, t = make(tokens, vocab, dim, seed=13)
    drop = torch.nonzero(t == IGNORE)[:, 0]
    assert len(drop) >= 3
    bad = h.clone()
    bad[drop[0]], bad[drop[1], 3], bad[drop[2], 0] = float("nan"), float("inf"), -float("inf")
    with group(2) as g:
        losses, lse, loss = forward(dt, g, h, w, t)
        dh = backward(dt, g, h, w, t, lse)[0]
        losses_b, lse_b, loss_b = forward(dt, g, bad, w, t)
        dh_b = backward(dt, g, bad, w, t, lse_b)[0]
        assert torch.equal(losses, losses_b) and torch.equal(loss, loss_b) and torch.equal(dh, dh_b)
        assert not dh_b[drop].any() and not losses_b[drop].any()
        assert dt.dt_group_check(g) == dt.DT_OK


def test_gradients_against_differences(dt):
    # the loss along random directions of hidden and weight, by central
    # differences of the definition in 64 bits
    h, w, t = make(24, [70, 58], 40, seed=12)
    with group(2) as g:
        _, lse, _ = forward(dt, g, h, w, t)
        dh, dw = backward(dt, g, h, w, t, lse)
    keep = t != IGNORE
    at = (h.double(), torch.cat(w).double())

    def value(h, w):
        l = h @ w.t()
        each = torch.logsumexp(l, 1) - l.gather(1, torch.where(keep, t, 0).long()[:, None])[:, 0]
        return float(each[keep].mean())

    gen = torch.Generator("cuda").manual_seed(1)
    for k, grad in enumerate((dh, torch.cat(dw))):
        d = torch.randn(at[k].shape, generator=gen, device="cuda", dtype=torch.float64)
        lo, hi = ([v + s * 1e-4 * d if i == k else v for i, v in enumerate(at)] for s in (-1, 1))
        diff = (value(*hi) - value(*lo)) / 2e-4
        got = float((grad.double() * d).sum())
        # p - [target] and the result are rounded to bf16: two half ulps of each term, on sums about
        # three times their result
        tol = float((grad.double() * d).abs().sum()) * 3 * 2.0 ** -8
        assert abs(got - diff) <= tol, (k, got, diff, tol)


def test_another_stream_and_graph_replay(dt):
    h, w, t = make(100, [700, 900], 192, seed=2)
    grad = torch.tensor([0.5], device="cuda")
    vocab = [700, 900]
    with group(2) as g:
        losses, lse, loss = forward(dt, g, h, w, t)
        want = backward(dt, g, h, w, t, lse, grad)
        out = [torch.zeros_like(x) for x in (losses, lse, loss)]
        dh, dw = torch.zeros_like(h), [torch.zeros_like(x) for x in w]
        ws = torch.empty(max(dt.dt_vocab_loss_workspace(g, vocab, 0, 100, 192, "bf16", b) for b in (False, True)),
                         dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()

        def both(stream):
            dt.dt_vocab_loss(g, h, w, vocab, 0, t, 100, 192, "bf16", "avg", IGNORE, *out, ws, stream)
            dt.dt_vocab_loss_backward(g, h, w, vocab, 0, t, out[1], grad, 100, 192, "bf16", "avg", IGNORE, dh, dw, ws,
                                      stream)

        side = torch.cuda.Stream()
        both(side)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            both(side)
        for x in (*out, dh, *dw):
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, (losses, lse, loss)))
        assert torch.equal(dh, want[0]) and all(torch.equal(a, b) for a, b in zip(dw, want[1]))


def test_refusals(dt):
    h, w, t = make(16, [64, 64], 32, seed=2)
    vocab = [64, 64]
    losses, lse = (torch.zeros(16, device="cuda") for _ in range(2))
    loss = torch.zeros(1, device="cuda")
    dh, dw = torch.zeros_like(h), [torch.zeros_like(x) for x in w]
    with group(2) as g:
        size = [dt.dt_vocab_loss_workspace(g, vocab, 0, 16, 32, "bf16", b) for b in (False, True)]
        ws = torch.empty(max(size) + 256, dtype=torch.uint8, device="cuda")

        def fwd(status, h=h, w=w, vocab=vocab, t=t, n=16, dim=32, dtype="bf16", op="avg", losses=losses, lse=lse,
                loss=loss, ws=ws):
            with pytest.raises(dt.DtError) as e:
                dt.dt_vocab_loss(g, h, w, vocab, 0, t, n, dim, dtype, op, IGNORE, losses, lse, loss, ws)
            assert e.value.status == status

        def bwd(status, h=h, w=w, lse=lse, grad=None, dh=dh, dw=dw, ws=ws, op="avg", dtype="bf16"):
            with pytest.raises(dt.DtError) as e:
                dt.dt_vocab_loss_backward(g, h, w, vocab, 0, t, lse, grad, 16, 32, dtype, op, IGNORE, dh, dw, ws)
            assert e.value.status == status

        bad, no = dt.DT_ERR_INVALID, dt.DT_ERR_UNSUPPORTED
        for call in (fwd, bwd):
            call(no, dtype="f32")
            call(no, dtype="i32")
            call(bad, dtype=7)
            call(no, op="max")
            call(bad, op=-3)
            call(bad, h=0)
            call(bad, h=h.data_ptr() + 1)
            call(bad, w=[w[0], 0])
            call(bad, w=[w[0], w[1].data_ptr() + 1])
            call(bad, ws=None)
            call(bad, ws=(ws.data_ptr() + 16, ws.numel() - 16))
        fwd(bad, ws=(ws.data_ptr(), size[0] - 1))
        bwd(bad, ws=(ws.data_ptr(), size[1] - 1))
        fwd(bad, dim=0)
        fwd(bad, dim=(1 << 20) + 1)
        fwd(bad, n=(1 << 30) + 1)
        fwd(bad, vocab=[0, 0])
        fwd(bad, vocab=[1 << 30, 1])
        fwd(bad, t=0)
        fwd(bad, losses=lse)                                  # two outputs in one place
        fwd(bad, lse=h.data_ptr())
        fwd(bad, loss=loss.data_ptr() + 2)
        fwd(bad, losses=ws.data_ptr())
        bwd(bad, lse=0)
        bwd(bad, grad=loss.data_ptr() + 1)
        bwd(bad, dh=0)
        bwd(bad, dh=h)
        bwd(bad, dw=[dw[0], 0])
        bwd(bad, dw=[dw[0], dw[0]])
        bwd(bad, dw=[dw[0], w[1]])
        with pytest.raises(ValueError):
            dt.dt_vocab_loss(g, h.t(), w, vocab, 0, t, 16, 32, "bf16", "avg", IGNORE, losses, lse, loss, ws)
        assert dt.dt_vocab_loss_workspace(g, vocab, 0, 16, 32, "f32", False) == 0
        assert dt.dt_vocab_loss_workspace(g, vocab, 0, 16, 0, "bf16", False) == 0
        torch.cuda.synchronize()
        assert not dh.any() and not losses.any() and dt.dt_group_check(g) == dt.DT_OK


# Narrow heads give every CTA or pair many short tiles in a row, so that the
# warps that hand their column group's results on run ahead of those that join
# them: as many tiles as the results have room for, and several times that.
@pytest.mark.parametrize("tokens,vocab,dim", [(2048, [40000, 3], 64), (700, [90001, 40000], 16), (100, [131072], 64)])
def test_many_short_tiles_in_a_row_keep_their_results_apart(dt, tokens, vocab, dim):
    h, w, t = make(tokens, vocab, dim, seed=tokens + 1)
    with group(len(vocab)) as g:
        first = forward(dt, g, h, w, t)
        check_forward(h, w, t, *first)
        for _ in range(20):
            assert all(torch.equal(a, b) for a, b in zip(first, forward(dt, g, h, w, t)))
        assert dt.dt_group_check(g) == dt.DT_OK


# Tokens of a trained model: one word takes nearly all.  Every logit is a single
# product of two bf16 numbers or the exact sum of two, so that logits are exact.
# Relative to the maximum the sum of exponentials is 1 + s; s is off by 2^-18 of
# itself (exponents up to 64 rounded to fp32, the powers, the additions), the
# sum and its logarithm by 2^-22, and lse, where it is rounded, by 2^-24 of
# itself.  As the sum is 1 at least, no loss is negative.
def confident(top, tokens, words, down):
    """Word t has the logit `top` for token t (bf16 products near it), every other one `down` less of itself."""
    gen = torch.Generator("cuda").manual_seed(17)
    dim = tokens + 1
    a = (torch.rand(tokens, generator=gen, device="cuda") + 1).bfloat16()
    h = torch.zeros(tokens, dim, dtype=torch.bfloat16, device="cuda")
    h[torch.arange(tokens), torch.arange(tokens)] = a
    h[:, tokens] = 1
    w = torch.zeros(words, dim, dtype=torch.bfloat16, device="cuda")
    w[torch.arange(tokens), torch.arange(tokens)] = (top / a.float()).bfloat16()
    w[:, tokens] = -down
    t = torch.arange(tokens, device="cuda", dtype=torch.int32)
    return h, [w[:words // 3].contiguous(), w[words // 3:].contiguous()], t


@pytest.mark.parametrize("tokens", [100, 300])
@pytest.mark.parametrize("top,down", [(0.75, 80), (15.0, 0), (15.0, 40), (30.0, 4), (120.0, 0), (3000.0, 0), (3e9, 0), (1e30, 0)])
def test_losses_of_confident_tokens_are_not_negative(dt, tokens, top, down):
    h, w, t = confident(top, tokens, 900, down)
    with group(2) as g:
        losses, lse, loss = forward(dt, g, h, w, t)
    l = h.double() @ torch.cat(w).double().t()
    want = torch.logsumexp(l, 1)
    each = torch.log1p((l - l.gather(1, t.long()[:, None])).exp().sum(1) - 1)
    assert (losses >= 0).all() and float(loss) >= 0
    tol = 2.0 ** -22 + 2.0 ** -18 * (1 - torch.exp(-each)) + 2.0 ** -24 * want.abs()
    assert ((lse.double() - want).abs() <= tol).all()
    # lse and the logit cancel; the difference is rounded once more
    assert ((losses.double() - each).abs() <= tol + 2.0 ** -24 * each).all()


# Confident tokens of a wide head: word t is a multiple of token t's hidden row,
# so that its logit is a sum of `dim` products of one sign.  Both passes make
# the same logits, so what their sums cut off is nearly the same in l and in
# lse: with e the error of a logit, (1 - p) * 2e is left of it in l - lse.
# Beside that lse is rounded once (2^-24 of it), and the distance, its power and
# their product by 2^-21.
def wide_head(tokens, vocab, dim, target):
    gen = torch.Generator("cuda").manual_seed(dim + tokens)
    h = torch.randn(tokens, dim, generator=gen, device="cuda").bfloat16()
    w = torch.randn(vocab, dim, generator=gen, device="cuda") * dim ** -0.5
    w[:tokens] = h.float() * (target / h.float().square().sum(1, keepdim=True))
    w = w.bfloat16()
    t = torch.arange(tokens, device="cuda", dtype=torch.int32)
    return h, [w[:vocab // 2].contiguous(), w[vocab // 2:].contiguous()], t


@pytest.mark.parametrize("tokens,dim", [(1, 4096), (7, 1032), (100, 4096), (128, 2056), (300, 4096), (257, 1100), (300, 4100)])
def test_confident_tokens_of_wide_heads(dt, tokens, dim):
    vocab = 2000
    h, w, t = wide_head(tokens, vocab, dim, 17.5)
    with group(2) as g:
        losses, lse, loss = forward(dt, g, h, w, t)
        dh, dw = backward(dt, g, h, w, t, lse)
    hd, wd = h.double(), torch.cat(w).double()
    l, size = hd @ wd.t(), hd.abs() @ wd.abs().t()
    want, at = torch.logsumexp(l, 1), l.gather(1, t.long()[:, None])[:, 0]
    p = torch.exp(l - want[:, None])
    gone = 1 - p.gather(1, t.long()[:, None])[:, 0]
    assert 1e-5 < float(gone.min()) and float(gone.max()) < 1e-2
    e = (sum_error(1024) * size + 4 * 2.0 ** -24 * size).amax(1)   # sums of 1024, and those added in fp32
    near = 2.0 ** -24 * want.abs() + 2.0 ** -21
    assert ((losses.double() - (want - at)).abs() <= near + 2 * e * gone).all()
    check_forward(h, w, t, losses, lse, loss)
    g = p.clone()
    g[torch.arange(tokens), t.long()] -= 1
    off = 2.0 ** -8 * g.abs() + p * ((1 - p) * 2 * e[:, None] + near[:, None])
    for got, g, off, x in ((dh, g, off, wd), (torch.cat(dw), g.t(), off.t(), hd)):
        want = g @ x / tokens
        tol = (off @ x.abs() + sum_error(len(x)) * (g.abs() @ x.abs())) / tokens + 2.0 ** -8 * want.abs()
        assert ((got.double() - want).abs() <= tol).all(), float(((got.double() - want).abs() / tol).max())


# With a single word its logit is lse itself, p is 1 and there is no gradient,
# however long the sum: both passes have the same logits.
@pytest.mark.parametrize("tokens,vocab,dim", [(1, [1], 64), (5, [0, 1], 4096), (128, [1], 1500), (129, [1, 0], 4096),
                                              (300, [1], 4100), (1000, [1], 2048)])
def test_a_single_word_has_no_gradient(dt, tokens, vocab, dim):
    h, w, t = make(tokens, vocab, dim, seed=dim, std=1.0)
    with group(len(vocab)) as g:
        losses, lse, loss = forward(dt, g, h, w, t)
        check_forward(h, w, t, losses, lse, loss)
        dh, dw = backward(dt, g, h, w, t, lse)
        assert not losses.any() and not loss.any() and not dh.any() and not any(x.any() for x in dw)


# ... and a long sum is those of 1024 products each, added in fp32 in their order.
@pytest.mark.parametrize("tokens,dim", [(1, 4096), (50, 2048), (128, 3000), (300, 4096), (200, 1100)])
def test_logits_are_sums_of_1024_products(dt, tokens, dim):
    h, w, t = make(tokens, [1], dim, seed=dim + 1, std=1.0)
    with group(1) as g:
        lse = forward(dt, g, h, w, t)[1]
        want = torch.zeros_like(lse)
        for k in range(0, dim, 1024):
            part = forward(dt, g, h[:, k:k + 1024].contiguous(), [w[0][:, k:k + 1024].contiguous()], t)[1]
            want = part if k == 0 else want + part
        assert torch.equal(lse, want)


# Logits past 100 with sharp and flat tokens in one batch.  With d = l - lse, of
# the lse that is given: the distance, its product with log2(e) and that
# constant are off by 2^-24 of d each, the power by 2^-22, and powers under
# 2^-126 are zero.
@pytest.mark.parametrize("tokens,vocab", [(130, [500, 600]), (40, [500, 600]), (300, [4000, 3001])])
def test_gradients_of_peaked_distributions(dt, tokens, vocab):
    h, w, t = make(tokens, vocab, 256, seed=3, std=4.0)
    with group(2) as g:
        losses, lse, loss = forward(dt, g, h, w, t)
        dh, dw = backward(dt, g, h, w, t, lse)
    assert float(lse.max()) > 100
    l, dl = logits(h, w)
    keep = (t != IGNORE)[:, None]
    d = l - lse.double()[:, None]
    p = torch.exp(d)
    g = p.clone()
    g[torch.arange(tokens), torch.where(keep[:, 0], t, 0).long()] -= 1
    g *= keep
    off = (2.0 ** -8 * g.abs() + 1.01 * p * (dl + 2.0 ** -22 * (1 + d.abs())) + 2.0 ** -126) * keep
    c = 1 / int(keep.sum())
    for got, g, off, x in ((dh, g, off, torch.cat(w).double()), (torch.cat(dw), g.t(), off.t(), h.double())):
        want = c * (g @ x)
        tol = c * (off @ x.abs() + sum_error(len(x)) * (g.abs() @ x.abs())) + 2.0 ** -8 * want.abs()
        assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("tokens,vocab,dim", [(1, [9000], 4096), (100, [700, 800], 2056), (128, [512], 1032),
                                              (300, [2000], 4096), (33, [100, 30], 1025), (64, [5000], 3000)])
def test_sums_of_several_accumulators(dt, tokens, vocab, dim):
    h, w, t = make(tokens, vocab, dim, seed=dim)
    with group(len(vocab)) as g:
        losses, lse, loss = forward(dt, g, h, w, t)
        check_forward(h, w, t, losses, lse, loss)
        dh, dw = backward(dt, g, h, w, t, lse)
        check_backward(h, w, t, lse, dh, dw)
        assert dt.dt_group_check(g) == dt.DT_OK


# The counted tokens are added over every CTA's part of them.
@pytest.mark.parametrize("tokens,vocab,dim", [(5000, [300, 41], 32), (20001, [77], 16), (600, [70000, 70001], 64), (31, [9000], 16)])
def test_many_tokens_of_a_small_head_are_counted(dt, tokens, vocab, dim):
    h, w, t = make(tokens, vocab, dim, seed=tokens, drop=0.9)
    t[0], t[-1] = 1, 2
    grad = torch.tensor([3.0], device="cuda")
    with group(len(vocab)) as g:
        losses, lse, loss = forward(dt, g, h, w, t)
        check_forward(h, w, t, losses, lse, loss)
        dh, dw = backward(dt, g, h, w, t, lse, grad)
        check_backward(h, w, t, lse, dh, dw, 3.0)
        for bad in (0, tokens // 2, tokens - 1):
            wrong = t.clone()
            wrong[bad] = 1 << 30
            kept = t.clone()
            kept[bad] = IGNORE
            dh, dw = backward(dt, g, h, w, wrong, lse, grad)
            check_backward(h, w, kept, lse, dh, dw, 3.0)
            torch.cuda.synchronize()
            assert dt.dt_group_error_detail(g) == (dt.DT_ERR_INVALID, -1, bad, 1 << 30)
            dt.dt_group_reset(g)


def test_counting_tokens_does_not_outlast_the_products(dt):
    # the gradient makes the loss's products three times and moves p - [target]
    # through memory; a count that ran beside them on one warp took 15 times the loss
    h, w, t = make(65536, [250] * 4, 64, seed=1)
    n, dim, vocab = 65536, 64, [250] * 4
    out = [torch.empty(k, device="cuda") for k in (n, n, 1)]
    dh, dw = torch.empty_like(h), [torch.empty_like(x) for x in w]
    with group(4) as g:
        ws = torch.empty(max(dt.dt_vocab_loss_workspace(g, vocab, 0, n, dim, "bf16", b) for b in (False, True)),
                         dtype=torch.uint8, device="cuda")
        calls = (dt.prepare(dt.dt_vocab_loss, g, h, w, vocab, 0, t, n, dim, "bf16", "avg", IGNORE, *out, ws),
                 dt.prepare(dt.dt_vocab_loss_backward, g, h, w, vocab, 0, t, out[1], None, n, dim, "bf16", "avg", IGNORE,
                            dh, dw, ws))

        def best(call):
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

        loss, back = best(calls[0]), best(calls[1])
        assert back <= 8 * loss, (loss, back)
