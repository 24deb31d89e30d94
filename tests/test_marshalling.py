"""The binding's checks of tensors and lists that the layer norm and loss calls would otherwise
read as something else: a type, a layout or a number of entries that the call does not have.
CPU only: the arguments are marshalled, no call is made."""
from __future__ import annotations

import pytest
import torch

BF16, F32 = torch.bfloat16, torch.float32


class OnGpu(torch.Tensor):
    """A host tensor that says it lies on a GPU."""

    is_cuda = property(lambda self: True)


def made(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


@pytest.fixture(scope="module")
def dt():
    import __graft_entry__
    __graft_entry__.build()
    from same_device_collective_gb300 import dt as mod
    return mod


@pytest.fixture
def calls(dt):
    """Every call's arguments by name, and the function that marshals them (no group, stream 0)."""
    P, n, d, v = 2, 6, 8, [5, 7]
    x, y, dy, dx = ([made(n, d, dtype=BF16) for _ in range(P)] for _ in range(4))
    mean, rstd = ([made(n) for _ in range(P)] for _ in range(2))
    w, b, dw, db = (made(d) for _ in range(4))
    ws = made(64, dtype=torch.uint8)
    h, dh = made(n, d, dtype=BF16), made(n, d, dtype=BF16)
    W, dW = ([made(k, d, dtype=BF16) for k in v] for _ in range(2))
    t = made(n, dtype=torch.int32)
    norm = dict(g=0, x=x, weight=w, bias=b, y=y, mean=mean, rstd=rstd, rows=[n, n], rows_equal=0, cols=d, eps=1e-5,
                dtype="bf16", weight_dtype="f32", stream=0)
    back = dict(g=0, x=x, dy=dy, weight=w, mean=mean, rstd=rstd, dx=dx, dweight=dw, dbias=db, rows=[n, n], rows_equal=0,
                cols=d, dtype="bf16", weight_dtype="f32", op="sum", workspace=ws, stream=0)
    loss = dict(g=0, hidden=h, weight=W, vocab=v, vocab_equal=0, targets=t, tokens=n, dim=d, dtype="bf16", op="avg",
                ignore_index=-100, losses=made(n), lse=made(n), loss=made(1), workspace=ws, stream=0)
    grad = dict(g=0, hidden=h, weight=W, vocab=v, vocab_equal=0, targets=t, lse=made(n), grad_loss=made(1), tokens=n,
                dim=d, dtype="bf16", op="avg", ignore_index=-100, dhidden=dh, dweight=dW, workspace=ws, stream=0)
    return {"norm": (dt._m_layer_norm, norm), "norm_bwd": (dt._m_layer_norm_backward, back),
            "loss": (dt._m_vocab_loss, loss), "loss_bwd": (dt._m_vocab_loss_backward, grad)}


def test_the_calls_as_they_should_be(calls):
    for marshal, kw in calls.values():
        marshal(**kw)
    for name, off in (("norm", dict(weight=None, bias=None, mean=None, rstd=None, rows=None)),
                      ("norm", dict(mean=[None, None])), ("norm_bwd", dict(dweight=None, dbias=None, workspace=None)),
                      ("loss", dict(losses=None, loss=None)), ("loss_bwd", dict(grad_loss=None)),
                      # addresses are taken as they are
                      ("loss", dict(hidden=4096, targets=8192, workspace=(1 << 20, 64)))):
        marshal, kw = calls[name]
        marshal(**{**kw, **off})


@pytest.mark.parametrize("call,arg,dtype", [
    ("loss", "targets", torch.int64), ("loss_bwd", "targets", torch.int64), ("loss", "hidden", F32),
    ("loss", "hidden", torch.float16), ("loss", "losses", BF16), ("loss", "lse", torch.float64), ("loss", "loss", BF16),
    ("loss_bwd", "lse", torch.float64), ("loss_bwd", "grad_loss", BF16), ("loss_bwd", "dhidden", F32),
    ("norm", "weight", BF16), ("norm", "bias", torch.float64), ("norm_bwd", "dweight", BF16), ("norm_bwd", "dbias", BF16),
])
def test_another_type_is_refused(calls, call, arg, dtype):
    marshal, kw = calls[call]
    with pytest.raises(ValueError, match="where the call reads or writes"):
        marshal(**{**kw, arg: kw[arg].to(dtype)})


@pytest.mark.parametrize("call,arg", [("norm", "x"), ("norm", "y"), ("norm", "mean"), ("norm", "rstd"), ("norm_bwd", "dy"),
                                      ("norm_bwd", "dx"), ("loss", "weight"), ("loss_bwd", "dweight")])
def test_another_type_of_one_rank_is_refused(calls, call, arg):
    marshal, kw = calls[call]
    with pytest.raises(ValueError, match="where the call reads or writes"):
        marshal(**{**kw, arg: [kw[arg][0], kw[arg][1].to(torch.float64)]})


@pytest.mark.parametrize("call,arg", [("norm", "y"), ("norm", "mean"), ("norm", "rows"), ("norm_bwd", "dy"),
                                      ("norm_bwd", "rstd"), ("norm_bwd", "rows"), ("loss", "vocab"), ("loss_bwd", "vocab"),
                                      ("loss_bwd", "dweight")])
@pytest.mark.parametrize("entries", [0, 1, 3])
def test_an_entry_for_each_rank(calls, call, arg, entries):
    marshal, kw = calls[call]
    with pytest.raises(ValueError, match="ranks"):
        marshal(**{**kw, arg: (kw[arg] * 2)[:entries]})


def test_strides_and_host_memory_are_refused(calls):
    marshal, kw = calls["loss"]
    with pytest.raises(ValueError, match="not contiguous"):
        marshal(**{**kw, "hidden": made(8, 6, dtype=BF16).t()})
    with pytest.raises(ValueError, match="reaches"):
        marshal(**{**kw, "targets": torch.zeros(6, dtype=torch.int32)})


def test_types_that_the_library_refuses_reach_it(calls):
    for name, dtype in (("norm", "i32"), ("norm_bwd", 9), ("loss", "f32"), ("loss_bwd", "i32")):
        marshal, kw = calls[name]
        marshal(**{**kw, "dtype": dtype})
