"""What the binding of the linear layers and the residual norm refuses on the host, and the calls without a
group.  Nothing here needs a GPU: no call reaches a kernel."""
from __future__ import annotations

import pytest
import torch

BF16, F32 = torch.bfloat16, torch.float32


class OnGpu(torch.Tensor):
    """A host tensor that says it is on a GPU: the marshallers look at types, strides and places only."""
    is_cuda = True


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
    n, d, f, rows = 6, 8, [5, 7], [2, 4]
    b = lambda *s: made(*s, dtype=BF16)
    tokens, inner = (lambda: [b(k, d) for k in rows]), (lambda: [b(n, k) for k in f])
    w1, w2 = (lambda: [b(k, d) for k in f]), (lambda: [b(d, k) for k in f])
    stats = lambda: [made(k) for k in rows]
    ws = made(64, dtype=torch.uint8)
    sizes = dict(g=0, rows=rows, rows_equal=0, dim=d, features=f, features_equal=0, dtype="bf16", workspace=ws, stream=0)
    norm = dict(g=0, post_weight=made(d), gate=made(d), pre_weight=made(d), residual_scale=1.0, rstd_post=stats(),
                rstd_pre=stats(), rows=rows, rows_equal=0, cols=d, dtype="bf16", weight_dtype="f32", stream=0)
    return {
        "gather": (dt._m_gather_linear, dict(sizes, x=tokens(), weight=w1(), bias=[b(k) for k in f], pre=inner(), y=inner(), act="gelu")),
        "gather_bwd": (dt._m_gather_linear_backward, dict(sizes, x=tokens(), weight=w1(), pre=inner(), dy=inner(), dx=tokens(),
                                                          dweight=w1(), dbias=[b(k) for k in f], act="silu")),
        "reduce": (dt._m_linear_reduce, dict(sizes, x=inner(), weight=w2(), bias=b(d), residual=tokens(), y=tokens())),
        "reduce_bwd": (dt._m_linear_reduce_backward, dict(sizes, x=inner(), weight=w2(), dy=tokens(), dx=inner(), dweight=w2(),
                                                          dbias=b(d))),
        "norm": (dt._m_residual_norm, dict(norm, x=tokens(), branch=tokens(), y=tokens(), z=tokens(), eps=1e-6)),
        "norm_bwd": (dt._m_residual_norm_backward, dict(norm, branch=tokens(), y=tokens(), dy=tokens(), dz=tokens(), dx=tokens(),
                                                        dbranch=tokens(), dpost_weight=made(d), dgate=made(d),
                                                        dpre_weight=made(d), op="sum", workspace=ws)),
    }


def test_the_calls_as_they_should_be(calls):
    for marshal, kw in calls.values():
        marshal(**kw)
    for name, off in (("gather", dict(bias=None, pre=None, act="none")), ("gather_bwd", dict(pre=None, dbias=None, act=0)),
                      ("reduce", dict(bias=None, residual=None, rows=None)), ("reduce_bwd", dict(dbias=None, features=None)),
                      ("norm", dict(post_weight=None, gate=None, pre_weight=None, rstd_post=None, rstd_pre=None)),
                      ("norm_bwd", dict(dy=None, dgate=None, dpost_weight=None, dpre_weight=None, workspace=None))):
        marshal, kw = calls[name]
        marshal(**{**kw, **off})


LISTS = [("gather", "x"), ("gather", "weight"), ("gather", "bias"), ("gather", "pre"), ("gather", "y"), ("gather_bwd", "x"),
         ("gather_bwd", "weight"), ("gather_bwd", "pre"), ("gather_bwd", "dy"), ("gather_bwd", "dx"), ("gather_bwd", "dweight"),
         ("gather_bwd", "dbias"), ("reduce", "x"), ("reduce", "weight"), ("reduce", "residual"), ("reduce", "y"),
         ("reduce_bwd", "x"), ("reduce_bwd", "weight"), ("reduce_bwd", "dy"), ("reduce_bwd", "dx"), ("reduce_bwd", "dweight"),
         ("norm", "x"), ("norm", "branch"), ("norm", "y"), ("norm", "z"), ("norm", "rstd_post"), ("norm", "rstd_pre"),
         ("norm_bwd", "branch"), ("norm_bwd", "y"), ("norm_bwd", "dy"), ("norm_bwd", "dz"), ("norm_bwd", "dx"),
         ("norm_bwd", "dbranch"), ("norm_bwd", "rstd_post"), ("norm_bwd", "rstd_pre")]
ONES = [("reduce", "bias"), ("reduce_bwd", "dbias"), ("norm", "post_weight"), ("norm", "gate"), ("norm", "pre_weight"),
        ("norm_bwd", "dpost_weight"), ("norm_bwd", "dgate"), ("norm_bwd", "dpre_weight")]


@pytest.mark.parametrize("call,arg", LISTS)
def test_another_type_or_length_of_a_list_is_refused(calls, call, arg):
    marshal, kw = calls[call]
    with pytest.raises(ValueError, match="where the call reads or writes"):
        marshal(**{**kw, arg: [kw[arg][0], kw[arg][1].to(torch.float64)]})
    for entries in (0, 1, 3):
        with pytest.raises(ValueError, match="ranks"):
            marshal(**{**kw, arg: (kw[arg] * 2)[:entries], **({} if arg != "x" else {"rows": kw["rows"]})})


@pytest.mark.parametrize("call,arg", ONES)
def test_another_type_is_refused(calls, call, arg):
    marshal, kw = calls[call]
    with pytest.raises(ValueError, match="where the call reads or writes"):
        marshal(**{**kw, arg: kw[arg].to(torch.float64)})


@pytest.mark.parametrize("call", ["gather", "gather_bwd", "reduce", "reduce_bwd"])
def test_an_entry_of_sizes_for_each_rank(calls, call):
    marshal, kw = calls[call]
    for arg in ("rows", "features"):
        with pytest.raises(ValueError, match="ranks"):
            marshal(**{**kw, arg: [1, 2, 3]})


def test_strides_and_host_memory_are_refused(calls):
    for call, arg in (("gather", "weight"), ("reduce", "x"), ("norm", "branch")):
        marshal, kw = calls[call]
        with pytest.raises(ValueError, match="not contiguous"):
            marshal(**{**kw, arg: [kw[arg][0], made(*reversed(kw[arg][1].shape), dtype=BF16).t()]})
        with pytest.raises(ValueError, match="reaches"):
            marshal(**{**kw, arg: [kw[arg][0], torch.zeros(kw[arg][1].shape, dtype=BF16)]})


def test_an_unknown_activation_is_refused(calls):
    marshal, kw = calls["gather"]
    with pytest.raises(KeyError):
        marshal(**{**kw, "act": "tanh"})


def test_operator_calls_without_a_group_are_invalid(dt):
    lib, none = dt.library(), [None]
    assert lib.dt_gather_linear(*none * 7, 0, 0, None, 0, 1, 0, None, 0, None) == dt.DT_ERR_INVALID
    assert lib.dt_gather_linear_backward(*none * 9, 0, 0, None, 0, 1, 0, None, 0, None) == dt.DT_ERR_INVALID
    assert lib.dt_linear_reduce(*none * 7, 0, 0, None, 0, 1, None, 0, None) == dt.DT_ERR_INVALID
    assert lib.dt_linear_reduce_backward(*none * 8, 0, 0, None, 0, 1, None, 0, None) == dt.DT_ERR_INVALID
    assert lib.dt_residual_norm(*none * 6, 1.0, *none * 5, 0, 8, 1e-6, 0, 0, None) == dt.DT_ERR_INVALID
    assert lib.dt_residual_norm_backward(*none * 8, 1.0, *none * 8, 0, 8, 0, 0, 0, None, 0, None) == dt.DT_ERR_INVALID
    assert lib.dt_gather_linear_workspace(None, None, 8, 8, None, 8, 1, 0) == 0
    assert lib.dt_linear_reduce_workspace(None, None, 8, 8, None, 8, 1, 1) == 0
    assert lib.dt_residual_norm_workspace(None, 8) == 0
