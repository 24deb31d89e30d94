"""The block's six calls one by one: each one's results against its definition in 64 bits of what it read, with
the operators' own tolerances, so that a wrong buffer, scale or weight between two calls shows."""
from __future__ import annotations

import pytest
import torch

from test_gpu_block_step import filled
from test_gpu_linear import Layer
from test_gpu_residual_norm import Rows

pytestmark = pytest.mark.gpu


def layer(which, rows, dim, features, **fields):
    a = Layer.__new__(Layer)
    a.which, a.rows, a.dim, a.features, a.P, a.n, a.offset = which, rows, dim, features, len(rows), sum(rows), 0
    a.__dict__.update(fields)
    return a


@pytest.mark.parametrize("rows,dim,features,scale,act", [([3, 0, 2], 64, [40, 24, 100], 1.0, "gelu"), ([90, 33], 192, [300, 21], 0.7, "silu"),
                                                         ([256, 300, 100], 520, [512, 1000, 0], 1.0, "gelu"),
                                                         ([700], 1000, [3000], 0.5, "relu"), ([1, 1, 1, 1], 512, [256] * 4, 1.0, "silu")])
def test_each_call_of_the_block(rows, dim, features, scale, act):
    from same_device_collective_gb300 import dt
    step = filled(rows, dim, features, scale, act, seed=dim + 1)
    step.forward()
    step.backward()
    torch.cuda.synchronize()
    assert dt.dt_group_check(step.g) == dt.DT_OK
    gather = layer("gather_linear", rows, dim, features, x=step.z, w=step.W1, b=step.b1, pre=step.pre_h, dy=step.dh)
    gather.check_forward((step.h, step.pre_h), act)
    gather.check_backward((step.dz, step.dW1, step.db1), act)
    reduce = layer("linear_reduce", rows, dim, features, x=step.h, w=step.W2, b=step.b2, res=None, dy=step.do)
    reduce.check_forward(step.o)
    reduce.check_backward((step.dh, step.dW2, step.db2))
    norm = Rows.__new__(Rows)
    norm.rows, norm.cols, norm.scale, norm.offset, norm.dtype, norm.wdtype = rows, dim, scale, 0, "bf16", "f32"
    norm.x, norm.branch, norm.dy, norm.dz, norm.y = step.x, step.o, step.dy, step.dzn, step.y
    norm.post, norm.gate, norm.pre, norm.r1, norm.r2 = step.post, step.gate, step.pre, step.rpost, step.rpre
    norm.check_forward((step.y, step.zn, step.rpost, step.rpre))
    norm.check_backward((step.dx, step.do, (step.dpost, step.dgate, step.dpre)))
    step.close()
