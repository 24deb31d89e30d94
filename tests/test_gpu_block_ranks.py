"""The linear layers and the residual norm for groups that other tests do not have: every rank of the most
there can be, and last ranks without features.  Definitions, tolerances and classes are those of the two
operators' own tests."""
from __future__ import annotations

import pytest
import torch

from gpu_util import group
from test_gpu_linear import WHICH, Layer
from test_gpu_residual_norm import Rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dt():
    from same_device_collective_gb300 import dt as mod
    assert torch.cuda.is_available()
    return mod


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [96, 777])
@pytest.mark.parametrize("rows", [[1] * 14, [2] * 15, [1] * 16, [40 + r for r in range(16)], [5, 0] * 7 + [0, 3]], ids=str)
def test_residual_norm_of_many_ranks(dt, rows, cols, dtype):
    a = Rows(dt, rows, cols, dtype, "f32", seed=len(rows))
    with group(len(rows)) as g:
        a.check_forward(a.forward(g))
        a.check_backward(a.backward(g, op="avg"), op="avg")
        a.check_forward(a.forward(g, stats=False))
        assert dt.dt_group_check(g) == dt.DT_OK


# last ranks without features beside an odd number of 128 features: the second half of a pair's last tile has none
@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("rows,dim,features", [([1024, 1024], 512, [1100, 0]), ([2000, 0, 48, 0], 264, [1500, 700, 0, 0]),
                                               ([300, 212, 1], 1030, [129, 0, 0]), ([0, 700, 0, 333], 1000, [0, 40, 0, 0]),
                                               ([2, 1], 64, [72, 0]), ([60, 17], 200, [0, 130])], ids=str)
def test_last_ranks_without_features(dt, which, offset, rows, dim, features):
    a = Layer(dt, which, rows, dim, features, seed=dim + offset, offset=offset)
    act = "gelu" if which == "gather_linear" else "none"
    with group(a.P) as g:
        a.check_forward(a.forward(g, act) if which == "gather_linear" else a.forward(g), act)
        a.check_backward(a.backward(g, act), act)
        assert dt.dt_group_check(g) == dt.DT_OK
