"""The linear layers, the residual norm and their gradients as one block, against PyTorch's autograd in 64
bits.

Tolerance: between the inputs and a result at most seven roundings to bf16 lie in a row (pre_h, h, o, y,
dbranch, dh, the gradient before the activation, the result itself), each off by at most 2^-8 of a term, so
that a result is off by at most 8 * 2^-8 of its size in the 2-norm when the terms do not cancel; twice that
is allowed."""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def filled(rows, dim, features, scale, act, seed):
    from same_device_collective_gb300.block_step import BlockStep
    gen = torch.Generator("cuda").manual_seed(seed)
    step = BlockStep(rows, dim, features, scale, act)
    normal = lambda t, std=1.0, mean=0.0: t.copy_(torch.randn(t.shape, generator=gen, device="cuda") * std + mean)
    for t in (*step.x, *step.z, *step.dy, *step.dzn):
        normal(t)
    for t in step.W1:
        normal(t, dim ** -0.5)
    for t in step.W2:
        normal(t, sum(features) ** -0.5)
    for t in (*step.b1, step.b2):
        normal(t, 0.2)
    for t in (step.post, step.gate, step.pre):
        normal(t, 0.2, 1.0)
    return step


def check(step, rows, dim, features, scale, act, eps=1e-6):
    d = lambda t: t.double().requires_grad_()
    x, z, W1, b1 = (d(torch.cat(t)) for t in (step.x, step.z, step.W1, step.b1))
    W2, b2, post, gate, pre = d(torch.cat(step.W2, 1)), *(d(t) for t in (step.b2, step.post, step.gate, step.pre))
    v = z @ W1.t() + b1
    h = {"gelu": lambda: v * 0.5 * torch.erfc(-v / math.sqrt(2)), "silu": lambda: v * torch.sigmoid(v), "relu": lambda: v.clamp(min=0),
         "none": lambda: v}[act]()
    norm = lambda t: t / torch.sqrt(t.square().mean(1, keepdim=True) + eps)
    y = scale * x + gate * post * norm(h @ W2.t() + b2)
    zn = norm(y) * pre
    loss = (y * torch.cat(step.dy).double()).sum() + (zn * torch.cat(step.dzn).double()).sum()
    loss.backward()
    got = {"y": (torch.cat(step.y), y.detach()), "zn": (torch.cat(step.zn), zn.detach()), "dx": (torch.cat(step.dx), x.grad),
           "dz": (torch.cat(step.dz), z.grad), "dW1": (torch.cat(step.dW1), W1.grad), "db1": (torch.cat(step.db1), b1.grad),
           "dW2": (torch.cat(step.dW2, 1), W2.grad), "db2": (step.db2, b2.grad), "dpost": (step.dpost, post.grad),
           "dgate": (step.dgate, gate.grad), "dpre": (step.dpre, pre.grad)}
    for name, (a, b) in got.items():
        assert float((a.double() - b).norm()) <= 16 * 2.0 ** -8 * float(b.norm()), name


@pytest.mark.parametrize("rows,dim,features,scale,act", [([3, 0, 2], 64, [40, 24, 100], 1.0, "gelu"), ([90, 33], 192, [300, 21], 0.7, "silu"),
                                                         ([256, 300, 100], 520, [512, 1000, 200], 1.0, "gelu"),
                                                         ([700], 1000, [3000], 0.5, "relu")])
def test_the_block_matches_autograd(rows, dim, features, scale, act):
    from same_device_collective_gb300 import dt
    P = max(len(rows), len(features))
    rows, features = rows + [0] * (P - len(rows)), features + [0] * (P - len(features))
    step = filled(rows, dim, features, scale, act, seed=dim)
    step.forward()
    step.backward()
    torch.cuda.synchronize()
    assert dt.dt_group_check(step.g) == dt.DT_OK
    check(step, rows, dim, features, scale, act)
    step.close()


def test_one_block_after_another_in_a_graph():
    """The block's calls captured together, replayed on other inputs, while an eager autograd graph of the
    same tensors is alive."""
    rows, dim, features = [40, 50], 128, [96, 160]
    step, other = (filled(rows, dim, features, 1.0, "gelu", seed=s) for s in (1, 2))
    alive = (step.post.requires_grad_() * 2).sum()
    step.forward(), step.backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):   # the prepared calls, on the capture's stream
        stream = torch.cuda.current_stream().cuda_stream
        for call in (*step._forward, *step._backward):
            assert call._fn(*call._args[:-1], stream) == 0
    for name in ("x", "z", "dy", "dzn", "W1", "b1", "W2"):
        for t, v in zip(getattr(step, name), getattr(other, name)):
            t.copy_(v)
    with torch.no_grad():
        for name in ("b2", "post", "gate", "pre"):
            getattr(step, name).copy_(getattr(other, name))
    graph.replay()
    torch.cuda.synchronize()
    step.post.requires_grad_(False)
    check(step, rows, dim, features, 1.0, "gelu")
    other.forward(), other.backward()
    torch.cuda.synchronize()
    for a, b in zip((*step.zn, *step.dz, *step.dW1, step.db2), (*other.zn, *other.dz, *other.dW1, other.db2)):
        assert torch.equal(a, b)
    del alive
    step.close(), other.close()


def test_the_example_runs():
    from same_device_collective_gb300 import block_step
    losses = block_step.main(steps=4)
    assert len(losses) == 4 and all(math.isfinite(x) for x in losses)
