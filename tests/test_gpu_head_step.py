"""The layer norm, the gather, the vocabulary loss and their gradients as one step, against
PyTorch's autograd in 64 bits.

Tolerance: between the inputs and a result at most four roundings to bf16 lie in a row (y, p -
[target], dh, the result), each off by at most 2^-8 of a term, so that a result is off by at most
4 * 2^-8 of its size in the 2-norm when the terms do not cancel; twice that is allowed."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_step_matches_autograd():
    from same_device_collective_gb300 import dt
    from same_device_collective_gb300.head_step import IGNORE, HeadStep
    P, rows, dim, vocab = 3, 100, 192, [500, 0, 901]
    gen = torch.Generator("cuda").manual_seed(7)
    step = HeadStep(P, rows, dim, vocab)
    for x in step.x:
        x.copy_(torch.randn(rows, dim, generator=gen, device="cuda") * 2 + 1)
    for w in step.W:
        w.copy_(torch.randn(w.shape, generator=gen, device="cuda") * 0.1)
    step.gamma.copy_(torch.randn(dim, generator=gen, device="cuda") * 0.1 + 1)
    step.beta.copy_(torch.randn(dim, generator=gen, device="cuda") * 0.1)
    step.targets.copy_(torch.randint(0, sum(vocab), (P * rows,), generator=gen, device="cuda"))
    step.targets[::7] = IGNORE
    step()
    torch.cuda.synchronize()
    assert dt.dt_group_check(step.g) == dt.DT_OK

    x = torch.cat(step.x).double().requires_grad_()
    W = torch.cat(step.W).double().requires_grad_()
    gamma, beta = (t.double().requires_grad_() for t in (step.gamma, step.beta))
    h = torch.nn.functional.layer_norm(x, (dim,), gamma, beta, 1e-5)
    loss = torch.nn.functional.cross_entropy(h @ W.t(), step.targets.long(), ignore_index=IGNORE)
    loss.backward()
    loss = loss.detach()
    # y's rounding moves a logit by 2^-9 of it at most on average: far less than this on a mean
    assert abs(float(step.loss) - float(loss)) <= 2.0 ** -8 * float(loss)
    for got, want in ((torch.cat(step.dx), x.grad), (torch.cat(step.dW), W.grad), (step.dgamma, gamma.grad),
                      (step.dbeta, beta.grad)):
        assert float((got.double() - want).norm() / want.norm()) <= 8 * 2.0 ** -8
    step.close()


def test_the_example_trains():
    from same_device_collective_gb300 import head_step
    losses = head_step.main(steps=8)
    assert losses[-1] < losses[0] and all(b <= a for a, b in zip(losses, losses[1:]))
