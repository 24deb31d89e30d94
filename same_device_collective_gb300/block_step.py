"""One block of a model that is sequence- and tensor-parallel over P logical ranks of one GPU, forward
and backward, from the library's calls alone.

Rank r holds its own tokens' residual stream (S(0)) and its own piece of the block's inner features; the
norms' weights and the gate are one copy for all ranks (R).  With z_r the block's normed input, one step is

    h_r        = gelu(Z W1_r^T + b1_r), Z all ranks' z            dt_gather_linear
    o_r        = rank r's rows of sum_q h_q W2_q^T + b2           dt_linear_reduce
    y_r        = scale x_r + gate post norm(o_r)
    z'_r       = pre norm(y_r), the next block's input            dt_residual_norm

and back from the gradients of y and z'

    dx_r, do_r, dpost, dgate, dpre                                dt_residual_norm_backward
    dh_r, dW2_r, db2                                              dt_linear_reduce_backward
    dz_r, dW1_r, db1_r                                            dt_gather_linear_backward

after which dx_r and dz_r go to the block below and the rest to the optimizer.  ``python -m
same_device_collective_gb300.block_step`` trains the block on one batch and prints the loss.
"""
from __future__ import annotations

import torch

from . import dt


class BlockStep:
    """Buffers, workspaces and prepared calls of the block for ``rows`` tokens of each rank and ``features``
    inner features of each rank.

    Fill ``x[r]`` and ``z[r]`` ([rows[r], dim] bf16) and call ``forward``; it enqueues the block on the
    stream it was made on, and ``y[r]`` and ``zn[r]`` hold the results in stream order.  Then fill ``dy[r]``
    and ``dzn[r]`` and call ``backward`` for ``dx``, ``dz`` and the weights' gradients."""

    def __init__(self, rows: list, dim: int, features: list, scale: float = 1.0, act: str = "gelu", eps: float = 1e-6,
                 device: int = 0):
        dev = torch.device("cuda", device)
        bf16, f32 = dict(dtype=torch.bfloat16, device=dev), dict(dtype=torch.float32, device=dev)
        P, n = len(rows), sum(rows)
        self.g = g = dt.dt_group_create(P, device)
        tokens = lambda: [torch.zeros(k, dim, **bf16) for k in rows]
        inner = lambda: [torch.zeros(n, f, **bf16) for f in features]
        self.x, self.z, self.o, self.y, self.zn = (tokens() for _ in range(5))
        self.dx, self.dz, self.do, self.dy, self.dzn = (tokens() for _ in range(5))
        self.h, self.pre_h, self.dh = (inner() for _ in range(3))
        self.W1, self.b1 = [torch.zeros(f, dim, **bf16) for f in features], [torch.zeros(f, **bf16) for f in features]
        self.W2, self.b2 = [torch.zeros(dim, f, **bf16) for f in features], torch.zeros(dim, **bf16)
        self.post, self.gate, self.pre = (torch.ones(dim, **f32) for _ in range(3))
        self.dW1, self.db1, self.dW2 = ([torch.empty_like(t) for t in ts] for ts in (self.W1, self.b1, self.W2))
        self.db2 = torch.empty_like(self.b2)
        self.dpost, self.dgate, self.dpre = (torch.empty(dim, **f32) for _ in range(3))
        self.rpost, self.rpre = ([torch.empty(k, **f32) for k in rows] for _ in range(2))
        # the calls run one after the other, so one workspace serves them all
        size = dt.dt_residual_norm_workspace(g, dim)
        for query in (dt.dt_gather_linear_workspace, dt.dt_linear_reduce_workspace):
            size = max(size, *(query(g, rows, 0, dim, features, 0, "bf16", back) for back in (False, True)))
        self.ws = ws = torch.empty(size, dtype=torch.uint8, device=dev)
        self._forward = [
            dt.prepare(dt.dt_gather_linear, g, self.z, self.W1, self.b1, self.pre_h, self.h, rows, 0, dim, features, 0,
                       "bf16", act, ws),
            dt.prepare(dt.dt_linear_reduce, g, self.h, self.W2, self.b2, None, self.o, rows, 0, dim, features, 0, "bf16", ws),
            dt.prepare(dt.dt_residual_norm, g, self.x, self.o, self.post, self.gate, self.pre, scale, self.y, self.zn,
                       self.rpost, self.rpre, rows, 0, dim, eps, "bf16", "f32"),
        ]
        self._backward = [
            dt.prepare(dt.dt_residual_norm_backward, g, self.o, self.y, self.dy, self.dzn, self.post, self.gate, self.pre,
                       scale, self.rpost, self.rpre, self.dx, self.do, self.dpost, self.dgate, self.dpre, rows, 0, dim,
                       "bf16", "f32", "sum", ws),
            dt.prepare(dt.dt_linear_reduce_backward, g, self.h, self.W2, self.do, self.dh, self.dW2, self.db2, rows, 0, dim,
                       features, 0, "bf16", ws),
            dt.prepare(dt.dt_gather_linear_backward, g, self.z, self.W1, self.pre_h, self.dh, self.dz, self.dW1, self.db1,
                       rows, 0, dim, features, 0, "bf16", act, ws),
        ]

    def forward(self) -> None:
        for call in self._forward:
            call()

    def backward(self) -> None:
        for call in self._backward:
            call()

    def weights(self) -> list:
        """(weight, gradient) pairs."""
        pairs = [*zip(self.W1, self.dW1), *zip(self.b1, self.db1), *zip(self.W2, self.dW2)]
        return pairs + [(self.b2, self.db2), (self.post, self.dpost), (self.gate, self.dgate), (self.pre, self.dpre)]

    def close(self) -> None:
        dt.dt_group_destroy(self.g)


def main(P: int = 4, rows: int = 64, dim: int = 256, features: int = 256, steps: int = 20) -> list:
    """A few steps of gradient descent of the normed output towards a target; the losses (mean squares)."""
    gen = torch.Generator("cuda").manual_seed(0)
    step = BlockStep([rows] * P, dim, [features] * P)
    for t in (*step.x, *step.z):
        t.normal_(generator=gen)
    for w, width in ((step.W1, dim), (step.W2, P * features)):
        for t in w:
            t.normal_(0, width ** -0.5, generator=gen)
    target = [torch.randn(rows, dim, generator=gen, device="cuda") for _ in range(P)]
    losses = []
    for _ in range(steps):
        step.forward()
        off = [z.float() - t for z, t in zip(step.zn, target)]
        for d, e in zip(step.dzn, off):
            d.copy_(e)
        step.backward()
        losses.append(float(sum(e.square().sum() for e in off)) / (P * rows * dim))
        for w, d in step.weights():
            w.add_(d, alpha=-2.0 / (P * rows))
    status = dt.dt_group_check(step.g)
    step.close()
    if status != dt.DT_OK:
        raise dt.DtError(status, "block step")
    return losses


if __name__ == "__main__":
    for k, loss in enumerate(main()):
        print(f"step {k}: loss {loss:.4f}")
