"""The end of a training step of a model that is sequence- and vocabulary-parallel over P logical
ranks of one GPU, from the library's calls alone.

Rank r holds its own tokens' activations (S(0)) and its own piece of the vocabulary (S(0)); the
layer norm's weights are one copy for all ranks (R).  One step is

    y_r            = layer_norm(x_r)                       dt_layer_norm
    h              = y_0 .. y_{P-1}             S(0) -> R   dt_all_gather, one shared result
    loss           = cross entropy of h under the ranks' vocabulary rows      dt_vocab_loss
    dh, dW_r       = its gradient, dh reduced over the ranks                  dt_vocab_loss_backward
    dy_r           = rank r's rows of dh         R -> S(0)  dt_replicate_to_shard
    dx_r, dgamma, dbeta = the norm's gradient, dgamma and dbeta reduced       dt_layer_norm_backward

after which dW_r, dgamma and dbeta go to the optimizer (or, data-parallel, to
``dt_bucket_allreduce``) and dx_r to the layers below.  ``python -m
same_device_collective_gb300.head_step`` trains the weights on one batch and prints the loss.
"""
from __future__ import annotations

import torch

from . import dt

IGNORE = -100


class HeadStep:
    """Buffers, workspaces and prepared calls of the step for ``rows`` tokens on each of P ranks.

    Fill ``x[r]`` ([rows, dim] bf16) and ``targets`` ([P * rows] int32, or IGNORE), then call the
    object: it enqueues the step on the stream it was made on.  ``loss``, ``dx``, ``dgamma``,
    ``dbeta`` and ``dW`` hold the results in stream order."""

    def __init__(self, P: int, rows: int, dim: int, vocab: list, eps: float = 1e-5, device: int = 0):
        dev = torch.device("cuda", device)
        bf16 = dict(dtype=torch.bfloat16, device=dev)
        f32 = dict(dtype=torch.float32, device=dev)
        n = P * rows
        self.g = g = dt.dt_group_create(P, device)
        self.x, self.y, self.dy, self.dx = ([torch.zeros(rows, dim, **bf16) for _ in range(P)] for _ in range(4))
        self.mean, self.rstd = ([torch.empty(rows, **f32) for _ in range(P)] for _ in range(2))
        self.gamma, self.beta = torch.ones(dim, **f32), torch.zeros(dim, **f32)
        self.dgamma, self.dbeta = torch.empty(dim, **f32), torch.empty(dim, **f32)
        self.W = [torch.zeros(v, dim, **bf16) for v in vocab]
        self.dW = [torch.empty_like(w) for w in self.W]
        self.h, self.dh = torch.empty(n, dim, **bf16), torch.empty(n, dim, **bf16)
        self.targets = torch.full((n,), IGNORE, dtype=torch.int32, device=dev)
        self.losses, self.lse, self.loss = torch.empty(n, **f32), torch.empty(n, **f32), torch.empty(1, **f32)
        # the calls run one after the other, so one workspace serves them all
        size = max(dt.dt_layer_norm_workspace(g, dim),
                   *(dt.dt_vocab_loss_workspace(g, vocab, 0, n, dim, "bf16", back) for back in (False, True)))
        self.ws = torch.empty(size, dtype=torch.uint8, device=dev)
        ALL = dt.DT_ALL_RANKS
        self.calls = [
            dt.prepare(dt.dt_layer_norm, g, self.x, self.gamma, self.beta, self.y, self.mean, self.rstd, None, rows,
                       dim, eps, "bf16", "f32"),
            dt.prepare(dt.dt_all_gather, g, ALL, self.y, [self.h] * P, None, rows, dim * 2, dt.DT_SHARED_OUTPUT),
            dt.prepare(dt.dt_vocab_loss, g, self.h, self.W, vocab, 0, self.targets, n, dim, "bf16", "avg", IGNORE,
                       self.losses, self.lse, self.loss, self.ws),
            dt.prepare(dt.dt_vocab_loss_backward, g, self.h, self.W, vocab, 0, self.targets, self.lse, None, n, dim,
                       "bf16", "avg", IGNORE, self.dh, self.dW, self.ws),
            dt.prepare(dt.dt_replicate_to_shard, g, ALL, [self.dh] * P, self.dy, None, n, dim * 2),
            dt.prepare(dt.dt_layer_norm_backward, g, self.x, self.dy, self.gamma, self.mean, self.rstd, self.dx,
                       self.dgamma, self.dbeta, None, rows, dim, "bf16", "f32", "sum", self.ws),
        ]

    def __call__(self) -> None:
        for call in self.calls:
            call()

    def close(self) -> None:
        dt.dt_group_destroy(self.g)


def main(P: int = 4, rows: int = 64, dim: int = 256, vocab: int = 1000, steps: int = 20) -> list:
    """A few steps of gradient descent on one batch; the losses."""
    gen = torch.Generator("cuda").manual_seed(0)
    step = HeadStep(P, rows, dim, [vocab] * P)
    for x in step.x:
        x.normal_(generator=gen)
    for w in step.W:
        w.normal_(0, dim ** -0.5, generator=gen)
    step.targets.random_(0, P * vocab, generator=gen)
    losses = []
    for _ in range(steps):
        step()
        for w, d in zip([*step.W, step.gamma, step.beta], [*step.dW, step.dgamma, step.dbeta]):
            w.add_(d, alpha=-1.0)
        losses.append(float(step.loss))
    status = dt.dt_group_check(step.g)
    step.close()
    if status != dt.DT_OK:
        raise dt.DtError(status, "head step")
    return losses


if __name__ == "__main__":
    for k, loss in enumerate(main()):
        print(f"step {k}: loss {loss:.4f}")
