"""Cases of the layer norm and vocabulary loss operators: what they compute in plain torch, and the library's calls.

The ranks are logical ranks of one GPU. A layer norm case has the tokens of every rank (a tensor per rank) and one
copy of the weights; a loss case has every rank's piece of the vocabulary (a tensor per rank), and the tokens once.
`run` computes an operator from elementary torch operations in 32 bits, or, where `own` is set, calls the library.
"""
import math

import torch

own = False

EPS = 1e-5
IGNORE = -100
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}

# No case costs more than these: elements of a norm, products of a head.
MOST_ELEMS = 65536 * 4096
MOST_PRODUCTS = {"loss": 8192 * 131072 * 4096, "loss_bwd": 8192 * 65536 * 4096}


def _norm(name, op, P, rows, dim, dtype, wdtype, uneven=False):
    return {"name": name, "op": op, "P": P, "rows": rows, "uneven": uneven, "dim": dim, "dtype": dtype, "wdtype": wdtype}


def _loss(name, op, P, tokens, vocab, dim, uneven=False):
    return {"name": name, "op": op, "P": P, "tokens": tokens, "vocab": vocab, "uneven": uneven, "dim": dim}


def listed():
    return [
        # one new token on each of four ranks: a decoding step, where only the latency counts
        _norm("norm 4x1x4096 bf16", "norm", 4, 1, 4096, "bf16", "bf16"),
        # the shards that a ReduceScatter of four ranks' [8192, 4096] leaves
        _norm("norm 4x2048x4096 bf16", "norm", 4, 2048, 4096, "bf16", "bf16"),
        # uneven f32 shards of an odd width, rows that begin at any 4-byte address
        _norm("norm 3x5000x1021 f32 uneven", "norm", 3, 5000, 1021, "f32", "f32", True),
        # the same step's backward pass
        _norm("norm_bwd 4x2048x4096 bf16", "norm_bwd", 4, 2048, 4096, "bf16", "bf16"),
        # 65536 tokens of eight ranks with f32 weights beside bf16 activations: the largest batch
        _norm("norm_bwd 8x8192x4096 bf16", "norm_bwd", 8, 8192, 4096, "bf16", "f32"),
        # a small f32 model with uneven shards of an odd width
        _norm("norm_bwd 3x600x777 f32 uneven", "norm_bwd", 3, 600, 777, "f32", "f32", True),
        # the score of a single token under a small head: latency
        _loss("loss 1 of 8192x1024", "loss", 4, 1, 8192, 1024),
        # an ordinary evaluation batch
        _loss("loss 2048 of 32768x4096", "loss", 4, 2048, 32768, 4096),
        # a long batch under a large vocabulary in eight pieces: 4 GiB of logits, were they kept
        _loss("loss 8192 of 131072x4096", "loss", 8, 8192, 131072, 4096),
        # a ragged micro-batch, uneven pieces, a width that is no multiple of a vector
        _loss("loss_bwd 77 of 10007x500", "loss_bwd", 3, 77, 10007, 500, True),
        # an ordinary training micro-batch
        _loss("loss_bwd 2048 of 32768x4096", "loss_bwd", 4, 2048, 32768, 4096),
        # the largest training batch
        _loss("loss_bwd 8192 of 65536x4096", "loss_bwd", 8, 8192, 65536, 4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "loss", "loss_bwd"])
    P = rng.choice([1, 2, 3, 4, 5, 8])
    uneven = rng.random() < 0.5
    dim = _log(rng, 64, 4096)
    if rng.random() < 0.6:
        dim = -(-dim // 8) * 8
    if op in ("norm", "norm_bwd"):
        rows = max(1, min(_log(rng, 1, 8192), MOST_ELEMS // (P * dim)))
        dtype = rng.choice(["bf16", "f32"])
        c = _norm("", op, P, rows, dim, dtype, rng.choice([dtype, "f32"]), uneven)
    else:
        tokens, vocab = _log(rng, 1, 8192), _log(rng, 1000, 131072)
        tokens = max(1, min(tokens, MOST_PRODUCTS[op] // (vocab * dim)))
        c = _loss("", op, P, tokens, vocab, dim, uneven)
    del c["name"]
    return c


def _pieces(total, P, uneven):
    """How many of `total` rows each rank has: even pieces, or pieces that grow with the rank (the first may be empty)."""
    at = [(total * r * r) // (P * P) if uneven else (total * r) // P for r in range(P + 1)]
    return [b - a for a, b in zip(at, at[1:])]


def _rows(case):
    return _pieces(case["P"] * case["rows"], case["P"], case["uneven"])


def _vocab(case):
    return _pieces(case["vocab"], case["P"], case["uneven"])


def _normal(gen, *shape, std=1.0, mean=0.0):
    return torch.randn(*shape, generator=gen, device="cuda") * std + mean


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = {"case": case, "P": case["P"], "op": case["op"]}
    dim = case["dim"]
    if case["op"] in ("norm", "norm_bwd"):
        dt_, wdt = DTYPE[case["dtype"]], DTYPE[case["wdtype"]]
        # activations with an offset and a scale of their own in each feature, as residual streams have
        scale = torch.exp(0.5 * _normal(gen, dim))
        shift = _normal(gen, dim, std=0.3)
        s["rows"] = _rows(case)
        s["x"] = [(_normal(gen, n, dim) * scale + shift).to(dt_) for n in s["rows"]]
        s["w"] = _normal(gen, dim, std=0.1, mean=1.0).to(wdt)
        s["b"] = _normal(gen, dim, std=0.1).to(wdt)
        if case["op"] == "norm_bwd":
            s["dy"] = [_normal(gen, n, dim, std=0.1).to(dt_) for n in s["rows"]]
            s["mean"], s["rstd"] = [], []
            for x in s["x"]:
                m = x.float().mean(1)
                s["mean"].append(m)
                s["rstd"].append(torch.rsqrt((x.float() - m[:, None]).square().mean(1) + EPS))
    else:
        n = case["tokens"]
        s["vocab"] = _vocab(case)
        s["h"] = _normal(gen, n, dim).bfloat16()
        s["w"] = [_normal(gen, v, dim, std=0.02).bfloat16() for v in s["vocab"]]
        s["targets"] = torch.randint(0, case["vocab"], (n,), generator=gen, device="cuda", dtype=torch.int32)
        # prompts and padding are not trained on: one token in eight
        drop = torch.rand(n, generator=gen, device="cuda") < 0.125
        drop[0] = False
        s["targets"][drop] = IGNORE
        if case["op"] == "loss_bwd":
            s["grad"] = torch.rand(1, generator=gen, device="cuda") + 0.5   # the gradient of the loss: a loss scale
            s["lse"] = torch.cat([torch.logsumexp(h.float() @ torch.cat(s["w"]).float().t(), 1)
                                  for h in s["h"].split(2048)])
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """The handle, the outputs and the workspace that a program keeps, and its call with these arguments."""
    from same_device_collective_gb300 import dt
    case, P, dim = s["case"], s["P"], s["case"]["dim"]
    g = _group(dt, P)
    f32 = dict(dtype=torch.float32, device="cuda")
    if s["op"] == "norm":
        s["y"] = [torch.empty_like(x) for x in s["x"]]
        s["mean"], s["rstd"] = ([torch.empty(n, **f32) for n in s["rows"]] for _ in range(2))
        s["call"] = dt.prepare(dt.dt_layer_norm, g, s["x"], s["w"], s["b"], s["y"], s["mean"], s["rstd"],
                               s["rows"], 0, dim, EPS, case["dtype"], case["wdtype"])
        s["out"] = [s["y"], s["mean"], s["rstd"]]
    elif s["op"] == "norm_bwd":
        s["dx"] = [torch.empty_like(x) for x in s["x"]]
        s["dw"], s["db"] = torch.empty_like(s["w"]), torch.empty_like(s["b"])
        s["ws"] = torch.empty(dt.dt_layer_norm_workspace(g, dim), dtype=torch.uint8, device="cuda")
        s["call"] = dt.prepare(dt.dt_layer_norm_backward, g, s["x"], s["dy"], s["w"], s["mean"], s["rstd"], s["dx"],
                               s["dw"], s["db"], s["rows"], 0, dim, case["dtype"], case["wdtype"], "sum", s["ws"])
        s["out"] = [s["dx"], s["dw"], s["db"]]
    else:
        n, back = case["tokens"], s["op"] == "loss_bwd"
        s["ws"] = torch.empty(dt.dt_vocab_loss_workspace(g, s["vocab"], 0, n, dim, "bf16", back), dtype=torch.uint8,
                              device="cuda")
        if back:
            s["dh"], s["dw"] = torch.empty_like(s["h"]), [torch.empty_like(w) for w in s["w"]]
            s["call"] = dt.prepare(dt.dt_vocab_loss_backward, g, s["h"], s["w"], s["vocab"], 0, s["targets"], s["lse"],
                                   s["grad"], n, dim, "bf16", "avg", IGNORE, s["dh"], s["dw"], s["ws"])
            s["out"] = [s["dh"], s["dw"]]
        else:
            s["losses"], s["lse"] = torch.empty(n, **f32), torch.empty(n, **f32)
            s["loss"] = torch.empty(1, **f32)
            s["call"] = dt.prepare(dt.dt_vocab_loss, g, s["h"], s["w"], s["vocab"], 0, s["targets"], n, dim, "bf16",
                                   "avg", IGNORE, s["losses"], s["lse"], s["loss"], s["ws"])
            s["out"] = [s["losses"], s["lse"], s["loss"]]


_GROUPS = {}


def _group(dt, P):
    if P not in _GROUPS:
        _GROUPS[P] = dt.dt_group_create(P, torch.cuda.current_device())
    return _GROUPS[P]


def run(s):
    if own:
        s["call"]()
        return s["out"]
    return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "loss": _plain_loss, "loss_bwd": _plain_loss_bwd}[s["op"]](s)


def _plain_norm(s):
    x = torch.cat(s["x"]).float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = torch.rsqrt(c.square().mean(1) + EPS)
    y = c * rstd[:, None] * s["w"].float() + s["b"].float()
    return [list(y.to(s["x"][0].dtype).split(s["rows"])), list(mean.split(s["rows"])), list(rstd.split(s["rows"]))]


def _plain_norm_bwd(s):
    x, dy = torch.cat(s["x"]).float(), torch.cat(s["dy"]).float()
    rstd = torch.cat(s["rstd"])[:, None]
    h = (x - torch.cat(s["mean"])[:, None]) * rstd
    q = dy * s["w"].float()
    dx = rstd * (q - q.mean(1, keepdim=True) - h * (q * h).mean(1, keepdim=True))
    dw, db = (dy * h).sum(0), dy.sum(0)
    return [list(dx.to(s["x"][0].dtype).split(s["rows"])), dw.to(s["w"].dtype), db.to(s["b"].dtype)]


def _plain_loss(s):
    logits = s["h"].float() @ torch.cat(s["w"]).float().t()
    top = logits.amax(1)
    lse = top + (logits - top[:, None]).exp().sum(1).log()
    keep = s["targets"] != IGNORE
    at = logits.gather(1, s["targets"].clamp(min=0).long()[:, None])[:, 0]
    losses = torch.where(keep, lse - at, 0.0)
    return [losses, lse, (losses.sum() / keep.sum()).reshape(1)]


def _plain_loss_bwd(s):
    h, w = s["h"].float(), torch.cat(s["w"]).float()
    p = (h @ w.t() - s["lse"][:, None]).exp()
    keep = s["targets"] != IGNORE
    p.scatter_add_(1, s["targets"].clamp(min=0).long()[:, None], torch.full_like(s["lse"], -1.0)[:, None])
    p *= (keep * (s["grad"] / keep.sum()))[:, None]
    return [(p @ w).bfloat16(), list((p.t() @ h).bfloat16().split(s["vocab"]))]


def work(case):
    dim = case["dim"]
    if case["op"] in ("norm", "norm_bwd"):
        es, ws = (2 if case[k] == "bf16" else 4 for k in ("dtype", "wdtype"))
        rows = sum(_rows(case))
        passes, flops = (2, 8) if case["op"] == "norm" else (3, 14)
        vectors = 2 if case["op"] == "norm" else 3   # weights and bias in; weights in, both gradients out
        return {"bytes": passes * rows * dim * es + 8 * rows + vectors * dim * ws, "flops": flops * rows * dim}
    n, v = case["tokens"], case["vocab"]
    if case["op"] == "loss":
        return {"bytes": 2 * (n + v) * dim + 4 * n + 8 * n, "flops": 2 * n * v * dim}
    return {"bytes": 2 * 2 * (n + v) * dim + 8 * n, "flops": 6 * n * v * dim}


def exact(case, seed):
    if case["op"] in ("loss", "loss_bwd") and work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_bwd"):
        w, b = s["w"].double(), s["b"].double()
        y, mean, rstd, dx = [], [], [], []
        dw, db = torch.zeros_like(w), torch.zeros_like(b)
        for r, x in enumerate(s["x"]):
            x = x.double()
            if case["op"] == "norm":
                v, m = torch.var_mean(x, 1, correction=0)
                i = 1 / torch.sqrt(v + EPS)
                y.append(torch.addcmul(b, (x - m[:, None]) * i[:, None], w))
                mean.append(m)
                rstd.append(i)
                continue
            m, i, dy = s["mean"][r].double()[:, None], s["rstd"][r].double()[:, None], s["dy"][r].double()
            h = (x - m) * i
            dw += torch.einsum("td,td->d", dy, h)
            db += dy.sum(0)
            q = dy * w
            dot = torch.einsum("td,td->t", q, h)[:, None] / case["dim"]
            dx.append((q - q.sum(1, keepdim=True) / case["dim"] - h * dot) * i)
        return [y, mean, rstd] if case["op"] == "norm" else [dx, dw, db]
    w = torch.cat(s["w"]).double()
    keep = s["targets"] != IGNORE
    if case["op"] == "loss":
        losses, lses = [], []
        for h, t, k in zip(s["h"].split(1024), s["targets"].split(1024), keep.split(1024)):
            l = h.double() @ w.t()
            lses.append(torch.logsumexp(l, 1))
            losses.append(torch.where(k, lses[-1] - l[torch.arange(len(t), device=l.device), t.clamp(min=0).long()], 0.0))
        losses = torch.cat(losses)
        return [losses, torch.cat(lses), (losses.sum() / keep.sum()).reshape(1)]
    dh, dw = [], torch.zeros_like(w)
    scale = s["grad"].double() / keep.sum()
    for h, t, k, lse in zip(s["h"].split(1024), s["targets"].split(1024), keep.split(1024), s["lse"].split(1024)):
        h = h.double()
        g = torch.exp(h @ w.t() - lse.double()[:, None])
        g[torch.arange(len(t), device=g.device), t.clamp(min=0).long()] -= 1
        g *= (k * scale)[:, None]
        dh.append(g @ w)
        dw += g.t() @ h
    return [torch.cat(dh), list(dw.split(s["vocab"]))]
