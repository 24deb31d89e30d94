"""Cases of the operators of a tensor- and sequence-parallel block: what they compute in plain torch, and the library's calls.

The ranks are logical ranks of one GPU. Tokens are split over them (a tensor per rank, each of `dim` columns), and so are
the features of the block's inner layer: a gathering linear layer takes every rank's tokens to each rank's own features,
a reducing one takes the ranks' features back to `dim` columns, summed over the ranks, each rank keeping its own tokens.
A residual norm is what follows: the norm of the block's output, its gate, the residual sum and the next block's norm.
`run` computes an operator from elementary torch operations in 32 bits, or, where `own` is set, calls the library.
"""
import math

import torch

own = False

EPS = 1e-6
SCALE = 0.75   # of the residual stream
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ["none", "relu", "gelu", "silu"]

# No case costs more than these: products of a layer, elements of a norm.
MOST_PRODUCTS = 8192 * 16384 * 4096
MOST_ELEMS = 8 * 4096 * 4096


def _linear(name, op, P, tokens, dim, features, uneven=False, act="none", keep=False, bias=True, residual=False):
    return {"name": name, "op": op, "P": P, "tokens": tokens, "dim": dim, "features": features, "uneven": uneven,
            "act": act, "keep": keep, "bias": bias, "residual": residual}


def _norm(name, op, P, rows, dim, dtype, wdtype, uneven=False):
    return {"name": name, "op": op, "P": P, "tokens": P * rows, "dim": dim, "uneven": uneven, "dtype": dtype, "wdtype": wdtype}


def listed():
    return [
        # one new token on each of four ranks into a small inner layer: a decoding step, where latency counts
        _linear("gather_linear 4x1 of 1024 to 4x1024", "gather", 4, 4, 1024, 4 * 1024, act="silu"),
        # an ordinary training micro-batch, which keeps what its backward pass needs
        _linear("gather_linear 4x512 of 4096 to 4x4096", "gather", 4, 2048, 4096, 4 * 4096, act="gelu", keep=True),
        # a ragged micro-batch, uneven tokens and features, widths that are no multiples of a vector
        _linear("gather_linear_bwd 77 of 500 to 2003", "gather_bwd", 3, 77, 500, 2003, uneven=True, act="gelu"),
        # the largest training batch
        _linear("gather_linear_bwd 4x2048 of 4096 to 4x4096", "gather_bwd", 4, 8192, 4096, 4 * 4096, act="gelu"),
        # the way back of that decoding step in a large layer: the weights' way from memory
        _linear("linear_reduce 4x1 of 4x4096 to 4096", "reduce", 4, 4, 4096, 4 * 4096, residual=True),
        # the largest batch's way back, with the residual stream's sum
        _linear("linear_reduce 8x1024 of 8x2048 to 4096", "reduce", 8, 8192, 4096, 8 * 2048, residual=True),
        # a small model's micro-batch with uneven tokens and features
        _linear("linear_reduce_bwd 300 of 1500 to 1024", "reduce_bwd", 3, 300, 1024, 1500, uneven=True),
        # an ordinary training micro-batch
        _linear("linear_reduce_bwd 4x512 of 4x4096 to 4096", "reduce_bwd", 4, 2048, 4096, 4 * 4096),
        # a decoding step
        _norm("residual_norm 4x1x4096 bf16", "norm", 4, 1, 4096, "bf16", "bf16"),
        # the tokens of four ranks' [8192, 4096]
        _norm("residual_norm 4x2048x4096 bf16", "norm", 4, 2048, 4096, "bf16", "bf16"),
        # a small f32 model with uneven tokens and an odd width
        _norm("residual_norm_bwd 3x600x777 f32 uneven", "norm_bwd", 3, 600, 777, "f32", "f32", True),
        # the training batch's backward pass, f32 weights beside bf16 activations
        _norm("residual_norm_bwd 4x2048x4096 bf16", "norm_bwd", 4, 2048, 4096, "bf16", "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gather", "gather_bwd", "reduce", "reduce_bwd", "norm", "norm_bwd"])
    P = rng.choice([1, 2, 3, 4, 5, 8])
    uneven = rng.random() < 0.5
    dim = _log(rng, 64, 4096)
    if rng.random() < 0.6:
        dim = -(-dim // 8) * 8
    tokens = _log(rng, 1, 8192)
    if op in ("norm", "norm_bwd"):
        rows = max(1, min(tokens, MOST_ELEMS // (P * dim)))
        dtype = rng.choice(["bf16", "f32"])
        c = _norm("", op, P, rows, dim, dtype, rng.choice([dtype, "f32"]), uneven)
    else:
        features = _log(rng, 64, 32768)
        if rng.random() < 0.6:
            features = -(-features // (8 * P)) * 8 * P
        tokens = max(1, min(tokens, MOST_PRODUCTS // (dim * features)))
        c = _linear("", op, P, tokens, dim, features, uneven, bias=rng.random() < 0.7)
        if op in ("gather", "gather_bwd"):
            c["act"] = rng.choice(ACTS)
            c["keep"] = rng.random() < 0.5
        if op == "reduce":
            c["residual"] = rng.random() < 0.7
    del c["name"]
    return c


def _pieces(total, P, uneven):
    """How many of `total` each rank has: even pieces, or pieces that grow with the rank (the first may be empty)."""
    at = [(total * r * r) // (P * P) if uneven else (total * r) // P for r in range(P + 1)]
    return [b - a for a, b in zip(at, at[1:])]


def _rows(case):
    return _pieces(case["tokens"], case["P"], case["uneven"])


def _features(case):
    return _pieces(case["features"], case["P"], case["uneven"])


def _normal(gen, *shape, std=1.0, mean=0.0):
    return torch.randn(*shape, generator=gen, device="cuda") * std + mean


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = {"case": case, "op": case["op"], "rows": _rows(case)}
    op, dim, n = case["op"], case["dim"], case["tokens"]
    if op in ("norm", "norm_bwd"):
        dt_, wdt = DTYPE[case["dtype"]], DTYPE[case["wdtype"]]
        # a residual stream with a scale of its own in each feature, and a block's output of another size
        scale = torch.exp(0.5 * _normal(gen, dim))
        x = [(_normal(gen, k, dim) * scale).to(dt_) for k in s["rows"]]
        s["branch"] = [_normal(gen, k, dim, std=0.2).to(dt_) for k in s["rows"]]
        s["post"], s["pre"] = (_normal(gen, dim, std=0.1, mean=1.0).to(wdt) for _ in range(2))
        s["gate"] = _normal(gen, dim, std=0.3, mean=0.5).to(wdt)
        if op == "norm":
            s["x"] = x
        else:
            s["dy"], s["dz"] = ([_normal(gen, k, dim, std=0.1).to(dt_) for k in s["rows"]] for _ in range(2))
            s["y"], s["rpost"], s["rpre"] = [], [], []
            for a, b in zip(x, s["branch"]):
                y, _, r1, r2 = _plain_norm_rows(a, b, s)
                s["y"].append(y.to(dt_))
                s["rpost"].append(r1)
                s["rpre"].append(r2)
    else:
        s["features"] = _features(case)
        bf16 = torch.bfloat16
        if op in ("gather", "gather_bwd"):
            s["x"] = [_normal(gen, k, dim).to(bf16) for k in s["rows"]]   # a norm's output
            s["w"] = [_normal(gen, f, dim, std=dim ** -0.5).to(bf16) for f in s["features"]]
            s["b"] = [_normal(gen, f, std=0.1).to(bf16) for f in s["features"]] if case["bias"] else None
            if op == "gather_bwd":
                s["pre"] = [_normal(gen, n, f).to(bf16) for f in s["features"]] if case["act"] != "none" else None
                s["dy"] = [_normal(gen, n, f, std=0.1).to(bf16) for f in s["features"]]
        else:
            s["x"] = [_act(_normal(gen, n, f), "gelu").to(bf16) for f in s["features"]]   # an activation's output
            s["w"] = [_normal(gen, dim, f, std=case["features"] ** -0.5).to(bf16) for f in s["features"]]
            s["b"] = _normal(gen, dim, std=0.1).to(bf16) if case["bias"] else None
            s["res"] = [_normal(gen, k, dim, std=2.0).to(bf16) for k in s["rows"]] if case["residual"] else None
            if op == "reduce_bwd":
                s["dy"] = [_normal(gen, k, dim, std=0.1).to(bf16) for k in s["rows"]]
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """The handle, the outputs and the workspace that a program keeps, and its call with these arguments."""
    from same_device_collective_gb300 import dt
    case, op, dim, n = s["case"], s["op"], s["case"]["dim"], s["case"]["tokens"]
    g = _group(dt, case["P"])
    f32 = dict(dtype=torch.float32, device="cuda")
    if op == "norm":
        s["y"], s["z"] = ([torch.empty_like(x) for x in s["x"]] for _ in range(2))
        s["rpost"], s["rpre"] = ([torch.empty(k, **f32) for k in s["rows"]] for _ in range(2))
        s["call"] = dt.prepare(dt.dt_residual_norm, g, s["x"], s["branch"], s["post"], s["gate"], s["pre"], SCALE, s["y"],
                               s["z"], s["rpost"], s["rpre"], s["rows"], 0, dim, EPS, case["dtype"], case["wdtype"])
        s["out"] = [s["y"], s["z"], s["rpost"], s["rpre"]]
    elif op == "norm_bwd":
        s["dx"], s["dbranch"] = ([torch.empty_like(x) for x in s["y"]] for _ in range(2))
        s["dpost"], s["dgate"], s["dpre"] = (torch.empty_like(s["post"]) for _ in range(3))
        s["ws"] = torch.empty(dt.dt_residual_norm_workspace(g, dim), dtype=torch.uint8, device="cuda")
        s["call"] = dt.prepare(dt.dt_residual_norm_backward, g, s["branch"], s["y"], s["dy"], s["dz"], s["post"], s["gate"],
                               s["pre"], SCALE, s["rpost"], s["rpre"], s["dx"], s["dbranch"], s["dpost"], s["dgate"],
                               s["dpre"], s["rows"], 0, dim, case["dtype"], case["wdtype"], "sum", s["ws"])
        s["out"] = [s["dx"], s["dbranch"], s["dpost"], s["dgate"], s["dpre"]]
    else:
        query = dt.dt_gather_linear_workspace if op in ("gather", "gather_bwd") else dt.dt_linear_reduce_workspace
        size = query(g, s["rows"], 0, dim, s["features"], 0, "bf16", op.endswith("bwd"))
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        if op == "gather":
            s["y"] = [torch.empty(n, f, dtype=torch.bfloat16, device="cuda") for f in s["features"]]
            s["out"] = [s["y"]]
            s["pre"] = None
            if case["keep"]:
                s["pre"] = [torch.empty_like(y) for y in s["y"]]
                s["out"].append(s["pre"])
            s["call"] = dt.prepare(dt.dt_gather_linear, g, s["x"], s["w"], s["b"], s["pre"], s["y"], s["rows"], 0, dim,
                                   s["features"], 0, "bf16", case["act"], s["ws"])
        elif op == "gather_bwd":
            s["dx"], s["dw"] = [torch.empty_like(x) for x in s["x"]], [torch.empty_like(w) for w in s["w"]]
            s["db"] = [torch.empty_like(b) for b in s["b"]] if s["b"] else None
            s["call"] = dt.prepare(dt.dt_gather_linear_backward, g, s["x"], s["w"], s["pre"], s["dy"], s["dx"], s["dw"],
                                   s["db"], s["rows"], 0, dim, s["features"], 0, "bf16", case["act"], s["ws"])
            s["out"] = [s["dx"], s["dw"]] + ([s["db"]] if s["b"] else [])
        elif op == "reduce":
            s["y"] = [torch.empty(k, dim, dtype=torch.bfloat16, device="cuda") for k in s["rows"]]
            s["call"] = dt.prepare(dt.dt_linear_reduce, g, s["x"], s["w"], s["b"], s["res"], s["y"], s["rows"], 0, dim,
                                   s["features"], 0, "bf16", s["ws"])
            s["out"] = [s["y"]]
        else:
            s["dx"], s["dw"] = [torch.empty_like(x) for x in s["x"]], [torch.empty_like(w) for w in s["w"]]
            s["db"] = torch.empty_like(s["b"]) if s["b"] is not None else None
            s["call"] = dt.prepare(dt.dt_linear_reduce_backward, g, s["x"], s["w"], s["dy"], s["dx"], s["dw"], s["db"],
                                   s["rows"], 0, dim, s["features"], 0, "bf16", s["ws"])
            s["out"] = [s["dx"], s["dw"]] + ([s["db"]] if s["b"] is not None else [])


_GROUPS = {}


def _group(dt, P):
    if P not in _GROUPS:
        _GROUPS[P] = dt.dt_group_create(P, torch.cuda.current_device())
    return _GROUPS[P]


def run(s):
    if own:
        s["call"]()
        return s["out"]
    return {"gather": _plain_gather, "gather_bwd": _plain_gather_bwd, "reduce": _plain_reduce,
            "reduce_bwd": _plain_reduce_bwd, "norm": _plain_norm, "norm_bwd": _plain_norm_bwd}[s["op"]](s)


# erfc, not 1 + erf: far below zero nothing of the difference would be left
def _act(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "gelu":
        return v * (0.5 * torch.erfc(v * -math.sqrt(0.5)))
    if act == "silu":
        return v / (1 + torch.exp(-v))
    return v


def _slope(v, act):
    if act == "relu":
        return (v > 0).to(v.dtype)
    if act == "gelu":
        return 0.5 * torch.erfc(v * -math.sqrt(0.5)) + v * torch.exp(-0.5 * v * v) * (0.5 / math.pi) ** 0.5
    if act == "silu":
        p = 1 / (1 + torch.exp(-v))
        return p * (1 + v * (1 - p))
    return torch.ones_like(v)


def _plain_gather(s):
    case = s["case"]
    pre = torch.cat(s["x"]).float() @ torch.cat(s["w"]).float().t()
    if s["b"]:
        pre = pre + torch.cat(s["b"]).float()
    split = lambda v: [t.contiguous() for t in v.bfloat16().split(s["features"], 1)]
    out = [split(_act(pre, case["act"]))]
    return out + [split(pre)] if case["keep"] else out


def _plain_gather_bwd(s):
    g = torch.cat(s["dy"], 1).float()
    if s["pre"]:
        g = g * _slope(torch.cat(s["pre"], 1).float(), s["case"]["act"])
    x, w = torch.cat(s["x"]).float(), torch.cat(s["w"]).float()
    out = [list((g @ w).bfloat16().split(s["rows"])), list((g.t() @ x).bfloat16().split(s["features"]))]
    return out + [list(g.sum(0).bfloat16().split(s["features"]))] if s["b"] else out


def _plain_reduce(s):
    y = torch.cat(s["x"], 1).float() @ torch.cat(s["w"], 1).float().t()
    if s["b"] is not None:
        y = y + s["b"].float()
    if s["res"]:
        y = y + torch.cat(s["res"]).float()
    return [list(y.bfloat16().split(s["rows"]))]


def _plain_reduce_bwd(s):
    g = torch.cat(s["dy"]).float()
    dx = g @ torch.cat(s["w"], 1).float()
    dw = g.t() @ torch.cat(s["x"], 1).float()
    out = [[t.contiguous() for t in v.bfloat16().split(s["features"], 1)] for v in (dx, dw)]
    return out + [g.sum(0).bfloat16()] if s["b"] is not None else out


def _plain_norm_rows(x, branch, s):
    o = branch.float()
    r1 = torch.rsqrt(o.square().mean(1) + EPS)
    y = SCALE * x.float() + s["gate"].float() * (o * r1[:, None] * s["post"].float())
    r2 = torch.rsqrt(y.square().mean(1) + EPS)
    return y, y * r2[:, None] * s["pre"].float(), r1, r2


def _plain_norm(s):
    t = s["x"][0].dtype
    y, z, r1, r2 = _plain_norm_rows(torch.cat(s["x"]), torch.cat(s["branch"]), s)
    return [list(y.to(t).split(s["rows"])), list(z.to(t).split(s["rows"])), list(r1.split(s["rows"])),
            list(r2.split(s["rows"]))]


def _plain_norm_bwd(s):
    t, wt = s["y"][0].dtype, s["post"].dtype
    o, y, dy, dz = (torch.cat(s[k]).float() for k in ("branch", "y", "dy", "dz"))
    r1, r2 = torch.cat(s["rpost"])[:, None], torch.cat(s["rpre"])[:, None]
    post, gate, pre = (s[k].float() for k in ("post", "gate", "pre"))
    n, q = y * r2, dz * pre
    d = dy + r2 * (q - n * (q * n).mean(1, keepdim=True))
    h, c = o * r1, d * (gate * post)
    do = r1 * (c - h * (c * h).mean(1, keepdim=True))
    dh = (d * h).sum(0)
    return [list((SCALE * d).to(t).split(s["rows"])), list(do.to(t).split(s["rows"])), (dh * gate).to(wt),
            (dh * post).to(wt), (dz * n).sum(0).to(wt)]


def work(case):
    n, dim, op = case["tokens"], case["dim"], case["op"]
    if op in ("norm", "norm_bwd"):
        es, ws = (2 if case[k] == "bf16" else 4 for k in ("dtype", "wdtype"))
        passes, vectors, flops = (4, 3, 10) if op == "norm" else (6, 6, 22)
        return {"bytes": passes * n * dim * es + 8 * n + vectors * dim * ws, "flops": flops * n * dim}
    f = case["features"]
    if op == "gather":
        return {"bytes": 2 * (n * dim + f * dim + n * f * (1 + case["keep"]) + case["bias"] * f), "flops": 2 * n * dim * f}
    if op == "gather_bwd":
        reads = 2 if case["act"] != "none" else 1
        return {"bytes": 2 * (2 * n * dim + 2 * f * dim + reads * n * f + case["bias"] * f), "flops": 4 * n * dim * f}
    if op == "reduce":
        return {"bytes": 2 * (n * f + f * dim + n * dim * (1 + case["residual"]) + case["bias"] * dim),
                "flops": 2 * n * dim * f}
    return {"bytes": 2 * (n * dim + 2 * n * f + 2 * f * dim + case["bias"] * dim), "flops": 4 * n * dim * f}


def exact(case, seed):
    s = prepare(case, seed)
    op, rows = case["op"], s["rows"]
    if op == "norm":
        out = [[], [], [], []]
        for x, o in zip(s["x"], s["branch"]):
            x, o = x.double(), o.double()
            r1 = 1 / torch.sqrt(torch.einsum("td,td->t", o, o) / case["dim"] + EPS)
            y = SCALE * x + torch.einsum("td,t,d,d->td", o, r1, s["post"].double(), s["gate"].double())
            r2 = 1 / torch.sqrt(torch.einsum("td,td->t", y, y) / case["dim"] + EPS)
            for k, v in enumerate((y, torch.einsum("td,t,d->td", y, r2, s["pre"].double()), r1, r2)):
                out[k].append(v)
        return out
    if op == "norm_bwd":
        post, gate, pre = (s[k].double() for k in ("post", "gate", "pre"))
        dx, do, sums = [], [], [torch.zeros_like(post) for _ in range(3)]
        for r in range(len(rows)):
            o, y, dy, dz = (s[k][r].double() for k in ("branch", "y", "dy", "dz"))
            r1, r2 = s["rpost"][r].double()[:, None], s["rpre"][r].double()[:, None]
            sums[2] += torch.einsum("td,td,t->d", dz, y, r2[:, 0])
            d = dy + dz * pre * r2 - y * r2 ** 3 * ((dz * pre * y).sum(1, keepdim=True) / case["dim"])
            dx.append(SCALE * d)
            c = d * gate * post
            do.append(c * r1 - o * r1 ** 3 * ((c * o).sum(1, keepdim=True) / case["dim"]))
            dh = torch.einsum("td,td,t->d", d, o, r1[:, 0])
            sums[0] += dh * gate
            sums[1] += dh * post
        return [dx, do, *sums]
    if op == "gather":
        y, pre = [], []
        x = torch.cat(s["x"]).double()
        for k, w in enumerate(s["w"]):
            v = torch.einsum("td,fd->tf", x, w.double())
            if s["b"]:
                v += s["b"][k].double()
            pre.append(v)
            y.append(_exact_act(v, case["act"]))
        return [y, pre] if case["keep"] else [y]
    if op == "gather_bwd":
        x = torch.cat(s["x"]).double()
        dx, dw, db = torch.zeros_like(x), [], []
        for k, w in enumerate(s["w"]):
            g = s["dy"][k].double()
            if s["pre"]:
                v = s["pre"][k].double().requires_grad_()
                g, = torch.autograd.grad(_exact_act(v, case["act"]), v, g)
            dx += torch.einsum("tf,fd->td", g, w.double())
            dw.append(torch.einsum("tf,td->fd", g, x))
            db.append(torch.einsum("tf->f", g))
        return [list(dx.split(rows)), dw] + ([db] if s["b"] else [])
    if op == "reduce":
        y = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
        for x, w in zip(s["x"], s["w"]):
            y += torch.einsum("tf,df->td", x.double(), w.double())
        if s["b"] is not None:
            y += s["b"].double()
        y = list(y.split(rows))
        return [[a + b.double() for a, b in zip(y, s["res"])] if s["res"] else y]
    g = torch.cat(s["dy"]).double()
    dx = [torch.einsum("td,df->tf", g, w.double()) for w in s["w"]]
    dw = [torch.einsum("td,tf->df", g, x.double()) for x in s["x"]]
    return [dx, dw] + ([torch.einsum("td->d", g)] if s["b"] is not None else [])


def _exact_act(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "gelu":
        return v * torch.exp(torch.special.log_ndtr(v))
    if act == "silu":
        return v * torch.sigmoid(v)
    return v
