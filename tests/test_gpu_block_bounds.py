"""The bounds-checked flavour of the library (DT_BOUNDS=1 when building) over the linear layers and the
residual norm: with DT_BOUNDS_TRIM=16 every output is recorded 16 bytes short, so the kernels' last stores,
which lie inside the real buffers, are reported and skipped.  Skipped in the default build."""
from __future__ import annotations

import json
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

TESTS = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(TESTS)


@pytest.fixture(scope="module")
def dt():
    from same_device_collective_gb300 import dt as mod
    assert torch.cuda.is_available()
    if not mod.dt_build_flags() & mod.DT_BUILD_BOUNDS:
        pytest.skip("the default build has no bounds checks")
    return mod


OPERATORS = r"""
import json, sys
import torch
sys.path[:0] = [ROOT, TESTS]
from same_device_collective_gb300 import dt

res = {}
gen = torch.Generator("cuda").manual_seed(3)
bf16, f32 = torch.bfloat16, torch.float32
def made(*shape, dtype=bf16): return torch.randn(*shape, generator=gen, device="cuda").to(dtype)
MARK = 2.0 ** 100   # what no result is (results of bf16 do come out as a round number)
def marked(*shape, dtype=bf16): return torch.full(shape, MARK, dtype=dtype, device="cuda")
def tail(t, n):
    # the last n elements kept their value, all others were written
    t = t.reshape(-1)
    return bool((t[len(t) - n:] == MARK).all()) and bool((t[:len(t) - n] != MARK).all())

P = 2
g = dt.dt_group_create(P, 0)
def record(name, tails):
    torch.cuda.synchronize()
    code, kernel, buf, off = dt.dt_group_error_detail(g)
    res[name] = dict(code=code, kernel=kernel, buf=buf, off=off, tails=tails())
    dt.dt_group_reset(g)

# few tokens, small products, the tensor cores' tiles, and those with the inner axis split
for name, rows, dim, features in (("few", [3, 2], 64, [40, 24]), ("small", [20, 30], 64, [48, 96]),
                                  ("tiles", [400, 700], 1024, [1000, 1048]), ("splits", [40, 30], 8192, [2048, 1000])):
    n = sum(rows)
    x, h = [made(k, dim) for k in rows], [made(n, f) for f in features]
    w1, w2, b1, b2 = [made(f, dim) for f in features], [made(dim, f) for f in features], [made(f) for f in features], made(dim)
    args = (rows, 0, dim, features, 0, "bf16")
    ws = torch.empty(max(q(g, *args, b) for q in (dt.dt_gather_linear_workspace, dt.dt_linear_reduce_workspace) for b in (False, True)), dtype=torch.uint8, device="cuda")
    y, pre = ([marked(n, f) for f in features] for _ in range(2))
    dt.dt_gather_linear(g, x, w1, b1, pre, y, *args, "silu", ws)
    record(name + " gather", lambda: all(tail(t, 8) for t in (*y, *pre)))
    dx, dw, db = [marked(k, dim) for k in rows], [marked(f, dim) for f in features], [marked(f) for f in features]
    dt.dt_gather_linear_backward(g, x, w1, h, h, dx, dw, db, *args, "gelu", ws)
    record(name + " gather_bwd", lambda: all(tail(t, 8) for t in (*dx, *dw, *db)))
    z = [marked(k, dim) for k in rows]
    dt.dt_linear_reduce(g, h, w2, b2, x, z, *args, ws)
    record(name + " reduce", lambda: all(tail(t, 8) for t in z))
    dx, dw, db = [marked(n, f) for f in features], [marked(dim, f) for f in features], marked(dim)
    dt.dt_linear_reduce_backward(g, h, w2, x, dx, dw, db, *args, ws)
    record(name + " reduce_bwd", lambda: all(tail(t, 8) for t in (*dx, *dw, db)))

for name, rows, cols in (("few", [3, 2], 256), ("rings", [400, 200], 256), ("long", [2, 3], 9000)):
    x, o, dy, dz = ([made(k, cols) for k in rows] for _ in range(4))
    w = [made(cols, dtype=f32) for _ in range(3)]
    y, z, r1, r2 = [marked(k, cols) for k in rows], [marked(k, cols) for k in rows], [made(k, dtype=f32) for k in rows], [made(k, dtype=f32) for k in rows]
    dt.dt_residual_norm(g, x, o, *w, 1.0, y, z, None, None, rows, 0, cols, 1e-6, "bf16", "f32")
    record(name + " norm", lambda: all(tail(t, 8) for t in (*y, *z)))
    dx, do, dw = [marked(k, cols) for k in rows], [marked(k, cols) for k in rows], [marked(cols, dtype=f32) for _ in range(3)]
    ws = torch.empty(dt.dt_residual_norm_workspace(g, cols), dtype=torch.uint8, device="cuda")
    dt.dt_residual_norm_backward(g, o, x, dy, dz, *w, 1.0, r1, r2, dx, do, *dw, rows, 0, cols, "bf16", "f32", "sum", ws)
    record(name + " norm_bwd", lambda: all(tail(t, 8) for t in (*dx, *do)) and all(tail(t, 4) for t in dw))
dt.dt_group_destroy(g)
print("RESULT " + json.dumps(res))
"""


def test_trimmed_extents_of_every_output(dt):
    env = dict(os.environ, DT_BOUNDS_TRIM="16")
    code = OPERATORS.replace("ROOT", repr(ROOT)).replace("TESTS", repr(TESTS))
    out = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-3000:]
    res = json.loads([ln for ln in out.stdout.splitlines() if ln.startswith("RESULT ")][-1][len("RESULT "):])
    buffers = {"gather": [0, 1, 16, 17], "gather_bwd": [32, 33, 48, 49, 64, 65], "reduce": [0, 1],
               "reduce_bwd": [32, 33, 48, 49, 64], "norm": [64, 65, 80, 81], "norm_bwd": [64, 65, 80, 81, 131, 132, 133]}
    for name, r in res.items():
        which = name.split()[1]
        kernel = "residual" if which.startswith("norm") else "linear"
        assert r["code"] == dt.DT_ERR_INVALID and dt.BOUNDS_KERNELS[r["kernel"]] == kernel, (name, r)
        assert r["buf"] in buffers[which] and r["tails"], (name, r)
    assert len(res) == 4 * 4 + 3 * 2
