"""The bounds-checked flavour of the library (DT_BOUNDS=1 when building).

In that flavour every global load and store of the data kernels is checked
against its buffer's extent as the call's arguments give it; an access
outside is skipped and DT_ERR_INVALID is recorded in the group's error word.
tests/conftest.py turns every recorded access into a test failure, so
`pytest -m gpu` on that build runs the whole GPU suite under the checks.
Here the checker itself is shown to fire: with DT_BOUNDS_TRIM=16 every
destination is recorded 16 bytes short, so the kernels' last stores (inside
the real buffers) are reported and skipped.  Skipped in the default build.
"""
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

CHILD = r"""
import json, sys
import numpy as np, torch
sys.path[:0] = [ROOT, TESTS]
from same_device_collective_gb300 import dt
import oracle
from gpu_util import host, rand_inputs

res = {}
P, n = 4, 4096
xs = rand_inputs(P, n, "bf16", 11)
outs = [torch.full((n,), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(P)]
g = dt.dt_group_create(P, 0)
dt.dt_allreduce(g, dt.DT_ALL_RANKS, xs, outs, n, "bf16", "sum")
torch.cuda.synchronize()
code, kernel, buf, off = dt.dt_group_error_detail(g)
want = oracle.allreduce("bf16", "sum", [host(x) for x in xs])
got = [host(o) for o in outs]
res["allreduce"] = dict(
    code=code, kernel=kernel, buf=buf, off=off,
    body=all(np.array_equal(got[r][:n - 8], want[r][:n - 8]) for r in range(P)),
    tail=all(bool((got[r][n - 8:] == 0x40E0).all()) for r in range(P)))
dt.dt_group_destroy(g)

shard = 8192
ins = [torch.randint(0, 255, (shard,), dtype=torch.uint8, device="cuda") for _ in range(P)]
outs = [torch.full((P * shard,), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(P)]
g = dt.dt_group_create(P, 0)
dt.dt_all_gather(g, dt.DT_ALL_RANKS, ins, outs, None, 1, shard)
torch.cuda.synchronize()
code, kernel, buf, off = dt.dt_group_error_detail(g)
want = np.concatenate([x.cpu().numpy() for x in ins])
got = [o.cpu().numpy() for o in outs]
last = slice((P - 1) * shard, P * shard)
res["all_gather"] = dict(
    code=code, kernel=kernel, buf=buf, off=off,
    body=all(np.array_equal(o[:(P - 1) * shard], want[:(P - 1) * shard]) for o in got),
    last=all(bool(((o[last] == want[last]) | (o[last] == 0xA5)).all()) for o in got),
    tail=all(bool((o[-16:] == 0xA5).all()) for o in got))
dt.dt_group_destroy(g)
print("RESULT " + json.dumps(res))
"""


@pytest.fixture(scope="module")
def dt():
    from same_device_collective_gb300 import dt as mod
    assert torch.cuda.is_available()
    if not mod.dt_build_flags() & mod.DT_BUILD_BOUNDS:
        pytest.skip("needs the bounds-checked build (DT_BOUNDS=1 when building)")
    return mod


def test_checker_reports_and_skips_stores_past_a_trimmed_extent(dt):
    env = dict(os.environ, DT_BOUNDS_TRIM="16")
    code = CHILD.replace("ROOT", repr(ROOT)).replace("TESTS", repr(TESTS))
    out = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True,
                         timeout=300)
    assert out.returncode == 0, out.stderr[-3000:]
    line = [ln for ln in out.stdout.splitlines() if ln.startswith("RESULT ")][-1]
    res = json.loads(line[len("RESULT "):])

    ar = res["allreduce"]
    assert ar["code"] == dt.DT_ERR_INVALID
    assert dt.BOUNDS_KERNELS[ar["kernel"]] == "reduce"
    assert 16 <= ar["buf"] < 16 + 4                  # an output buffer
    assert ar["off"] == 4096 * 2 - 16                # its last 16-byte vector
    assert ar["body"] and ar["tail"]                 # the rest stored, the last vector skipped

    ag = res["all_gather"]
    assert ag["code"] == dt.DT_ERR_INVALID
    assert dt.BOUNDS_KERNELS[ag["kernel"]] in ("copy_bulk", "copy_vec")
    assert 256 <= ag["buf"] < 256 + 4                # a destination buffer
    assert ag["body"] and ag["last"] and ag["tail"]


OPERATORS = r"""
import json, sys
import torch
sys.path[:0] = [ROOT, TESTS]
from same_device_collective_gb300 import dt

res = {}
gen = torch.Generator("cuda").manual_seed(3)
bf16, f32 = torch.bfloat16, torch.float32
def made(*shape, dtype=bf16): return torch.randn(*shape, generator=gen, device="cuda").to(dtype)
def sevens(*shape, dtype=bf16): return torch.full(shape, 7.0, dtype=dtype, device="cuda")
def tail(t, n):
    # the last n elements kept their value, all others were written
    t = t.reshape(-1)
    return bool((t[len(t) - n:] == 7).all()) and bool((t[:len(t) - n] != 7).all())

P, rows, cols = 2, [20, 12], 64
g = dt.dt_group_create(P, 0)
def record(name, tails):
    torch.cuda.synchronize()
    code, kernel, buf, off = dt.dt_group_error_detail(g)
    res[name] = dict(code=code, kernel=kernel, buf=buf, off=off, tails=tails())
    dt.dt_group_reset(g)

x, dy, y, dx = [made(n, cols) for n in rows], [made(n, cols) for n in rows], [sevens(n, cols) for n in rows], [sevens(n, cols) for n in rows]
w = made(cols, dtype=f32)
dt.dt_layer_norm(g, x, w, w, y, None, None, rows, 0, cols, 1e-5, "bf16", "f32")
record("norm", lambda: all(tail(t, 8) for t in y))
mean, rstd = ([sevens(n, dtype=f32) for n in rows] for _ in range(2))
scratch = [torch.empty(n * cols + 8, dtype=bf16, device="cuda") for n in rows]
dt.dt_layer_norm(g, x, w, w, [t[:n * cols] for t, n in zip(scratch, rows)], mean, rstd, rows, 0, cols, 1e-5, "bf16", "f32")
record("stats", lambda: all(tail(t, 4) for t in (*mean, *rstd)))
mean, rstd = ([made(n, dtype=f32) for n in rows] for _ in range(2))
dw, db = sevens(cols, dtype=f32), sevens(cols, dtype=f32)
ws = torch.empty(dt.dt_layer_norm_workspace(g, cols), dtype=torch.uint8, device="cuda")
dt.dt_layer_norm_backward(g, x, dy, w, mean, rstd, dx, dw, db, rows, 0, cols, "bf16", "f32", "sum", ws)
record("norm_bwd", lambda: all(tail(t, 8) for t in dx) and tail(dw, 4) and tail(db, 4))

n, dim, vocab = 40, 64, [100, 60]
h, W = made(n, dim), [made(v, dim) for v in vocab]
t = torch.randint(0, 160, (n,), generator=gen, device="cuda", dtype=torch.int32)
losses, lse, loss = sevens(n, dtype=f32), sevens(n, dtype=f32), sevens(1, dtype=f32)
ws = torch.empty(max(dt.dt_vocab_loss_workspace(g, vocab, 0, n, dim, "bf16", b) for b in (False, True)), dtype=torch.uint8, device="cuda")
dt.dt_vocab_loss(g, h, W, vocab, 0, t, n, dim, "bf16", "avg", -100, losses, lse, loss, ws)
record("loss", lambda: tail(losses, 4) and tail(lse, 4) and tail(loss, 1))
lse = torch.logsumexp(h.float() @ torch.cat(W).float().t(), 1)
dh, dW = sevens(n, dim), [sevens(v, dim) for v in vocab]
dt.dt_vocab_loss_backward(g, h, W, vocab, 0, t, lse, None, n, dim, "bf16", "sum", -100, dh, dW, ws)
record("loss_bwd", lambda: tail(dh, 8) and all(tail(t, 8) for t in dW))
dt.dt_group_destroy(g)
print("RESULT " + json.dumps(res))
"""


def test_trimmed_extents_of_every_output_of_the_norm_and_the_loss(dt):
    env = dict(os.environ, DT_BOUNDS_TRIM="16")
    code = OPERATORS.replace("ROOT", repr(ROOT)).replace("TESTS", repr(TESTS))
    out = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-3000:]
    res = json.loads([ln for ln in out.stdout.splitlines() if ln.startswith("RESULT ")][-1][len("RESULT "):])
    buffers = {"norm": ("norm", range(32, 34)), "stats": ("norm", [32, 33, 48, 49, 64, 65]),
               "norm_bwd": ("norm", [32, 33, 82, 83]), "loss": ("vocab", [3, 4, 5]), "loss_bwd": ("vocab", [1, 16, 17])}
    for name, (kernel, which) in buffers.items():
        r = res[name]
        assert r["code"] == dt.DT_ERR_INVALID and dt.BOUNDS_KERNELS[r["kernel"]] == kernel, (name, r)
        assert r["buf"] in which and r["tails"], (name, r)
    assert res["norm"]["off"] == (20 if res["norm"]["buf"] == 32 else 12) * 64 * 2 - 16
