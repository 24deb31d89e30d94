"""The host's side of the linear layers and the residual norm, compiled with its launches taken out: what a
call registers, refuses and hands to the kernels.  CPU only, and nothing here launches on a GPU either."""
from __future__ import annotations

import os
import subprocess

from same_device_collective_gb300 import build as b

HERE = os.path.dirname(os.path.abspath(__file__))
CUDA = os.path.dirname(os.path.dirname(os.path.realpath(b.nvcc())))


def test_residual_norm_of_every_number_of_ranks(tmp_path):
    """Every buffer of up to 16 ranks is registered and checked against the others.  An index outside an
    array ends the program."""
    exe = str(tmp_path / "host_residual")
    res = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-fsanitize=bounds", "-fsanitize-undefined-trap-on-error",
                          "-fstack-protector-all", "-I", b.INCLUDE, "-I", b.CSRC, "-I", os.path.join(CUDA, "include"),
                          os.path.join(HERE, "host_residual.cpp"), "-o", exe], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0 and run.stdout == "ok\n", (run.returncode, run.stdout, run.stderr)


def test_linear_layers_load_through_maps_that_were_made(tmp_path):
    """Each load of each tile of the four large products, for groups with ranks that have no tokens or no
    features: a load through a tensor map that was never made would be an illegal instruction on a GPU.
    What a call lays out in its workspace lies within the query's bytes, apart, and where it is read."""
    exe = str(tmp_path / "host_linear")
    res = subprocess.run([b.nvcc(), *b.ARCH, "-std=c++17", "-O1",
                          "-Xcompiler", "-fsanitize=bounds", "-Xcompiler", "-fsanitize-undefined-trap-on-error",
                          "-I", b.INCLUDE, "-I", b.CSRC,
                          os.path.join(HERE, "host_linear.cu"), "-o", exe], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, (run.returncode, run.stdout, run.stderr)
