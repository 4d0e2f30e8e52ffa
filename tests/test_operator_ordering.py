"""The order of the training and adapter operators' accesses, within a kernel
and between calls: repeated calls on freshly copied inputs, early starts
against plain stream order, other streams than the current one."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

from parity_util import lib
from test_adapters import Case

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def s():
    return lib()


@pytest.mark.gpu
@pytest.mark.parametrize("R,n", [(16, 40), (32, 23), (64, 9)])
def test_passes_over_a_row_tile_do_not_meet(s, R, n):
    """128-row tiles of dozens of adapters, 2048 columns shared by clusters of
    eight CTAs: every pass but the last is followed by copies into the memory
    that held its sums, which the other CTAs have read.  Many calls on freshly
    copied inputs give one result, within its bounds."""
    c = Case(s, "whole", 2048, 2048, 2048, R, n)
    host = {k: v.cpu().pin_memory() for k, v in (("down", c.down), ("up", c.up), ("A", c.A))}
    C0, low0 = c.forward()
    c.check_forward(C0, low0)
    g0 = c.backward(low0)
    c.check_backward(low0, *g0)
    for _ in range(60):
        c.dev["down"], c.dev["up"] = host["down"].cuda(), host["up"].cuda()
        c.A_r = [host["A"].cuda()]
        C, low = c.forward()
        assert torch.equal(low, low0) and torch.equal(C[0], C0[0])
        g = c.backward(low)
        assert torch.equal(g[0][0], g0[0][0]) and torch.equal(g[1], g0[1]) and torch.equal(g[2], g0[2])


def test_a_stopped_ring_is_waited_for(tmp_path):
    """The row rings of the training LayerNorm, stopped after a given-up wait:
    every copy in flight is a stage's last entry, which the end waits for, with
    any number of stages and one or two copying threads (host arithmetic)."""
    if not shutil.which("g++"):
        pytest.skip("g++ not available")
    exe = str(tmp_path / "ring_order")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-I",
                        os.path.join(ROOT, "partial_sum_reduction_gb300", "csrc"),
                        os.path.join(ROOT, "tests", "c", "ring_order.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout


SIZES = """
import partial_sum_reduction_gb300 as s
for dt in ("bf16", "f32"):
    for I, J, K, n, R in ((1, 8, 8, 1, 1), (97, 40, 36, 2, 3), (6540, 160, 544, 17, 32), (8192, 4096, 16384, 8, 64)):
        print(s.Plan("{X:1}", "I,J", "J,K", "I,K", I, J, K, dt, dt).adapters_workspace_size(n, R))
    print(s.shmm_layernorm_backward_workspace_size(8192, 4096))
"""


@pytest.mark.gpu
def test_workspace_sizes_ask_no_device(s):
    """What a process without a device allocates for is what the calls of one
    with a device ask for."""
    got = [subprocess.run([sys.executable, "-c", touch + SIZES], cwd=ROOT, env=env, capture_output=True, text=True)
           for touch, env in (("", dict(os.environ, CUDA_VISIBLE_DEVICES="")),
                              ("import torch; torch.zeros(1, device='cuda')\n", dict(os.environ)))]
    assert all(r.returncode == 0 for r in got), got
    assert got[0].stdout == got[1].stdout and len(got[0].stdout.split()) == 10
