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


# ---- early starts, streams, the order of requests ------------------------------

def adapter_buffers(c):
    s, H = c.s, c.H
    nan = float("nan")
    return {"C": c.cut(s.TENSOR_C, c.base), "low": torch.full((c.I, c.R), nan, device="cuda"),
            "dA": H.alloc(c.plan, s.TENSOR_A, fill=nan), "dd": torch.full((c.n, c.R, c.J), nan, device="cuda"),
            "du": torch.full((c.n, c.R, c.K), nan, device="cuda"), "ws": H.adapters_workspace(c.plan, c.n, c.R),
            "dC": c.cut(s.TENSOR_C, c.dC), "dbase": c.cut(s.TENSOR_A, c.dbase)}


def adapter_step(c, b, A, stream=None):
    d = (c.dev["ids"], c.dev["down"], c.dev["up"], c.dev["scale"])
    c.plan.adapters_forward(A, *d, b["C"], b["C"], b["low"], stream=stream)
    c.plan.adapters_backward(b["dC"], A, *d, b["low"], b["dbase"], b["dA"], b["dd"], b["du"], b["ws"], stream=stream)


def results(b, keys):
    return [t.clone() for k in keys for t in (b[k] if isinstance(b[k], list) else [b[k]])]


ADAPTER_KEYS = ("C", "low", "dA", "dd", "du")
SIZES_OF_EACH_KIND = [("rows", 24, 512, 512, 16, 8, "bf16"),       # single tokens
                      ("columns", 640, 512, 2048, 32, 5, "bf16"),   # longer row tiles
                      ("whole", 2304, 1024, 1536, 16, 12, "bf16"),  # tensor-memory projection, several passes
                      ("contracted", 130, 256, 264, 12, 3, "f32")]


@pytest.mark.gpu
@pytest.mark.parametrize("layout,I,J,K,R,n,dt", SIZES_OF_EACH_KIND)
def test_early_starts_give_the_bits_of_plain_order(s, monkeypatch, layout, I, J, K, R, n, dt):
    """A chain of steps without a synchronisation, each with kernels that start
    before the one in front of them ends: the plan's own product into the base,
    the adapters over it, and their gradient, on other inputs every time, into
    the same buffers.  SHMM_PDL=0 with a synchronisation after every call gives
    the same bits."""
    c = Case(s, layout, I, J, K, R, n, dt, dt)
    As = [c.A_r] + [c.H.shard(c.plan, s.TENSOR_A, torch.randn(I, J, generator=torch.Generator().manual_seed(q)).to(c.ti))
                    for q in (1, 2)]
    B_r = c.H.shard(c.plan, s.TENSOR_B, torch.randn(J, K, generator=torch.Generator().manual_seed(9)).to(c.ti) / J ** 0.5)
    got = {}
    for pdl in ("1", "0"):
        monkeypatch.setenv("SHMM_PDL", pdl)
        b, ws = adapter_buffers(c), c.H.workspace(c.plan)
        wait = torch.cuda.synchronize if pdl == "0" else (lambda: None)
        kept = []
        torch.cuda.synchronize()
        d = (c.dev["ids"], c.dev["down"], c.dev["up"], c.dev["scale"])
        for i in range(9):
            A = As[i % 3]
            c.plan.run(A, B_r, b["C"], ws)
            wait()
            c.plan.adapters_forward(A, *d, b["C"], b["C"], b["low"])
            wait()
            c.plan.adapters_backward(b["dC"], A, *d, b["low"], b["dbase"], b["dA"], b["dd"], b["du"], b["ws"])
            wait()
            if i % 3 == 2:
                kept.append(results(b, ADAPTER_KEYS))
        s.shmm_sync_status()
        got[pdl] = kept
    for x, y in zip(got["1"], got["0"]):
        assert all(torch.isfinite(t.float()).all() and torch.equal(t, u) for t, u in zip(x, y))


def norm_buffers(s, rows, cols, dt, seed):
    from partial_sum_reduction_gb300 import helpers as H
    g = torch.Generator(device="cuda").manual_seed(seed)
    b = {k: torch.randn(rows, cols, generator=g, device="cuda").to(dt) for k in ("x", "res", "dy")}
    b.update({k: torch.empty(rows, cols, device="cuda", dtype=dt) for k in ("t", "y", "dx")})
    b.update({k: torch.empty(rows, device="cuda") for k in ("mean", "rstd")})
    b.update({k: torch.empty(cols, device="cuda") for k in ("dg", "db")})
    b["gamma"], b["beta"] = (torch.rand(cols, generator=g, device="cuda") + 0.5 for _ in range(2))
    b["ws"] = H.layernorm_workspace(rows, cols)
    return b


def norm_step(s, b, stream=None, wait=lambda: None):
    s.shmm_layernorm_forward(b["x"], b["gamma"], b["beta"], b["y"], b["mean"], b["rstd"], residual=b["res"],
                             total=b["t"], stream=stream)
    wait()
    s.shmm_layernorm_backward(b["dy"], b["t"], b["mean"], b["rstd"], b["gamma"], b["dx"], b["dg"], b["db"], b["ws"],
                              residual_grad=b["dy"], stream=stream)
    wait()


NORM_KEYS = ("t", "y", "mean", "rstd", "dx", "dg", "db")
NORM_SIZES = [(4, 4096, torch.bfloat16), (1100, 4096, torch.bfloat16), (1031, 1157, torch.float32), (64, 9000, torch.bfloat16)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols,dt", NORM_SIZES)
def test_norm_chain_gives_the_bits_of_plain_order(s, monkeypatch, rows, cols, dt):
    """The gradient reads what the forward pass in front of it has just
    written; every link's dx is the next one's x."""
    got = {}
    for pdl in ("1", "0"):
        monkeypatch.setenv("SHMM_PDL", pdl)
        b = norm_buffers(s, rows, cols, dt, 1)
        torch.cuda.synchronize()
        for i in range(6):
            norm_step(s, b, wait=torch.cuda.synchronize if pdl == "0" else (lambda: None))
            b["x"], b["dx"] = b["dx"], b["x"]
        s.shmm_sync_status()
        got[pdl] = results(b, NORM_KEYS)
    assert all(torch.isfinite(t.float()).all() and torch.equal(t, u) for t, u in zip(got["1"], got["0"]))


@pytest.mark.gpu
def test_calls_run_on_the_stream_they_are_given(s):
    """Inputs arrive late on a stream that is not the current one; the calls
    given that stream see them."""
    c = Case(s, "rows", 64, 512, 512, 16, 5)
    new = torch.randn(64, 512, generator=torch.Generator().manual_seed(3)).bfloat16()
    b = adapter_buffers(c)
    A = c.H.shard(c.plan, s.TENSOR_A, new)
    adapter_step(c, b, A)
    want = results(b, ADAPTER_KEYS)
    n = norm_buffers(s, 70, 1024, torch.bfloat16, 2)
    x = n["x"].clone()
    norm_step(s, n)
    want_n = results(n, NORM_KEYS)
    for give in ("torch", "handle"):
        side = torch.cuda.Stream()
        late = [torch.zeros_like(t) for t in A]
        b = adapter_buffers(c)
        n["x"].zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
            for t, u in zip(late, A):
                t.copy_(u)
            n["x"].copy_(x)
        to = side if give == "torch" else side.cuda_stream
        adapter_step(c, b, late, stream=to)
        norm_step(s, n, stream=to)
        torch.cuda.synchronize()
        assert all(torch.equal(t, u) for t, u in zip(results(b, ADAPTER_KEYS), want))
        assert all(torch.equal(t, u) for t, u in zip(results(n, NORM_KEYS), want_n))


@pytest.mark.gpu
def test_calls_on_two_streams_at_once(s):
    """Two of everything, each on a stream and a workspace of its own, thirty
    times: the bits of one after the other."""
    for spec in SIZES_OF_EACH_KIND:
        cs = [Case(s, *spec[:6], spec[6], spec[6], seed=q) for q in range(2)]
        bs = [adapter_buffers(c) for c in cs]
        ns = [norm_buffers(s, 1000 + q, 1536, torch.bfloat16, q) for q in range(2)]
        fresh = [[t.clone() for t in b["C"]] for b in bs]
        want = []
        for c, b, n in zip(cs, bs, ns):
            adapter_step(c, b, c.A_r)
            norm_step(s, n)
            want.append(results(b, ADAPTER_KEYS) + results(n, NORM_KEYS))
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        for i in range(30):
            for c, b, n, f, st in zip(cs, bs, ns, fresh, streams):
                with torch.cuda.stream(st):
                    for t, u in zip(b["C"], f):
                        t.copy_(u)
                    adapter_step(c, b, c.A_r)
                    norm_step(s, n)
        torch.cuda.synchronize()
        s.shmm_sync_status()
        for b, n, w in zip(bs, ns, want):
            assert all(torch.equal(t, u) for t, u in zip(results(b, ADAPTER_KEYS) + results(n, NORM_KEYS), w)), spec


@pytest.mark.gpu
@pytest.mark.parametrize("I,J,K,R,n,dt", [(320, 512, 264, 16, 5, "bf16"), (2304, 1024, 520, 16, 9, "bf16"),
                                          (320, 200, 136, 12, 5, "f32")])
def test_gradients_do_not_depend_on_the_order_of_requests(s, I, J, K, R, n, dt):
    """Rows of one adapter scattered over the batch give the bits of the same
    rows in runs: the gradient of A row by row, and that of the factors, whose
    rows are added in ascending order in both."""
    runs = torch.arange(I, dtype=torch.int32) // (I // n) % n
    c = Case(s, "whole", I, J, K, R, n, dt, dt, ids=runs)
    C, low = c.forward()
    dA, dd, du = c.backward(low)
    place = torch.empty(I)
    for a in range(n):  # round robin; ascending within each adapter
        idx = (runs == a).nonzero().flatten()
        place[idx] = torch.arange(len(idx)) * n + a + 0.0
    perm = place.argsort()
    d = Case(s, "whole", I, J, K, R, n, dt, dt, ids=runs[perm])
    for k in ("A", "base", "dC", "dbase"):
        setattr(d, k, getattr(c, k)[perm])
    d.A_r = d.H.shard(d.plan, s.TENSOR_A, d.A)
    Cp, lowp = d.forward()
    dAp, ddp, dup = d.backward(lowp)
    assert torch.equal(low[perm.cuda()], lowp) and torch.equal(C[0][perm.cuda()], Cp[0])
    assert torch.equal(dA[0][perm.cuda()], dAp[0])
    assert torch.equal(dd, ddp) and torch.equal(du, dup)
