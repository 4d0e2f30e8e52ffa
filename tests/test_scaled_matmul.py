"""The sharded matmul of 8-bit operands and its gradient against the
definition in 64 bits, on the tensor cores and on the CUDA cores, for every
case of the sharding."""
import ctypes

import pytest
import torch

import partial_sum_reduction_gb300 as s
from partial_sum_reduction_gb300 import shmm as m
from block_util import (BLOCK, DTYPES, E4M3, HALF_STEP, LAYOUTS, assert_ranks, box, cut, gathered, gen, normal, quantized,
                        restored, sum_error)

# sizes that every layout's edges allow on whole blocks, and sizes that they do not
ALIGNED = [(256, 512, 512), (512, 1024, 512), (1024, 512, 1536)]
RAGGED = [(8, 16, 16), (20, 72, 44), (264, 520, 136)]


def operands(seed, plan, I, J, K, scale_seed=None):
    """Per-rank codes and scales, and what they stand for in 64 bits."""
    g = gen(seed)
    A = normal(g, I, J) * torch.exp(normal(g, I, 1))
    A[:, ::9] *= 20.0
    B = normal(g, J, K) / max(J, 1) ** 0.5
    out = []
    for full, tensor, br in ((A.bfloat16(), s.TENSOR_A, 1), (B.bfloat16(), s.TENSOR_B, BLOCK)):
        codes, scales = s.helpers.shard_scaled(plan, tensor, full)
        if scale_seed is not None:  # scales that are no powers of two
            gs = gen(scale_seed)
            per_box = {}
            for r in range(plan.nranks):  # copies of a block have the same scales
                key = plan.rank_box(tensor, r)
                if key not in per_box:
                    per_box[key] = scales[r] * (0.5 + torch.rand(scales[r].shape, generator=gs, device="cuda"))
                scales[r] = per_box[key].clone()
        whole = gathered(plan, tensor, [restored(c, sc, br) for c, sc in zip(codes, scales)], *full.shape)
        out += [codes, scales, whole]
    return out


def run_and_check(layout, I, J, K, out, flags=0, seed=0, scale_seed=None):
    mesh, sa, sb, sc = LAYOUTS[layout]
    plan = s.Plan(mesh, sa, sb, sc, I, J, K, "e4m3", out, flags)
    A, As, wA, B, Bs, wB = operands(seed, plan, I, J, K, scale_seed)
    C = s.helpers.alloc(plan, s.TENSOR_C, fill=7.0)
    plan.run_scaled(A, As, B, Bs, C)
    want, size = wA @ wB, wA.abs() @ wB.abs()
    assert_ranks(plan, s.TENSOR_C, C, want, want.abs() * HALF_STEP[out] + sum_error(J, size), "C")
    return plan, (A, As, wA, B, Bs, wB), C


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("I,J,K", ALIGNED + RAGGED)
@pytest.mark.parametrize("layout", sorted(LAYOUTS))
def test_every_sharding(layout, I, J, K, out):
    run_and_check(layout, I, J, K, out)


@pytest.mark.gpu
@pytest.mark.parametrize("I,J,K", [(1, 128, 128), (1, 4096, 512), (16, 4096, 1024), (17, 1040, 2032), (100, 2048, 256),
                                   (128, 528, 272), (129, 400, 4112), (300, 16, 16), (1000, 1040, 2032), (700, 3000, 640)])
@pytest.mark.parametrize("flags", [0, s.FLAG_SIMT])
def test_sizes(I, J, K, flags):
    run_and_check("whole", I, J, K, "f32", flags, scale_seed=11)
    run_and_check("whole", I, J, K, "bf16", flags)


@pytest.mark.gpu
@pytest.mark.parametrize("layout,I,J,K", [("whole", 37, 53, 71), ("whole", 1, 1, 1), ("rows", 12, 130, 129),
                                          ("columns", 5, 7, 12), ("all_reduce", 6, 270, 33), ("grid", 2, 3, 2)])
def test_odd_sizes_on_the_cuda_cores(layout, I, J, K):
    run_and_check(layout, I, J, K, "f32", scale_seed=2)
    run_and_check(layout, I, J, K, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("layout,I,J,K", [("rows", 32, 1024, 512), ("rows", 96, 4096, 768), ("rows", 12, 512, 256), ("all_reduce", 48, 1024, 512),
                                          ("scatter_rows", 64, 2048, 256), ("columns", 24, 512, 2048), ("whole", 128, 16384, 128)])
def test_few_rows_of_many_ranks(layout, I, J, K):
    """Rows split over the ranks in groups of 8 (and not), long sums shared by several CTAs."""
    run_and_check(layout, I, J, K, "f32", scale_seed=2)
    run_and_check(layout, I, J, K, "bf16")


@pytest.mark.gpu
def test_many_ranks():
    mesh = "{X:32}"
    plan = s.Plan(mesh, "I_X,J", "J,K", "I_X,K", 4096, 256, 256, "e4m3", "bf16")
    A, As, wA, B, Bs, wB = operands(4, plan, 4096, 256, 256)
    C = s.helpers.alloc(plan, s.TENSOR_C)
    plan.run_scaled(A, As, B, Bs, C)
    want = wA @ wB
    assert_ranks(plan, s.TENSOR_C, C, want, want.abs() * HALF_STEP["bf16"] + sum_error(256, wA.abs() @ wB.abs()), "C")


@pytest.mark.gpu
def test_nan_stays_in_its_row():
    plan = s.Plan("{X:1}", "I,J", "J,K", "I,K", 300, 512, 512, "e4m3", "bf16")
    A, As, wA, B, Bs, wB = operands(4, plan, 300, 512, 512)
    clean = s.helpers.alloc(plan, s.TENSOR_C)
    plan.run_scaled(A, As, B, Bs, clean)
    A[0].view(torch.uint8)[7, 100] = 0x7F
    C = s.helpers.alloc(plan, s.TENSOR_C)
    plan.run_scaled(A, As, B, Bs, C)
    assert bool(torch.isnan(C[0][7]).all())
    keep = torch.arange(300, device="cuda") != 7
    assert torch.equal(C[0][keep], clean[0][keep])


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["columns", "all_reduce", "scatter_rows"])
def test_one_input_gives_one_result_and_nothing_else_is_written(layout):
    mesh, sa, sb, sc = LAYOUTS[layout]
    plan = s.Plan(mesh, sa, sb, sc, 512, 1024, 512, "e4m3", "bf16")
    A, As, wA, B, Bs, wB = operands(8, plan, 512, 1024, 512)
    first = None
    for _ in range(5):
        guard = 512
        raw, C = [], []
        for r in range(plan.nranks):
            e = plan.rank_box(s.TENSOR_C, r)[1]
            t = torch.full((guard * 2 + e[0] * e[1],), 3.0, dtype=torch.bfloat16, device="cuda")
            raw.append(t)
            C.append(t[guard:-guard].view(e))
        plan.run_scaled(A, As, B, Bs, C)
        for t in raw:
            assert bool((t[:guard] == 3.0).all()) and bool((t[-guard:] == 3.0).all())
        if first is None:
            first = [c.clone() for c in C]
        assert all(torch.equal(a, b) for a, b in zip(C, first))


# ---- the gradient ----------------------------------------------------------

def grad_and_check(layout, I, J, K, flags=0, seed=0):
    mesh, sa, sb, sc = LAYOUTS[layout]
    plan = s.Plan(mesh, sa, sb, sc, I, J, K, "e4m3", "bf16", flags)
    A, As, wA, B, Bs, wB = operands(seed, plan, I, J, K, 5)
    dC_full = (0.02 * normal(gen(seed + 99), I, K) * torch.exp(normal(gen(seed + 98), I, 1))).bfloat16()
    dC = cut(plan, s.TENSOR_C, dC_full)
    dA = s.helpers.alloc(plan, s.TENSOR_A, dtype=torch.bfloat16, fill=7.0)
    dB = s.helpers.alloc(plan, s.TENSOR_B, dtype=torch.bfloat16, fill=7.0)
    ws = s.helpers.scaled_workspace(plan)
    if ws is not None:
        ws.fill_(255)  # NaN wherever it is read before it is written
    plan.scaled_backward(dC, A, As, B, Bs, dA, dB, ws)
    q = gathered(plan, s.TENSOR_C, [restored(*quantized(t)) for t in dC], I, K)
    want = q @ wB.T
    # values of the restored A are rounded to bf16 where its scales are no powers of two
    assert_ranks(plan, s.TENSOR_A, dA, want, want.abs() * HALF_STEP["bf16"] + sum_error(K, q.abs() @ wB.abs().T), "dA")
    wide = gathered(plan, s.TENSOR_A, [restored(c, sc).bfloat16() for c, sc in zip(A, As)], I, J)
    d = dC_full.double()
    want = wide.T @ d
    assert_ranks(plan, s.TENSOR_B, dB, want, want.abs() * HALF_STEP["bf16"] + sum_error(I, wide.abs().T @ d.abs()), "dB")
    return plan, (A, As, B, Bs), dC, dA, dB, ws


@pytest.mark.gpu
@pytest.mark.parametrize("I,J,K", ALIGNED + RAGGED)
@pytest.mark.parametrize("layout", sorted(LAYOUTS))
def test_gradient_of_every_sharding(layout, I, J, K):
    grad_and_check(layout, I, J, K)


@pytest.mark.gpu
@pytest.mark.parametrize("I,J,K", [(1, 128, 256), (17, 1040, 2032), (1000, 1040, 2032), (300, 16, 16), (129, 400, 4112),
                                   (37, 53, 71)])
@pytest.mark.parametrize("flags", [0, s.FLAG_SIMT])
def test_gradient_sizes(I, J, K, flags):
    grad_and_check("whole", I, J, K, flags)


@pytest.mark.gpu
def test_one_gradient_alone_is_the_same():
    plan, ops, dC, dA, dB, ws = grad_and_check("columns", 512, 1024, 512)
    a, b = [torch.empty_like(t) for t in dA], [torch.empty_like(t) for t in dB]
    plan.scaled_backward(dC, *ops, a, None, ws)
    plan.scaled_backward(dC, *ops, None, b, ws)
    assert all(torch.equal(x, y) for x, y in zip(a + b, dA + dB))


@pytest.mark.gpu
def test_no_rows_and_nothing_to_contract():
    plan = s.Plan("{X:1}", "I,J", "J,K", "I,K", 0, 256, 128, "e4m3", "bf16")
    A, As, wA, B, Bs, wB = operands(1, plan, 0, 256, 128)
    C = s.helpers.alloc(plan, s.TENSOR_C)
    plan.run_scaled(A, As, B, Bs, C)
    dA, dB = (s.helpers.alloc(plan, t, dtype=torch.bfloat16) for t in (s.TENSOR_A, s.TENSOR_B))
    plan.scaled_backward(C, A, As, B, Bs, dA, dB, s.helpers.scaled_workspace(plan))
    assert bool((dB[0] == 0).all())
    plan = s.Plan("{X:1}", "I,J", "J,K", "I,K", 40, 0, 128, "e4m3", "bf16")
    C = s.helpers.alloc(plan, s.TENSOR_C, fill=5.0)
    empty = lambda *e: [torch.empty(*e, device="cuda")]  # noqa: E731
    plan.run_scaled([torch.empty(40, 0, device="cuda").to(E4M3)], empty(40, 0), [torch.empty(0, 128, device="cuda").to(E4M3)],
                    empty(0, 1), C)
    assert bool((C[0] == 0).all())


@pytest.mark.gpu
def test_gradient_against_differences():
    """dB is the gradient of sum(dC * C) by what B stands for; C is linear in
    it, so a difference of two forward calls gives it up to their rounding."""
    I, J, K = 64, 256, 384
    plan = s.Plan("{X:2}", "I,J", "J,K_X", "I,K_X", I, J, K, "e4m3", "f32")
    back = s.Plan("{X:2}", "I,J", "J,K_X", "I,K_X", I, J, K, "e4m3", "bf16")
    A, As, wA, B, Bs, wB = operands(3, plan, I, J, K)
    _, _, _, B2, Bs2, wB2 = operands(4, plan, I, J, K)
    dC_full = normal(gen(9), I, K).bfloat16()
    dA, dB = (s.helpers.alloc(back, t, dtype=torch.bfloat16) for t in (s.TENSOR_A, s.TENSOR_B))
    back.scaled_backward(cut(back, s.TENSOR_C, dC_full), A, As, B, Bs, dA, dB, s.helpers.scaled_workspace(back))
    C, C2 = (s.helpers.alloc(plan, s.TENSOR_C) for _ in range(2))
    plan.run_scaled(A, As, B, Bs, C)
    plan.run_scaled(A, As, B2, Bs2, C2)
    L, L2 = (float((gathered(plan, s.TENSOR_C, c, I, K) * dC_full.double()).sum()) for c in (C, C2))
    g = gathered(back, s.TENSOR_B, dB, J, K)
    by_grad = float((g * (wB2 - wB)).sum())
    # dB's rounding to bf16 on every term, and the forward calls' rounding of every sum
    allowed = float((g.abs() * (wB2 - wB).abs()).sum()) * 2.0 ** -8 + float(
        (sum_error(J, wA.abs() @ (wB.abs() + wB2.abs())) * dC_full.double().abs()).sum())
    assert abs((L2 - L) - by_grad) <= allowed


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    mesh, sa, sb, sc = LAYOUTS["all_reduce"]
    plan = s.Plan(mesh, sa, sb, sc, 256, 512, 512, "e4m3", "bf16")
    A, As, wA, B, Bs, wB = operands(1, plan, 256, 512, 512)
    dC = cut(plan, s.TENSOR_C, (0.1 * normal(gen(2), 256, 512)).bfloat16())
    new = lambda: (s.helpers.alloc(plan, s.TENSOR_C), s.helpers.alloc(plan, s.TENSOR_A, dtype=torch.bfloat16),  # noqa: E731
                   s.helpers.alloc(plan, s.TENSOR_B, dtype=torch.bfloat16))

    def step(C, dA, dB, ws, stream=None):
        plan.run_scaled(A, As, B, Bs, C, stream=stream)
        plan.scaled_backward(dC, A, As, B, Bs, dA, dB, ws, stream=stream)

    want = new()
    step(*want, s.helpers.scaled_workspace(plan))
    other = new()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    ws = s.helpers.scaled_workspace(plan)
    step(*other, ws, st)
    torch.cuda.synchronize()
    graph, third = torch.cuda.CUDAGraph(), new()
    with torch.cuda.graph(graph):
        step(*third, ws)
    for _ in range(2):
        for t in sum(map(list, third), []):
            t.fill_(9.0)
        graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, other, third):
        assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(a, b, c))


# ---- refusals: no GPU is reached ------------------------------------------

def _arr(*p):
    return (ctypes.c_void_p * len(p))(*p)


def _forward(plan, **kw):
    a = dict(A=_arr(1 << 20), As=_arr(1 << 24), B=_arr(1 << 25), Bs=_arr(1 << 26), C=_arr(1 << 27))
    a.update(kw)
    return s.lib().shmm_run_scaled(None if plan is None else plan.handle, a["A"], a["As"], a["B"], a["Bs"], a["C"], None)


def _backward(plan, **kw):
    a = dict(dC=_arr(1 << 27), A=_arr(1 << 20), As=_arr(1 << 24), B=_arr(1 << 25), Bs=_arr(1 << 26), dA=_arr(1 << 28),
             dB=_arr(1 << 29), ws=1 << 30, n=1 << 24)
    a.update(kw)
    return s.lib().shmm_scaled_backward(None if plan is None else plan.handle, a["dC"], a["A"], a["As"], a["B"], a["Bs"],
                                        a["dA"], a["dB"], a["ws"], a["n"], None)


def _plan(flags=0, dt="e4m3", out="bf16", I=64, J=256, K=128):
    return s.Plan("{X:1}", "I,J", "J,K", "I,K", I, J, K, dt, out, flags)


@pytest.mark.parametrize("call", [_forward, _backward])
@pytest.mark.parametrize("kw,status", [
    (dict(A=None), m.ERR_NULL), (dict(As=None), m.ERR_NULL), (dict(B=None), m.ERR_NULL), (dict(Bs=None), m.ERR_NULL),
    (dict(A=_arr(None)), m.ERR_NULL), (dict(As=_arr(None)), m.ERR_NULL), (dict(Bs=_arr(None)), m.ERR_NULL),
    (dict(A=_arr((1 << 20) + 8)), m.ERR_ALIGN), (dict(As=_arr((1 << 24) + 2)), m.ERR_ALIGN),
    (dict(Bs=_arr((1 << 26) + 1)), m.ERR_ALIGN)])
def test_operands_are_checked(call, kw, status):
    assert call(_plan(), **kw) == status


def test_refused_plans():
    assert _forward(None) == m.ERR_NULL and _backward(None) == m.ERR_NULL
    for call in (_forward, _backward):
        assert call(_plan(dt="bf16")) == m.ERR_DTYPE
        assert call(_plan(flags=s.FLAG_GELU)) == m.ERR_UNSUPPORTED
        assert call(_plan(I=1 << 31)) == m.ERR_SHAPE
        assert call(_plan(J=1 << 22)) == m.ERR_SHAPE
        assert call(_plan(K=1 << 22)) == m.ERR_SHAPE
    assert _backward(_plan(out="f32")) == m.ERR_DTYPE
    with pytest.raises(s.ShmmError) as e:
        _plan(dt="bf16").scaled_workspace_size()
    assert e.value.status == m.ERR_DTYPE


def test_a_workspace_over_an_operand_or_a_result_is_refused():
    p = _plan()
    need = p.scaled_workspace_size()
    for at in (1 << 20, 1 << 24, 1 << 25, 1 << 26, 1 << 27, 1 << 28, 1 << 29):
        assert _backward(p, ws=at) == m.ERR_UNSUPPORTED
        assert _backward(p, ws=at - need + 256 & -256) == m.ERR_UNSUPPORTED
    assert _backward(p, dB=_arr((1 << 30) + need - 16)) == m.ERR_UNSUPPORTED


def test_refused_results_and_workspaces():
    p = _plan()
    assert _forward(p, C=None) == m.ERR_NULL and _forward(p, C=_arr((1 << 27) + 4)) == m.ERR_ALIGN
    for over in (1 << 20, (1 << 20) + 64 * 256 - 16, 1 << 24, 1 << 25, 1 << 26):
        assert _forward(p, C=_arr(over)) == m.ERR_UNSUPPORTED
        assert _backward(p, dA=_arr(over)) == m.ERR_UNSUPPORTED
        assert _backward(p, dB=_arr(over)) == m.ERR_UNSUPPORTED
    assert _backward(p, dA=_arr(1 << 27)) == m.ERR_UNSUPPORTED  # over dC
    assert _backward(p, dB=_arr(1 << 28)) == m.ERR_UNSUPPORTED  # over dA
    need = p.scaled_workspace_size()
    assert need == 64 * 128 + 256 + 64 * 256 * 2
    assert _backward(p, n=need - 1) == m.ERR_NOMEM and _backward(p, ws=None) == m.ERR_NULL
    assert _backward(p, ws=(1 << 30) + 128) == m.ERR_ALIGN


def test_other_calls_refuse_the_plan():
    p, lib = _plan(flags=s.FLAG_FUSED), s.lib()
    A, B, C = _arr(1 << 20), _arr(1 << 25), _arr(1 << 27)
    assert lib.shmm_run(p.handle, A, B, C, None, 0, None) == m.ERR_DTYPE
    assert lib.shmm_run_static_workspace(p.handle, A, B, C, None) == m.ERR_DTYPE
    assert lib.shmm_run_host(p.handle, None, None, None, A, B, C, None, 0, None) == m.ERR_DTYPE
    assert lib.shmm_local_matmul(p.handle, A, B, C, None) == m.ERR_DTYPE
    assert lib.shmm_adapters_forward(p.handle, 1, 4, A, 4096, 4096, 4096, None, None, C, 4096, None) == m.ERR_DTYPE
    g = s.Plan("{X:2}", "I,J_X", "J,K", "I,K", 64, 256, 128, "e4m3", "bf16")
    two = _arr(1 << 20, 1 << 21)
    assert lib.shmm_all_gather(g.handle, s.TENSOR_A, two, two, None) == m.ERR_DTYPE


def test_injected_failure(monkeypatch):
    monkeypatch.setenv("SHMM_INJECT_FAIL", "shmm_run_scaled,shmm_scaled_backward")
    assert _forward(_plan()) == m.ERR_INJECTED and _backward(_plan()) == m.ERR_INJECTED


def test_the_plan_counts_bytes_of_8_bit_operands():
    p = s.Plan("{X:2}", "I,J_X", "J,K", "I,K", 64, 256, 128, "e4m3", "bf16")
    assert p.info.payload_operand_ag == 64 * 128  # a [64, 128] shard to one peer, a byte a value
    assert p.info.in_dtype == m.E4M3 and p.info.out_dtype == m.BF16 and p.info.tensor_core == 0
    assert box(p, s.TENSOR_A, 1, torch.zeros(64, 256)).shape == (64, 128)
    assert DTYPES["bf16"] is torch.bfloat16
