"""The gated first half of an MLP block and its gradient against the definition
in 64 bits, for every case of the sharding, every type that is kept, on the
tensor cores and on the CUDA cores."""
import ctypes

import pytest
import torch

import partial_sum_reduction_gb300 as s
from partial_sum_reduction_gb300 import shmm as m
from block_util import (DTYPES, HALF_STEP, LAYOUTS, assert_ranks, box, cut, gate_act, gathered, gen, normal, quantized,
                        restored, sum_error)

ALIGNED = [(256, 512, 512), (512, 1024, 512)]
RAGGED = [(8, 16, 16), (20, 72, 44), (264, 520, 136)]


def inputs(seed, I, J, K, dtype):
    g = gen(seed)
    dt = DTYPES[dtype]
    A = normal(g, I, J).to(dt)
    gate, up = ((1.5 * normal(g, J, K) / max(J, 1) ** 0.5).to(dt) for _ in range(2))
    return A, gate, up


def kept_values(saved):
    """What was kept, in 64 bits, per rank."""
    if saved.dtype == "e4m3":
        return [[restored(c, sc) for c, sc in zip(cs, scs)]
                for cs, scs in ((saved.gate, saved.gate_scale), (saved.up, saved.up_scale))]
    return [[t.double() for t in ts] for ts in (saved.gate, saved.up)]


def forward_and_check(layout, I, J, K, dtype, act, kept, flags=0, seed=0):
    mesh, sa, sb, sc = LAYOUTS[layout]
    plan = s.Plan(mesh, sa, sb, sc, I, J, K, dtype, dtype, flags)
    A, gate, up = inputs(seed, I, J, K, dtype)
    A_r, gate_r, up_r = cut(plan, s.TENSOR_A, A), cut(plan, s.TENSOR_B, gate), cut(plan, s.TENSOR_B, up)
    C = s.helpers.alloc(plan, s.TENSOR_C, fill=7.0)
    saved = None if kept == "none" else s.helpers.gated_saved(plan, kept)
    plan.gated_forward(A_r, gate_r, up_r, C, activation=act, saved=saved)
    a, g, u = A.double(), A.double() @ gate.double(), A.double() @ up.double()
    eg, eu = (sum_error(J, a.abs() @ w.double().abs()) for w in (gate, up))
    v, _ = gate_act(act, g)
    # the activations' slopes stay below 1.13; their own rounding is a few units of 2^-23 of the argument
    # (the exponential's) times the value
    ea = 1.13 * eg + (8 + 4 * g.abs()) * 2.0 ** -23 * v.abs()
    h = HALF_STEP[dtype]
    assert_ranks(plan, s.TENSOR_C, C, v * u, (v * u).abs() * (h + 2.0 ** -23) + ea * (u.abs() + eu) + v.abs() * eu, "C")
    if saved is not None:
        for got, want, e, what in zip(kept_values(saved), (g, u), (eg, eu), ("gate", "up")):
            if kept == "e4m3":
                # half a step of e4m3, or half of its smallest step times the scale (which a sum near its border may double)
                scale = gathered(plan, s.TENSOR_C, [restored(torch.ones_like(c.float()).to(c.dtype), sc) for c, sc in zip(
                    saved.gate if what == "gate" else saved.up,
                    saved.gate_scale if what == "gate" else saved.up_scale)], I, K)
                bound = torch.maximum((want.abs() + e) * 2.0 ** -4, scale * 2.0 ** -10) + e
            else:
                bound = want.abs() * h + e
            assert_ranks(plan, s.TENSOR_C, got, want, bound, what)
    return plan, (A, gate, up), (A_r, gate_r, up_r), C, saved


def kinds(dtype):
    return ["none", dtype, "e4m3"]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kept", [(d, k) for d in ("bf16", "f32") for k in kinds(d)])
@pytest.mark.parametrize("I,J,K", ALIGNED + RAGGED)
@pytest.mark.parametrize("layout", sorted(LAYOUTS))
def test_every_sharding(layout, I, J, K, dtype, kept):
    forward_and_check(layout, I, J, K, dtype, "silu", kept)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("kept", kinds("bf16"))
@pytest.mark.parametrize("I,J,K", [(1, 64, 128), (1, 4096, 512), (4, 2048, 1024), (16, 1024, 4096), (33, 1000, 264), (128, 520, 272),
                                   (129, 400, 4112), (300, 8, 16), (515, 1024, 2816), (37, 53, 71), (1, 1, 1), (260, 72, 1000)])
def test_sizes(I, J, K, act, kept):
    forward_and_check("whole", I, J, K, "bf16", act, kept)


@pytest.mark.gpu
@pytest.mark.parametrize("kept", kinds("bf16"))
@pytest.mark.parametrize("layout,I,J,K", [("rows", 32, 1024, 512), ("rows", 96, 4096, 768), ("rows", 12, 512, 256), ("all_reduce", 48, 1024, 512),
                                          ("scatter_rows", 64, 2048, 256), ("columns", 24, 512, 2048), ("whole", 128, 16384, 128)])
def test_few_rows_of_many_ranks(layout, I, J, K, kept):
    """Rows split over the ranks in groups of 8 (and not), long sums shared by several CTAs."""
    forward_and_check(layout, I, J, K, "bf16", "silu", kept)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("I,J,K", [(301, 1000, 1157), (1, 1, 1), (5, 37, 300), (64, 4096, 128)])
def test_fp32_sizes(I, J, K, act):
    for kept in kinds("f32"):
        forward_and_check("whole", I, J, K, "f32", act, kept)


@pytest.mark.gpu
def test_large_and_small_pre_activations():
    """Gates of hundreds: the activation is the value itself, or zero."""
    plan = s.Plan("{X:1}", "I,J", "J,K", "I,K", 256, 64, 128, "bf16", "bf16")
    A = torch.zeros(256, 64, device="cuda", dtype=torch.bfloat16)
    A[:, 0] = torch.linspace(-300, 300, 256).bfloat16()
    gate, up = (torch.zeros(64, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    gate[0], up[0] = 100.0, 0.01
    for act in ("silu", "gelu"):
        C = s.helpers.alloc(plan, s.TENSOR_C)
        saved = s.helpers.gated_saved(plan, "bf16")
        plan.gated_forward([A], [gate], [up], C, activation=act, saved=saved)
        g, u = A.double() @ gate.double(), A.double() @ up.double()
        assert bool(torch.isfinite(C[0]).all())
        want = gate_act(act, g)[0] * u
        # e^-z below 2^-126, fp32's smallest normal value, is taken as zero: the value is off by |g| 2^-126 |u| at most
        # (the definition's own, |g| e^-|g|, is 1e-49 at the first negative gate, -118, and no bf16 or fp32 number)
        assert bool(((C[0].double() - want).abs() <= want.abs() * 2.0 ** -7 + (g * u).abs() * 2.0 ** -126).all())
        dA, dg, du = s.helpers.alloc(plan, s.TENSOR_A), s.helpers.alloc(plan, s.TENSOR_B), s.helpers.alloc(plan, s.TENSOR_B)
        plan.gated_backward([torch.ones_like(C[0])], [A], [gate], [up], saved, dA, dg, du, s.helpers.gated_workspace(plan),
                            activation=act)
        assert all(bool(torch.isfinite(t[0]).all()) for t in (dA, dg, du))


# ---- the gradient ----------------------------------------------------------

def backward_and_check(layout, I, J, K, dtype, act, kept, flags=0, seed=0, rebuild=True):
    plan, (A, gate, up), ops, C, saved = forward_and_check(layout, I, J, K, dtype, act, kept, flags, seed)
    dC_full = (0.05 * normal(gen(seed + 77), I, K)).to(DTYPES[dtype])
    dC = cut(plan, s.TENSOR_C, dC_full)
    dA, dgate, dup = (s.helpers.alloc(plan, t, fill=7.0) for t in (s.TENSOR_A, s.TENSOR_B, s.TENSOR_B))
    again = s.helpers.alloc(plan, s.TENSOR_C, fill=7.0) if rebuild else None
    ws = s.helpers.gated_workspace(plan)
    if ws is not None:
        ws.fill_(255)  # NaN wherever it is read before it is written
    plan.gated_backward(dC, *ops, saved, dA, dgate, dup, ws, activation=act, C_r=again)
    # from the values as they were kept
    g, u = (gathered(plan, s.TENSOR_C, k, I, K) for k in kept_values(saved))
    v, slope = gate_act(act, g)
    d = dC_full.double()
    dg, du, h = d * u * slope, d * v, HALF_STEP[dtype]
    # their own rounding to the operands' type, and the activations' (as above; a slope is the sum of two such terms)
    few = (16 + 8 * g.abs()) * 2.0 ** -23
    eg = dg.abs() * h + (d * u).abs() * few * (1 + g.abs())
    eu = du.abs() * (h + few)
    a, wg, wu = A.double(), gate.double(), up.double()
    want = dg @ wg.T + du @ wu.T
    size = dg.abs() @ wg.abs().T + du.abs() @ wu.abs().T
    checks = [("dA", s.TENSOR_A, dA, want, eg @ wg.abs().T + eu @ wu.abs().T + sum_error(2 * K, size))]
    for what, got, x, e in (("dgate", dgate, dg, eg), ("dup", dup, du, eu)):
        checks.append((what, s.TENSOR_B, got, a.T @ x, a.abs().T @ e + sum_error(I, a.abs().T @ x.abs())))
    for what, tensor, got, want, e in checks:
        assert_ranks(plan, tensor, got, want, want.abs() * h + e, what)
        # errors of random sign: each rounding's root mean square is at most half a step / sqrt(3), and the operands'
        # and the result's add up in squares to 0.82 half steps of the result
        if dtype == "bf16" and want.numel() >= 10000:
            whole = gathered(plan, tensor, got, *want.shape)
            assert float((whole - want).norm()) <= 2.0 ** -8 * float(want.norm())
    if rebuild:
        want = v * u
        assert_ranks(plan, s.TENSOR_C, again, want, want.abs() * (h + (8 + 4 * g.abs()) * 2.0 ** -23), "C again")
    return plan, ops, dC, saved, (dA, dgate, dup), ws


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kept", [("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32"), ("f32", "e4m3")])
@pytest.mark.parametrize("I,J,K", ALIGNED + RAGGED)
@pytest.mark.parametrize("layout", sorted(LAYOUTS))
def test_gradient_of_every_sharding(layout, I, J, K, dtype, kept):
    backward_and_check(layout, I, J, K, dtype, "silu", kept)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("kept", ["bf16", "e4m3"])
@pytest.mark.parametrize("I,J,K", [(1, 64, 128), (4, 2048, 1024), (33, 1000, 264), (129, 400, 4112), (300, 8, 16), (515, 1024, 2816),
                                   (37, 53, 71), (260, 72, 1000)])
def test_gradient_sizes(I, J, K, act, kept):
    backward_and_check("whole", I, J, K, "bf16", act, kept)


@pytest.mark.gpu
def test_gradient_on_the_cuda_cores():
    backward_and_check("all_reduce", 256, 512, 512, "bf16", "gelu", "e4m3", s.FLAG_SIMT)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_against_differences(act):
    """Along a random direction of A, gate and up: the slope of sum(dC * C) by
    differences of the definition in 64 bits, against the fp32 gradients."""
    I, J, K = 40, 96, 160
    plan = s.Plan("{X:2}", "I,J", "J,K_X", "I,K_X", I, J, K, "f32", "f32")
    x = inputs(5, I, J, K, "f32")
    ops = [cut(plan, t, f) for t, f in zip((s.TENSOR_A, s.TENSOR_B, s.TENSOR_B), x)]
    saved, C = s.helpers.gated_saved(plan), s.helpers.alloc(plan, s.TENSOR_C)
    plan.gated_forward(*ops, C, activation=act, saved=saved)
    dC = normal(gen(6), I, K)
    outs = [s.helpers.alloc(plan, t) for t in (s.TENSOR_A, s.TENSOR_B, s.TENSOR_B)]
    plan.gated_backward(cut(plan, s.TENSOR_C, dC), *ops, saved, *outs, s.helpers.gated_workspace(plan), activation=act)
    way = [normal(gen(7 + i), *f.shape).double() for i, f in enumerate(x)]

    def loss(t):
        a, g, u = (f.double() + t * w for f, w in zip(x, way))
        return float((dC.double() * gate_act(act, a @ g)[0] * (a @ u)).sum())

    step = 1e-5
    slope = (loss(step) - loss(-step)) / (2 * step)
    grads = [gathered(plan, t, o, *f.shape) for t, o, f in zip((s.TENSOR_A, s.TENSOR_B, s.TENSOR_B), outs, x)]
    by_grad = sum(float((g * w).sum()) for g, w in zip(grads, way))
    size = sum(float((g * w).abs().sum()) for g, w in zip(grads, way))
    # fp32 sums of up to 2 * 160 products: 2^-23 * 400 of their size at most; the difference's own error is of order step^2
    assert abs(slope - by_grad) <= 400 * 2.0 ** -23 * size + 1e-6 * abs(slope)


@pytest.mark.gpu
def test_parts_of_the_gradient_alone():
    plan, ops, dC, saved, (dA, dgate, dup), ws = backward_and_check("columns", 512, 1024, 512, "bf16", "silu", "e4m3")
    a, g, u = ([torch.empty_like(t) for t in ts] for ts in (dA, dgate, dup))
    plan.gated_backward(dC, *ops, saved, a, None, None, ws)
    plan.gated_backward(dC, *ops, saved, None, g, u, ws)
    assert all(torch.equal(x, y) for x, y in zip(a + g + u, dA + dgate + dup))


@pytest.mark.gpu
def test_no_rows_and_nothing_to_contract():
    plan = s.Plan("{X:1}", "I,J", "J,K", "I,K", 0, 64, 128, "bf16", "bf16")
    ops = [s.helpers.alloc(plan, t, fill=1.0) for t in (s.TENSOR_A, s.TENSOR_B, s.TENSOR_B)]
    C, saved = s.helpers.alloc(plan, s.TENSOR_C), s.helpers.gated_saved(plan, "e4m3")
    plan.gated_forward(*ops, C, saved=saved)
    outs = [s.helpers.alloc(plan, t, fill=7.0) for t in (s.TENSOR_A, s.TENSOR_B, s.TENSOR_B)]
    plan.gated_backward(C, *ops, saved, *outs, s.helpers.gated_workspace(plan))
    assert bool((outs[1][0] == 0).all()) and bool((outs[2][0] == 0).all())
    plan = s.Plan("{X:1}", "I,J", "J,K", "I,K", 40, 0, 128, "bf16", "bf16")
    ops = [s.helpers.alloc(plan, t) for t in (s.TENSOR_A, s.TENSOR_B, s.TENSOR_B)]
    C, saved = s.helpers.alloc(plan, s.TENSOR_C, fill=7.0), s.helpers.gated_saved(plan, "bf16")
    plan.gated_forward(*ops, C, saved=saved)
    assert bool((C[0] == 0).all()) and bool((saved.gate[0] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("where", ["A", "gate"])
def test_nan_stays_where_it_is(where):
    plan = s.Plan("{X:1}", "I,J", "J,K", "I,K", 300, 512, 512, "bf16", "bf16")
    A, gate, up = inputs(4, 300, 512, 512, "bf16")
    clean, C = s.helpers.alloc(plan, s.TENSOR_C), s.helpers.alloc(plan, s.TENSOR_C)
    # the same call as below: what is kept may choose the kernel, and with it how a sum is split
    plan.gated_forward([A], [gate], [up], clean, saved=s.helpers.gated_saved(plan, "e4m3"))
    (A if where == "A" else gate)[7, 100] = float("nan")
    saved = s.helpers.gated_saved(plan, "e4m3")
    plan.gated_forward([A], [gate], [up], C, saved=saved)
    bad = torch.zeros(300, 512, dtype=torch.bool, device="cuda")
    if where == "A":
        bad[7] = True
    else:
        bad[:, 100] = True
    assert bool(torch.isnan(C[0][bad]).all()) and torch.equal(C[0][~bad], clean[0][~bad])
    assert bool(torch.isfinite(saved.gate_scale[0]).all())
    assert torch.equal(torch.isnan(saved.gate[0].float()), bad)


@pytest.mark.gpu
@pytest.mark.parametrize("kept", ["bf16", "e4m3"])
def test_one_input_gives_one_result_and_nothing_else_is_written(kept):
    mesh, sa, sb, sc = LAYOUTS["all_reduce"]
    I, J, K = 264, 512, 272
    plan = s.Plan(mesh, sa, sb, sc, I, J, K, "bf16", "bf16")
    x = inputs(3, I, J, K, "bf16")
    ops = [cut(plan, t, f) for t, f in zip((s.TENSOR_A, s.TENSOR_B, s.TENSOR_B), x)]
    raw = []

    def guarded(tensor, dtype):
        out = []
        for r in range(plan.nranks):
            e = plan.rank_box(tensor, r)[1]
            if dtype == "scale":
                e = s.scale_shape(*e)
            dt = {"scale": torch.float32, "e4m3": torch.uint8}.get(dtype, torch.bfloat16)
            t = torch.full((1024 + e[0] * e[1],), 3, dtype=dt, device="cuda")
            raw.append(t)
            v = t[512:-512].view(e)
            out.append(v.view(torch.float8_e4m3fn) if dtype == "e4m3" else v)
        return out

    first = None
    for _ in range(4):
        del raw[:]
        C = guarded(s.TENSOR_C, "bf16")
        e8 = kept == "e4m3"
        saved = s.GatedSaved(kept, guarded(s.TENSOR_C, kept), guarded(s.TENSOR_C, kept),
                             guarded(s.TENSOR_C, "scale") if e8 else None, guarded(s.TENSOR_C, "scale") if e8 else None)
        plan.gated_forward(*ops, C, saved=saved)
        outs = [guarded(t, "bf16") for t in (s.TENSOR_A, s.TENSOR_B, s.TENSOR_B)]
        plan.gated_backward(C, *ops, saved, *outs, s.helpers.gated_workspace(plan))
        for t in raw:
            assert bool((t[:512] == 3).all()) and bool((t[-512:] == 3).all())
        now = [t.clone() for t in raw]
        if first is None:
            first = now
        assert all(torch.equal(a, b) for a, b in zip(now, first))


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    mesh, sa, sb, sc = LAYOUTS["columns"]
    I, J, K = 256, 512, 512
    plan = s.Plan(mesh, sa, sb, sc, I, J, K, "bf16", "bf16")
    ops = [cut(plan, t, f) for t, f in zip((s.TENSOR_A, s.TENSOR_B, s.TENSOR_B), inputs(3, I, J, K, "bf16"))]
    dC = cut(plan, s.TENSOR_C, normal(gen(2), I, K).bfloat16())
    new = lambda: [s.helpers.alloc(plan, t) for t in (s.TENSOR_C, s.TENSOR_A, s.TENSOR_B, s.TENSOR_B)]  # noqa: E731

    def step(o, saved, ws, stream=None):
        plan.gated_forward(*ops, o[0], saved=saved, stream=stream)
        plan.gated_backward(dC, *ops, saved, *o[1:], ws, stream=stream)

    want, saved, ws = new(), s.helpers.gated_saved(plan, "e4m3"), s.helpers.gated_workspace(plan)
    step(want, saved, ws)
    other, st = new(), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    step(other, saved, ws, st)
    torch.cuda.synchronize()
    graph, third = torch.cuda.CUDAGraph(), new()
    with torch.cuda.graph(graph):
        step(third, saved, ws)
    for _ in range(2):
        for t in sum(third, []):
            t.fill_(9.0)
        graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, other, third):
        assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(a, b, c))


@pytest.mark.gpu
def test_the_mlp_block_together():
    """A gated MLP block's training step as it is used: first half, second
    matmul (row-parallel, all-reduced), and back: the second matmul's own
    gradient by plain products, C rebuilt from the 8-bit checkpoints."""
    T, D, F = 512, 256, 1024
    first = s.Plan("{X:4}", "I,J", "J,K_X", "I,K_X", T, D, F, "bf16", "bf16")
    second = s.Plan("{X:4}", "I,J_X", "J_X,K", "I,K", T, F, D, "bf16", "bf16", s.FLAG_FUSED)
    A, gate, up = inputs(1, T, D, F, "bf16")
    down = (normal(gen(2), F, D) / F ** 0.5).bfloat16()
    ops = [cut(first, t, f) for t, f in zip((s.TENSOR_A, s.TENSOR_B, s.TENSOR_B), (A, gate, up))]
    down_r = cut(second, s.TENSOR_B, down)
    H, Y, saved = s.helpers.alloc(first, s.TENSOR_C), s.helpers.alloc(second, s.TENSOR_C), s.helpers.gated_saved(first, "e4m3")
    first.gated_forward(*ops, H, saved=saved)
    second.run(H, down_r, Y, s.helpers.workspace(second))
    dY = (0.1 * normal(gen(3), T, D)).bfloat16()
    dH_full = (dY.double() @ down.double().T).bfloat16()
    outs = [s.helpers.alloc(first, t) for t in (s.TENSOR_A, s.TENSOR_B, s.TENSOR_B)]
    H2 = s.helpers.alloc(first, s.TENSOR_C)
    first.gated_backward(cut(first, s.TENSOR_C, dH_full), *ops, saved, *outs, s.helpers.gated_workspace(first), C_r=H2)
    # the whole block in 64 bits, differentiated by torch
    x = [t.double().requires_grad_() for t in (A, gate, up)]
    h = torch.nn.functional.silu(x[0] @ x[1]) * (x[0] @ x[2])
    y = h @ down.double()
    y.backward(dY.double())
    y_off = float((gathered(second, s.TENSOR_C, Y, T, D) - y.detach()).norm() / y.detach().norm())
    assert y_off <= 2.0 ** -7  # H's rounding and Y's, half a step of bf16 each
    for t, o, f in zip((s.TENSOR_A, s.TENSOR_B, s.TENSOR_B), outs, x):
        got = gathered(first, t, o, *f.shape)
        # 8-bit checkpoints: each of the two kept values is off by at most 2^-4, with a root mean square of 2^-4 / sqrt(3)
        # at most, and enters a gradient's terms with a weight of order one: two of them, 2^-4
        assert float((got - f.grad).norm()) <= 2.0 ** -4 * float(f.grad.norm())
    h_off = float((gathered(first, s.TENSOR_C, H2, T, F) - h.detach()).norm() / h.detach().norm())
    assert h_off <= 2.0 ** -3  # two values off by 2^-4 at most each


# ---- refusals: no GPU is reached ------------------------------------------

def _arr(*p):
    return (ctypes.c_void_p * len(p))(*p)


def _saved(dtype=m.E4M3, gate=1 << 32, up=1 << 33, gs=1 << 34, us=1 << 35):
    keep = [None if p is None else _arr(p) for p in (gate, up, gs, us)]
    st = m.shmm_gated_saved_t(dtype, *[None if k is None else ctypes.addressof(k) for k in keep])
    st.keep = keep
    return st


def _forward(plan, act=m.SILU, **kw):
    a = dict(A=_arr(1 << 20), gate=_arr(1 << 24), up=_arr(1 << 25), C=_arr(1 << 27), saved=None)
    a.update(kw)
    return s.lib().shmm_gated_forward(None if plan is None else plan.handle, act, a["A"], a["gate"], a["up"], a["C"],
                                      None if a["saved"] is None else ctypes.byref(a["saved"]), None)


def _backward(plan, act=m.SILU, **kw):
    a = dict(dC=_arr(1 << 27), A=_arr(1 << 20), gate=_arr(1 << 24), up=_arr(1 << 25), saved=_saved(), dA=_arr(1 << 28),
             dgate=_arr(1 << 29), dup=_arr(1 << 30), C=None, ws=1 << 31, n=1 << 24)
    a.update(kw)
    return s.lib().shmm_gated_backward(None if plan is None else plan.handle, act, a["dC"], a["A"], a["gate"], a["up"],
                                       None if a["saved"] is None else ctypes.byref(a["saved"]), a["dA"], a["dgate"],
                                       a["dup"], a["C"], a["ws"], a["n"], None)


def _plan(flags=0, dt="bf16", out="bf16", I=64, J=256, K=128):
    return s.Plan("{X:1}", "I,J", "J,K", "I,K", I, J, K, dt, out, flags)


def test_refused_plans():
    for call in (_forward, _backward):
        assert call(None) == m.ERR_NULL
        assert call(_plan(dt="e4m3")) == m.ERR_DTYPE
        assert call(_plan(out="f32")) == m.ERR_DTYPE
        assert call(_plan(flags=s.FLAG_GELU)) == m.ERR_UNSUPPORTED
        assert call(_plan(), act=7) == m.ERR_UNSUPPORTED
        assert call(_plan(I=1 << 31)) == m.ERR_SHAPE
        assert call(_plan(J=1 << 22)) == m.ERR_SHAPE
        assert call(_plan(K=1 << 22)) == m.ERR_SHAPE
    for dt, out in (("e4m3", "bf16"), ("bf16", "f32")):
        with pytest.raises(s.ShmmError) as e:
            _plan(dt=dt, out=out).gated_workspace_size()
        assert e.value.status == m.ERR_DTYPE


@pytest.mark.parametrize("call", [_forward, _backward])
def test_refused_pointers(call):
    p = _plan()
    for name, at in (("A", 1 << 20), ("gate", 1 << 24), ("up", 1 << 25)):
        assert call(p, **{name: None}) == m.ERR_NULL
        assert call(p, **{name: _arr(None)}) == m.ERR_NULL
        assert call(p, **{name: _arr(at + 8)}) == m.ERR_ALIGN
    for kw, status in ((dict(gate=None), m.ERR_NULL), (dict(up=None), m.ERR_NULL), (dict(gs=None), m.ERR_NULL),
                       (dict(us=None), m.ERR_NULL), (dict(gate=(1 << 32) + 4), m.ERR_ALIGN),
                       (dict(gs=(1 << 34) + 1), m.ERR_ALIGN), (dict(dtype=m.F32), m.ERR_DTYPE), (dict(dtype=8), m.ERR_DTYPE)):
        assert call(p, saved=_saved(**kw)) == status


def test_a_workspace_over_an_operand_or_a_result_is_refused():
    p = _plan()
    need = p.gated_workspace_size()
    for at in (1 << 20, 1 << 24, 1 << 25, 1 << 27, 1 << 28, 1 << 29, 1 << 30, 1 << 32, 1 << 35):
        assert _backward(p, ws=at) == m.ERR_UNSUPPORTED
        assert _backward(p, ws=at - need + 256) == m.ERR_UNSUPPORTED
    assert _backward(p, C=_arr((1 << 31) + need - 16)) == m.ERR_UNSUPPORTED


def test_refused_overlaps_and_workspaces():
    p = _plan()
    for over in (1 << 20, 1 << 24, (1 << 25) + 256 * 128 * 2 - 16):
        assert _forward(p, C=_arr(over)) == m.ERR_UNSUPPORTED
        assert _forward(p, saved=_saved(gate=over)) == m.ERR_UNSUPPORTED
        assert _forward(p, saved=_saved(us=over)) == m.ERR_UNSUPPORTED
        for out in ("dA", "dgate", "dup", "C"):
            assert _backward(p, **{out: _arr(over)}) == m.ERR_UNSUPPORTED
    for over in (1 << 27, 1 << 32, 1 << 35):
        assert _backward(p, dA=_arr(over)) == m.ERR_UNSUPPORTED
        assert _backward(p, C=_arr(over)) == m.ERR_UNSUPPORTED
    assert _backward(p, dup=_arr(1 << 29)) == m.ERR_UNSUPPORTED and _backward(p, C=_arr(1 << 28)) == m.ERR_UNSUPPORTED
    assert _forward(p, saved=_saved(up=1 << 32)) == m.ERR_UNSUPPORTED
    assert _forward(p, saved=_saved(gs=1 << 27)) == m.ERR_UNSUPPORTED
    assert _backward(p, saved=None) == m.ERR_NULL
    assert _backward(p, dgate=None) == m.ERR_NULL and _backward(p, dup=None) == m.ERR_NULL
    need = p.gated_workspace_size()
    assert need == 2 * 64 * 128 * 2
    assert _backward(p, n=need - 1) == m.ERR_NOMEM and _backward(p, ws=None) == m.ERR_NULL
    assert _backward(p, ws=(1 << 31) + 16) == m.ERR_ALIGN


def test_injected_failure(monkeypatch):
    monkeypatch.setenv("SHMM_INJECT_FAIL", "shmm_gated_forward,shmm_gated_backward")
    assert _forward(_plan()) == m.ERR_INJECTED and _backward(_plan()) == m.ERR_INJECTED


def test_the_binding_checks_arguments():
    p = _plan()
    t = [torch.zeros(64, 256, dtype=torch.bfloat16)]
    with pytest.raises(ValueError):
        p.gated_forward(t, t, t, t)
    with pytest.raises(ValueError):
        p._saved(s.GatedSaved("int4", t, t), -2)
    with pytest.raises(ValueError):
        m._activation("relu")
    assert box(p, s.TENSOR_B, 0, torch.zeros(256, 128)).shape == (256, 128)
    assert quantized(torch.ones(2, 3))[1].shape == (2, 1)
