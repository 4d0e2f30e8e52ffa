"""The order of the 8-bit and gated operators' accesses, within a kernel and
between calls: repeated calls on freshly copied inputs, calls on several streams
at once, early starts against plain stream order, a limit on the SMs."""
import pytest
import torch

import partial_sum_reduction_gb300 as s
from block_util import LAYOUTS, cut, gen, normal


def gated_step(layout, I, J, K, kept, seed=0):
    """(a call of the whole training step on fresh copies, its results)."""
    mesh, sa, sb, sc = LAYOUTS[layout]
    plan = s.Plan(mesh, sa, sb, sc, I, J, K, "bf16", "bf16")
    g = gen(seed)
    full = [(normal(g, *e) / d).bfloat16() for e, d in (((I, J), 1), ((J, K), J ** 0.5), ((J, K), J ** 0.5), ((I, K), 20))]
    tensors = (s.TENSOR_A, s.TENSOR_B, s.TENSOR_B, s.TENSOR_C)
    host = [[t.cpu().pin_memory() for t in cut(plan, k, f)] for k, f in zip(tensors, full)]

    def call(stream=None):
        A, gate, up, dC = ([t.cuda() for t in ts] for ts in host)
        C, saved = s.helpers.alloc(plan, s.TENSOR_C), None if kept == "none" else s.helpers.gated_saved(plan, kept)
        plan.gated_forward(A, gate, up, C, saved=saved, stream=stream)
        if saved is None:
            return C
        outs = [s.helpers.alloc(plan, t) for t in tensors[:3]]
        plan.gated_backward(dC, A, gate, up, saved, *outs, s.helpers.gated_workspace(plan), stream=stream)
        return sum(outs, C)
    return plan, call


def scaled_step(layout, I, J, K, seed=0):
    mesh, sa, sb, sc = LAYOUTS[layout]
    plan = s.Plan(mesh, sa, sb, sc, I, J, K, "e4m3", "bf16")
    g = gen(seed)
    full = [(normal(g, *e) / d).bfloat16() for e, d in (((I, J), 1), ((J, K), J ** 0.5), ((I, K), 20))]
    host = [[t.cpu().pin_memory() for t in cut(plan, k, f)] for k, f in zip((s.TENSOR_A, s.TENSOR_B, s.TENSOR_C), full)]

    def call(stream=None):
        A, B = ([s.helpers.quantize(t.cuda(), br) for t in ts] for ts, br in ((host[0], 1), (host[1], 128)))
        ops = [[x[i] for x in ts] for ts in (A, B) for i in (0, 1)]
        dC, C = [t.cuda() for t in host[2]], s.helpers.alloc(plan, s.TENSOR_C)
        plan.run_scaled(*ops, C, stream=stream)
        dA, dB = (s.helpers.alloc(plan, t, dtype=torch.bfloat16) for t in (s.TENSOR_A, s.TENSOR_B))
        plan.scaled_backward(dC, *ops, dA, dB, s.helpers.scaled_workspace(plan), stream=stream)
        return C + dA + dB
    return plan, call


STEPS = [("gated", "columns", 512, 1024, 2048, "e4m3"), ("gated", "all_reduce", 1024, 512, 1024, "bf16"),
         ("gated", "whole", 16, 4096, 2048, "bf16"), ("gated", "rows", 32, 4096, 4096, "none"), ("gated", "whole", 515, 1024, 1408, "e4m3"),
         ("scaled", "columns", 512, 1024, 2048), ("scaled", "whole", 16, 4096, 2048), ("scaled", "whole", 1000, 1040, 2032),
         ("scaled", "grid", 2048, 2048, 2048)]


def step(case, seed=0):
    return (gated_step if case[0] == "gated" else scaled_step)(*case[1:], seed=seed)


@pytest.mark.gpu
@pytest.mark.parametrize("case", STEPS, ids=lambda c: "-".join(map(str, c)))
def test_many_calls_give_one_result(case):
    _, call = step(case)
    first = call()
    for _ in range(25):
        assert all(torch.equal(a, b) for a, b in zip(call(), first))


@pytest.mark.gpu
def test_several_streams_at_once():
    """Kernels of different shapes side by side: each step's results are those
    of the step alone."""
    made = [step(c, seed=i) for i, c in enumerate(STEPS[:8:2])]
    alone = [call() for _, call in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(6):
        got = []
        for (_, call), st in zip(made, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(call())
        torch.cuda.synchronize()
        for a, b in zip(got, alone):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
@pytest.mark.parametrize("case", STEPS, ids=lambda c: "-".join(map(str, c)))
def test_early_starts_change_nothing(case, monkeypatch):
    _, call = step(case)
    first = call()
    monkeypatch.setenv("SHMM_PDL", "0")
    assert all(torch.equal(a, b) for a, b in zip(call(), first))


@pytest.mark.gpu
@pytest.mark.parametrize("case", STEPS, ids=lambda c: "-".join(map(str, c)))
def test_a_limit_on_the_sms_changes_no_result(case):
    plan, call = step(case)
    first = call()
    for limit in (2, 40):
        plan.set_sm_limit(limit)
        assert all(torch.equal(a, b) for a, b in zip(call(), first))


@pytest.mark.gpu
def test_beside_the_plans_own_matmuls():
    """The gated half, the plan's own matmul and a LayerNorm in turn on one
    stream, over the same buffers each time: nothing starts before what it reads
    is there."""
    T, D, F = 256, 512, 1024
    first = s.Plan("{X:1}", "I,J", "J,K", "I,K", T, D, F, "bf16", "bf16")
    second = s.Plan("{X:1}", "I,J", "J,K", "I,K", T, F, D, "bf16", "bf16")
    g = gen(1)
    x0 = normal(g, T, D).bfloat16()
    gate, up = ((normal(g, D, F) / D ** 0.5).bfloat16() for _ in range(2))
    down = (normal(g, F, D) / F ** 0.5).bfloat16()
    gamma, beta = torch.ones(D, device="cuda"), torch.zeros(D, device="cuda")

    def run(sync):
        x, h, y = x0.clone(), torch.empty(T, F, device="cuda", dtype=torch.bfloat16), torch.empty_like(x0)
        for _ in range(12):
            first.gated_forward([x], [gate], [up], [h])
            if sync:
                torch.cuda.synchronize()
            second.run([h], [down], [y])
            if sync:
                torch.cuda.synchronize()
            s.shmm_layernorm(y, gamma, beta, x)
            if sync:
                torch.cuda.synchronize()
        return x
    want = run(True)
    for _ in range(5):
        assert torch.equal(run(False), want)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f32", "scaled"])
@pytest.mark.parametrize("I,J,K", [(8, 128, 16384), (640, 256, 1024), (24, 4096, 256), (2048, 2048, 1024)])
def test_what_follows_a_backward_pass_waits_for_both_products(kind, I, J, K, monkeypatch):
    """The two products of a backward pass run side by side.  Library calls that
    read dA or overwrite what it is made of, right behind the pass, in a stream
    and from a graph, give what they give in plain stream order."""
    in_dt, dt = ("e4m3", "bf16") if kind == "scaled" else (kind, kind)
    plan = s.Plan("{X:1}", "I,J", "J,K", "I,K", I, J, K, in_dt, dt)
    tdt = torch.float32 if dt == "f32" else torch.bfloat16
    g = gen(3)
    sets = []
    for _ in range(2):
        A, gate, up, dC = ((normal(g, *e) / d).to(tdt) for e, d in (((I, J), 1), ((J, K), J ** 0.5), ((J, K), J ** 0.5), ((I, K), 20)))
        if kind == "scaled":
            a, b = s.helpers.quantize(A, 1), s.helpers.quantize(gate, 128)
            sets.append(([dC], [a[0]], [a[1]], [b[0]], [b[1]]))
        else:
            saved = s.helpers.gated_saved(plan, dt)
            plan.gated_forward([A], [gate], [up], s.helpers.alloc(plan, s.TENSOR_C), saved=saved)
            sets.append(([dC], [A], [gate], [up], saved))
    ws = s.helpers.scaled_workspace(plan) if kind == "scaled" else s.helpers.gated_workspace(plan)
    back = plan.scaled_backward if kind == "scaled" else plan.gated_backward
    out_dt = torch.bfloat16 if kind == "scaled" else tdt
    outs = [[torch.empty(e, device="cuda", dtype=out_dt)] for e in ((I, J), (J, K), (J, K))][:2 if kind == "scaled" else 3]
    codes = [torch.empty(o[0].shape, device="cuda", dtype=torch.float8_e4m3fn) for _ in range(4) for o in outs]
    scales = [torch.empty(s.scale_shape(*c.shape), device="cuda") for c in codes]

    def run():
        for i in range(4):  # one workspace, one set of results, other operands each time
            stream = torch.cuda.current_stream()
            back(*sets[i % 2], *outs, ws, stream=stream)
            for j, o in enumerate(outs):
                s.shmm_quantize(o[0], codes[i * len(outs) + j], scales[i * len(outs) + j], stream=stream)

    def result():
        torch.cuda.synchronize()
        return [c.view(torch.uint8).clone() for c in codes] + [x.clone() for x in scales]

    def clear():
        for c in codes:
            c.view(torch.uint8).zero_()

    monkeypatch.setenv("SHMM_PDL", "0")
    run()
    want = result()
    monkeypatch.delenv("SHMM_PDL")
    for _ in range(5):
        clear()
        run()
        assert all(torch.equal(a, b) for a, b in zip(result(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(5):
        clear()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(result(), want))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["gated", "scaled"])
def test_two_products_take_an_sm_limit_once(kind):
    """With a limit on the SMs a backward pass's products run one after the
    other: both take as long as each alone, together.  (Side by side on SMs of
    their own they would take the longer one's time, some half of it.)"""
    I, J, K = 2048, 2048, 2048
    scaled = kind == "scaled"
    plan = s.Plan("{X:1}", "I,J", "J,K", "I,K", I, J, K, "e4m3" if scaled else "bf16", "bf16")
    g = gen(5)
    A, gate, up, dC = (normal(g, *e).bfloat16() for e in ((I, J), (J, K), (J, K), (I, K)))
    new = lambda t: s.helpers.alloc(plan, t, dtype=torch.bfloat16)
    dA, dgate, dup = new(s.TENSOR_A), new(s.TENSOR_B), new(s.TENSOR_B)
    if scaled:
        (a, a_s), (b, b_s), ws = s.helpers.quantize(A, 1), s.helpers.quantize(gate, 128), s.helpers.scaled_workspace(plan)
        back = lambda x, w: plan.scaled_backward([dC], [a], [a_s], [b], [b_s], x, w, ws)
    else:
        saved, ws = s.helpers.gated_saved(plan, "bf16"), s.helpers.gated_workspace(plan)
        plan.gated_forward([A], [gate], [up], new(s.TENSOR_C), saved=saved)
        back = lambda x, w: plan.gated_backward([dC], [A], [gate], [up], saved, x, w, None if w is None else dup, ws)

    def ms(x, w):
        times = []
        for _ in range(4):
            e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            e0.record()
            back(x, w)
            e1.record()
            e1.synchronize()
            times.append(e0.elapsed_time(e1))
        return min(times)
    plan.set_sm_limit(8)
    assert ms(dA, dgate) > 0.8 * (ms(dA, None) + ms(None, dgate))


@pytest.mark.gpu
@pytest.mark.parametrize("I,J,K", [(0, 128, 256), (16, 0, 256), (16, 128, 0)])
def test_a_backward_pass_with_an_empty_dim(I, J, K):
    """Where a product is left out, the next one waits for what it needs."""
    plan = s.Plan("{X:1}", "I,J", "J,K", "I,K", I, J, K, "bf16", "bf16")
    new = lambda t: s.helpers.alloc(plan, t)
    saved = s.helpers.gated_saved(plan, "bf16")
    A, gate, up, dC, C = (new(t) for t in (s.TENSOR_A, s.TENSOR_B, s.TENSOR_B, s.TENSOR_C, s.TENSOR_C))
    for t in (A, gate, up, dC):
        t[0].normal_()
    outs = [new(t) for t in (s.TENSOR_A, s.TENSOR_B, s.TENSOR_B)]
    for o in outs:
        o[0].fill_(7.0)
    plan.gated_forward(A, gate, up, C, saved=saved)
    plan.gated_backward(dC, A, gate, up, saved, *outs, s.helpers.gated_workspace(plan))
    torch.cuda.synchronize()
    assert all(not o[0].any() for o in outs)
