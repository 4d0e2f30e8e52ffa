"""Buffers of the training and adapter operators that share memory: refused
where one is read while the other is written.  No GPU: the addresses are made
up and every call ends in its checks."""
import ctypes

import pytest

P = ctypes.c_void_p


def table(addresses):
    return (P * len(addresses))(*addresses)


@pytest.fixture(scope="module")
def s():
    import partial_sum_reduction_gb300 as s
    from partial_sum_reduction_gb300 import build
    build.build()
    return s


def apart(n, first, step=0x100000):
    return [first + i * step for i in range(n)]


def backward(s, plan, dC, A, dA, base=None):
    a = P(0x7000000)
    return s.lib().shmm_adapters_backward(plan.handle, 3, 8, table(dC), table(A), a, a, a, None, a,
                                          None if base is None else table(base), table(dA), a, a, P(0x8000000), 1 << 40, None)


@pytest.mark.parametrize("mesh,sa,sb,sc", [("{X:4}", "I,J", "J,K_X", "I,K_X"), ("{X:2,Y:2}", "I_X,J_Y", "J_Y,K", "I_X,K")])
def test_input_gradient_over_any_rank_s_inputs(s, mesh, sa, sb, sc):
    """A replicated block is read from its lowest rank, whatever rank writes
    over it; part of a buffer is enough."""
    plan = s.Plan(mesh, sa, sb, sc, 8, 32, 32)
    n = plan.nranks
    A, dC, free = apart(n, 0x1000000), apart(n, 0x2000000), apart(n, 0x3000000)
    rows, cols = plan.rank_box(s.TENSOR_A, 0)[1]
    size = rows * cols * 2
    c_rows, c_cols = plan.rank_box(s.TENSOR_C, 0)[1]
    for q in range(n):
        for r in range(n):
            for taken in (A[q], dC[q], A[q] + size - 16, A[q] - size + 16, dC[q] + c_rows * c_cols * 2 - 16):
                dA = list(free)
                dA[r] = taken
                assert backward(s, plan, dC, A, dA) == s.shmm.ERR_UNSUPPORTED, (q, r, hex(taken))
    # shared inputs are no overlap, nor are neighbours; these calls pass every
    # check and end at the device (or, with one, are not made)
    import torch
    if not torch.cuda.is_available():
        assert backward(s, plan, dC, [A[0]] * n, free) == s.shmm.ERR_CUDA
        assert backward(s, plan, dC, A, [a + size for a in A]) == s.shmm.ERR_CUDA


def forward(s, plan, base, C):
    a = P(0x7000000)
    return s.lib().shmm_adapters_forward(plan.handle, 3, 8, table(apart(plan.nranks, 0x1000000)), a, a, a, None,
                                         None if base is None else table(base), table(C), a, None)


@pytest.mark.parametrize("mesh,sa,sb,sc", [("{X:4}", "I,J", "J,K_X", "I,K_X"), ("{X:2,Y:2}", "I_X,J_Y", "J_Y,K", "I_X,K")])
def test_base_shared_by_ranks_and_written_in_place(s, mesh, sa, sb, sc):
    """A rank's base may be its own output, as the same buffer; nothing else
    of what any rank adds to may be written by another."""
    import torch
    plan = s.Plan(mesh, sa, sb, sc, 8, 32, 32)
    n = plan.nranks
    calls = {s.TENSOR_A: lambda base, out: backward(s, plan, apart(n, 0x2000000), apart(n, 0x1000000), out, base),
             s.TENSOR_C: lambda base, out: forward(s, plan, base, out)}
    for tensor, call in calls.items():
        rows, cols = plan.rank_box(tensor, 0)[1]
        size = rows * cols * 2
        free, other = apart(n, 0x3000000), apart(n, 0x4000000)
        for q in range(n):
            for r in range(n):
                for shift in (0, 16 - size, size - 16):
                    if q == r and shift == 0:
                        continue
                    base, out = list(other), list(free)
                    out[r] = base[q] + shift
                    assert call(base, out) == s.shmm.ERR_UNSUPPORTED, (tensor, q, r, shift)
        # one base for all ranks, written in place by one of them
        assert call([free[1]] * n, free) == s.shmm.ERR_UNSUPPORTED
        if not torch.cuda.is_available():  # these pass every check and end at the device
            assert call(free, free) == call([other[0]] * n, free) == call([o + size for o in free], free) == s.shmm.ERR_CUDA
            assert call(None, free) == s.shmm.ERR_CUDA


@pytest.mark.parametrize("mesh,sa,sc", [("{X:4}", "I_X,J", "I,K"), ("{X:2,Y:2}", "I_X,J", "I,K")])
def test_rows_gradient_over_another_rank_s_rows(s, mesh, sa, sc):
    """Ranks that hold copies of an owner block may share its rows, unless one
    of them is written in place."""
    import torch
    plan = s.Plan(mesh, sa, "J,K", sc, 8, 8, 64)
    n = plan.nranks
    rows, cols = plan.rank_box(s.TENSOR_C_REDUCED, 0)[1]
    size = rows * cols * 2
    a, stats = P(0x7000000), table(apart(n, 0x5000000))

    def call(shard, dshard):
        return s.lib().shmm_layernorm_all_gather_backward(
            plan.handle, 0, table(apart(n, 0x2000000)), table(shard), stats, stats, a, table(dshard), a, a,
            P(0x8000000), 1 << 40, None)

    free, other = apart(n, 0x3000000), apart(n, 0x4000000)
    for q in range(n):
        for r in range(n):
            for shift in (0, 16 - size, size - 16):
                if q == r and shift == 0:
                    continue
                out = list(free)
                out[r] = other[q] + shift
                assert call(other, out) == s.shmm.ERR_UNSUPPORTED, (q, r, shift)
    assert call([free[1]] * n, free) == s.shmm.ERR_UNSUPPORTED
    if not torch.cuda.is_available():  # these pass every check and end at the device
        assert call(free, free) == call([other[0]] * n, free) == call([o + size for o in free], free) == s.shmm.ERR_CUDA
