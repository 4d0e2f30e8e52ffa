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
