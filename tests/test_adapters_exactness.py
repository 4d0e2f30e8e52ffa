"""What the adapters' sums keep: every bit of the low-rank values that are
operands of the next product, and a rounding (not a cut) per step of a long
sum.

The first cases need no tolerance.  Their sums are exact in fp32 in any order: all
terms are multiples of 2^-20 and no partial sum exceeds 4."""
import pytest
import torch

from parity_util import lib

E = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def s():
    return lib()


def repeated(row, rows, dt):
    return torch.tensor(row).expand(rows, len(row)).contiguous().to(DT[dt]).cuda()


def padded(values, width):
    return values + [0.0] * (width - len(values))


@pytest.mark.gpu
@pytest.mark.parametrize("in_dt,out_dt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("rows,J,K", [(1, 8, 8), (5, 3, 5), (40, 16, 1032), (300, 24, 520), (9900, 8, 136)])
def test_low_values_keep_their_bits(s, rows, J, K, in_dt, out_dt):
    """low = (1 + 2^-8 + 2^-20, 1, 2^-8) times up = (1, -1, -1): the result is
    2^-20, which every type holds, and 0 if the first value lost its last bit.
    The same for the gradient of A, with dlow in low's place."""
    from partial_sum_reduction_gb300 import helpers as H
    parts = [1.0, 2.0 ** -8, 2.0 ** -20]
    narrow = torch.zeros(1, 3, max(J, K))
    narrow[0, 0, :3], narrow[0, 1, 0], narrow[0, 2, 1] = 1.0, 1.0, 1.0
    spread = torch.tensor([1.0, -1.0, -1.0]).reshape(1, 3, 1)
    ids = torch.zeros(rows, dtype=torch.int32, device="cuda")
    low = torch.empty(rows, 3, device="cuda")
    plan = s.Plan("{X:1}", "I,J", "J,K", "I,K", rows, J, K, in_dt, out_dt)
    down, up = narrow[:, :, :J].to(DT[in_dt]).cuda().contiguous(), spread.expand(1, 3, K).to(DT[in_dt]).cuda().contiguous()
    C = H.alloc(plan, s.TENSOR_C, fill=float("nan"))
    plan.adapters_forward([repeated(padded(parts, J), rows, in_dt)], ids, down, up, None, None, C, low)
    s.shmm_sync_status()
    assert (low == torch.tensor([1 + 2.0 ** -8 + 2.0 ** -20, 1.0, 2.0 ** -8], device="cuda")).all()
    assert (C[0].float() == 2.0 ** -20).all()
    up, down = narrow[:, :, :K].to(DT[in_dt]).cuda().contiguous(), spread.expand(1, 3, J).to(DT[in_dt]).cuda().contiguous()
    dA = H.alloc(plan, s.TENSOR_A, fill=float("nan"))
    dd, du = torch.empty(1, 3, J, device="cuda"), torch.empty(1, 3, K, device="cuda")
    A = torch.zeros(rows, J, dtype=DT[in_dt], device="cuda")
    plan.adapters_backward([repeated(padded(parts, K), rows, out_dt)], [A], ids, down, up, None, low, None, dA, dd, du,
                           H.adapters_workspace(plan, 1, 3))
    s.shmm_sync_status()
    assert (dA[0].float() == 2.0 ** -20).all()


@pytest.mark.gpu
@pytest.mark.parametrize("R", [4, 40])
def test_long_sums_round(s, R):
    """28671 positive products per value, 8192 rows: too many rows for a
    cluster to share the columns, and a width that no TMA load takes, so a
    thread sums 112 chunks of 32.  With E = 2^-24: a chunk is two matrix
    instructions, each off by at most 2 E of their sum (they cut); each of the
    112 additions rounds by at most E of what it has so far, half of the whole
    on average (56 E); three more join the warps.  So a value is off by at most
    4 + 56 + 3 = 63 E.  The mean over many values keeps only what does not
    average out: the cuts' 4 E, and of the roundings, 3.7 E of deviation per
    value (variance E^2 / 3 times 112 / 3 + 3), eight deviations of the mean of
    1024 values, 1 E.  6 E bounds both.  (Cutting at every one of the 224
    instructions is off by some 80 E, all to one side.)"""
    I, J, K = 8192, 28671, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    A = (torch.rand(I, J, generator=g, device="cuda") + 0.5).bfloat16()
    down = (torch.rand(1, R, J, generator=g, device="cuda") + 0.5).bfloat16()
    up = torch.zeros(1, R, K, device="cuda").bfloat16()
    plan = s.Plan("{X:1}", "I,J", "J,K", "I,K", I, J, K)
    low, C = torch.empty(I, R, device="cuda"), torch.empty(I, K, device="cuda").bfloat16()
    plan.adapters_forward([A], torch.zeros(I, dtype=torch.int32, device="cuda"), down, up, None, None, [C], low)
    s.shmm_sync_status()
    some = torch.arange(0, I, 32, device="cuda")
    want = A[some].double() @ down[0].double().T
    off = (low[some].double() - want) / want
    assert off.abs().max().item() <= 63 * E
    assert abs(off.mean().item()) <= 6 * E


@pytest.mark.gpu
@pytest.mark.parametrize("R", [4, 40])
def test_long_fp32_sums(s, R):
    """8192 positive fp32 products per value, 40000 rows: a thread sums them
    all, in 256 chunks of 32.  The i-th of n additions is off by i / n of E =
    2^-24 of the result at most, evenly spread: a variance of E^2 n / 9 for all.
    256 chunks: (16 / 3 E)^2, and their own sums a 256th of E^2 32 / 9 each,
    nothing beside it.  The root of the mean over 1000 values is within 1.2 of
    that.  (8192 additions in a row: 30 E.)"""
    I, J, K = 40000, 8192, 8
    g = torch.Generator(device="cuda").manual_seed(4)
    A = torch.rand(I, J, generator=g, device="cuda") + 0.5
    down, up = torch.rand(1, R, J, generator=g, device="cuda") + 0.5, torch.zeros(1, R, K, device="cuda")
    plan = s.Plan("{X:1}", "I,J", "J,K", "I,K", I, J, K, "f32", "f32")
    low, C = torch.empty(I, R, device="cuda"), torch.empty(I, K, device="cuda")
    plan.adapters_forward([A], torch.zeros(I, dtype=torch.int32, device="cuda"), down, up, None, None, [C], low)
    s.shmm_sync_status()
    some = torch.arange(0, I, 160, device="cuda")
    want = A[some].double() @ down[0].double().T
    assert ((low[some].double() - want) / want).square().mean().sqrt().item() <= 1.2 * 16 / 3 * E
