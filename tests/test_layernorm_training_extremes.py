"""Layer normalisation's gradient where fp32 is short: rows so small that
rstd^2 is no fp32 value, though rstd and the result are, and the long sums of
the gains' gradient."""
import pytest
import torch

from parity_util import lib
from test_layernorm_training import DT, E, HALF, backward, formula, formula_grad, inputs, within


@pytest.fixture(scope="module")
def s():
    return lib()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(37, 512), (37, 4096), (37, 1001), (37, 9000), (1301, 4096), (1301, 8192)])
def test_backward_of_tiny_rows(s, rows, cols, dtype):
    """x of 2^-70, eps = 0: rstd is 2^70, dx some 2^70 dy, which every type
    holds.  The bounds are test_layernorm_training's: they are relative, and no
    step of the formula leaves the normal range (xh and w are of order 1)."""
    x, gamma, beta, r = inputs(rows, cols, "f32")
    x = (x * 2.0 ** -70).to(DT[dtype])
    dy = r(rows, cols).to(DT[dtype])
    _, wm, wr, _ = formula(x, gamma, beta, 0.0)
    mean, rstd = wm.float(), wr.float()
    assert (rstd > 2.0 ** 66).all() and torch.isfinite(rstd).all()
    dx, dg, db = backward(s, dy, x, mean, rstd, gamma)
    wx, wg, wb, sx, sg, sb = formula_grad(x, dy, mean, rstd, gamma)
    amp = 1 + ((x.double().abs() + mean.double().abs()[:, None]) * rstd.double()[:, None]).amax()
    within(dx, wx, 128 * E * amp * sx + HALF[DT[dtype]] * (wx.abs() + 128 * E * amp * sx), "dx")
    within(dg, wg, (rows + 64) * E * amp * (sg + sb), "dgamma")
    within(db, wb, (rows + 64) * E * sb, "dbeta")


@pytest.mark.gpu
def test_sums_over_rows_are_few_additions_deep(s):
    """dbeta of 600 rows of positive values, a row per partial sum.  An addition
    of two positive values is off by at most E = 2^-24 of its result, evenly
    spread: a variance of E^2 / 3.  Added in pairs, the errors of one level up
    count half as much together as those of the level below it, so the variance
    is at most E^2 / 3 (1 + 1/2 + 1/4 + ...) = 2/3 E^2 of the value; the root of
    the mean over 2314 values is within 1.1 of that (five of its own deviations,
    1/68 each, are 0.07).  (32 additions in a row: the i-th is off by i / 32 of
    that, 32 / 9 E^2.)"""
    rows, cols = 600, 1157
    g = torch.Generator().manual_seed(1)
    x, dy = torch.randn(rows, cols, generator=g), torch.rand(rows, cols, generator=g) + 0.5
    _, wm, wr, _ = formula(x, torch.ones(cols), torch.zeros(cols), 1e-5)
    off = []
    for _ in range(2):
        _, _, db = backward(s, dy, x, wm.float(), wr.float(), torch.ones(cols))
        want = dy.double().sum(0)
        off.append((db.double().cpu() - want) / want)
        dy = torch.rand(rows, cols, generator=g) + 0.5
    assert torch.cat(off).square().mean().sqrt().item() <= 1.1 * (2 / 3) ** 0.5 * E
