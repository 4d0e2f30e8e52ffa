"""Layer normalisation's gradient at the ends of the range: rows so small that
rstd^2 is no fp32 value, though rstd and the result are."""
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
