"""Layer normalisation for training: shmm_layernorm_forward (saved statistics,
residual), shmm_layernorm_backward, and the gathered pair
shmm_layernorm_all_gather_forward / _backward, against the formulas in 64 bits
and against differences.

Tolerances.  u = 2^-8 is a bf16 half step, 2^-24 an fp32 one.  With n columns,
fp32 sums of n terms in a tree of depth < 32 are off by at most 40 * 2^-24 of
the sum of magnitudes (5 shuffle levels, at most 16 terms per thread and 16
warps in order, and the operations of a term).  So, per element and in fp32:
  y      2^-24 * 64 * (|xh gamma| (1 + max|t| rstd) + |beta|): the deviation
         t - mean is off by the mean's error, 40 * 2^-24 * mean|t|, times
         rstd; and rstd by as much, relative
  dx     2^-24 * 128 * rstd * (|w| + mean|w| + |xh| mean|w xh|)
  dgamma 2^-24 * (rows + 64) * sum|dy xh| (sequential over a CTA's rows)
plus half a step of the stored type of the value itself."""
import ctypes

import numpy as np
import pytest
import torch

from parity_util import lib

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
E = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def s():
    return lib()


def inputs(rows, cols, dtype, seed=0, offset=0.0):
    g = torch.Generator().manual_seed(seed + rows * 131 + cols)
    r = lambda *sh: torch.randn(*sh, generator=g)
    x = (r(rows, cols) * torch.exp(0.3 * r(rows, 1)) + offset).to(DT[dtype])
    return x, 1.0 + 0.2 * r(cols), 0.2 * r(cols), r


def formula(t, gamma, beta, eps):
    """y, mean, rstd in float64, and the bound's scale for y."""
    t = t.double()
    mean = t.mean(1)
    d = t - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(1) + eps)
    xh = d * rstd[:, None]
    y = xh * gamma.double() + beta.double()
    scale = (xh * gamma.double()).abs() * (1 + t.abs().amax(1, keepdim=True) * rstd[:, None]) + beta.double().abs() \
        + gamma.double().abs() * (t.abs().mean(1, keepdim=True) * rstd[:, None])
    return y, mean, rstd, scale


def formula_grad(t, dy, mean, rstd, gamma):
    t, dy = t.double(), dy.double()
    r = rstd.double()[:, None]
    xh = (t - mean.double()[:, None]) * r
    w = dy * gamma.double()
    dx = r * (w - w.mean(1, keepdim=True) - xh * (w * xh).mean(1, keepdim=True))
    scale = r * (w.abs() + w.abs().mean(1, keepdim=True) + xh.abs() * (w * xh).abs().mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0), scale, (dy * xh).abs().sum(0), dy.abs().sum(0)


def within(got, want, bound, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    over = ((got - want).abs() - bound).max().item()
    assert over <= 0, "%s: %.3g over its bound" % (what, over)


def forward(s, x, gamma, beta, residual=None, eps=1e-5):
    dev = x.cuda()
    rows, cols = x.shape
    nan = float("nan")
    y = torch.full_like(dev, nan)
    total = torch.full_like(dev, nan) if residual is not None else None
    mean, rstd = (torch.full((rows,), nan, device="cuda") for _ in range(2))
    s.shmm_layernorm_forward(dev, gamma.cuda(), beta.cuda(), y, mean, rstd,
                             residual=None if residual is None else residual.cuda(), total=total, eps=eps)
    torch.cuda.synchronize()
    return y, mean, rstd, total


SHAPES = [(1, 1), (1, 8), (3, 7), (2, 64), (9, 512), (257, 520), (5, 1001), (33, 1000), (4, 4096), (300, 4096),
          (17, 8192), (3, 8191), (6, 8200), (2, 20001)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", SHAPES + [(1003, 4096), (920, 520), (950, 8192), (2500, 1544)])
def test_forward(s, rows, cols, dtype, residual):
    x, gamma, beta, r = inputs(rows, cols, dtype)
    res = r(rows, cols).to(DT[dtype]) if residual else None
    y, mean, rstd, total = forward(s, x, gamma, beta, res)
    t = x
    if residual:
        t = (x.float() + res.float()).to(DT[dtype])
        assert torch.equal(total.cpu(), t)
    wy, wm, wr, scale = formula(t, gamma, beta, 1e-5)
    amp = t.double().abs().mean(1)
    within(mean, wm, 64 * E * (amp + wm.abs()), "mean")
    within(rstd, wr, 64 * E * wr * (1 + t.double().abs().amax(1) * wr), "rstd")
    within(y, wy, 64 * E * scale + HALF[DT[dtype]] * (wy.abs() + 64 * E * scale), "y")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_in_flight_do_not_meet(s, dtype):
    """Many calls on freshly copied inputs, whose first rows arrive late and
    their followers early: every row is its own, forward and backward."""
    rows, cols = 1003, 4096
    x, gamma, beta, r = inputs(rows, cols, dtype)
    res, dy = (r(rows, cols).to(DT[dtype]) for _ in range(2))
    want = (x.float() + res.float()).to(DT[dtype]).cuda()
    first = None
    for _ in range(150):
        y, mean, rstd, total = forward(s, x, gamma, beta, res)
        assert torch.equal(total, want)
        got = (y, mean, rstd) + backward(s, dy, total, mean, rstd, gamma, res)
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))


@pytest.mark.gpu
def test_forward_equals_the_inference_call_within_a_step(s):
    """shmm_layernorm and shmm_layernorm_forward compute the same function;
    the sums' order may differ, so bf16 results differ by a step at most."""
    x, gamma, beta, _ = inputs(64, 4096, "bf16")
    y, *_ = forward(s, x, gamma, beta)
    z = torch.empty_like(y)
    s.shmm_layernorm(x.cuda(), gamma.cuda(), beta.cuda(), z)
    d = (y.float() - z.float()).abs()
    assert (d <= 2 ** -7 * z.float().abs() + 1e-6).all()


@pytest.mark.gpu
def test_forward_special_rows(s):
    """A constant row has xh = 0 and y = beta; a row with an infinity or a NaN
    is NaN and leaves its neighbours alone; eps = 0 works."""
    x, gamma, beta, _ = inputs(6, 1000, "f32")
    x[1] = 3.0
    x[2, 5] = float("inf")
    x[4, 7] = float("nan")
    y, mean, rstd, _ = forward(s, x, gamma, beta)
    y = y.cpu()
    assert torch.equal(y[1], beta) and mean[1].item() == 3.0
    assert y[2].isnan().all() and y[4].isnan().all()
    keep = [0, 3, 5]
    clean = x[keep]
    y2, *_ = forward(s, clean, gamma, beta)
    assert torch.equal(y[keep], y2.cpu())
    y0, _, r0, _ = forward(s, clean, gamma, beta, eps=0.0)
    wy, _, wr, scale = formula(clean, gamma, beta, 0.0)
    within(y0, wy, 64 * E * scale + E * wy.abs(), "y, eps 0")


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(37, 512), (37, 4096), (37, 1001), (37, 9000), (1301, 4096)])
def test_forward_in_place(s, rows, cols):
    x, gamma, beta, r = inputs(rows, cols, "bf16")
    res = r(rows, cols).to(torch.bfloat16)
    y, mean, rstd, total = forward(s, x, gamma, beta, res)
    xa, ra = x.cuda(), res.cuda()
    m2, r2 = torch.empty_like(mean), torch.empty_like(rstd)
    s.shmm_layernorm_forward(xa, gamma.cuda(), beta.cuda(), xa, m2, r2, residual=ra, total=ra)  # y is x, total residual
    torch.cuda.synchronize()
    assert torch.equal(xa, y) and torch.equal(ra, total) and torch.equal(m2, mean) and torch.equal(r2, rstd)


def backward(s, dy, x, mean, rstd, gamma, res=None, ws=None):
    from partial_sum_reduction_gb300 import helpers as H
    rows, cols = x.shape
    nan = float("nan")
    dx = torch.full((rows, cols), nan, dtype=x.dtype, device="cuda")
    dg, db = (torch.full((cols,), nan, device="cuda") for _ in range(2))
    ws = H.layernorm_workspace(rows, cols) if ws is None else ws
    if ws is not None:
        ws.fill_(0xff)  # NaN in every word: nothing is read before it is written
    s.shmm_layernorm_backward(dy.cuda(), x.cuda(), mean.cuda(), rstd.cuda(), gamma.cuda(), dx, dg, db, ws,
                              residual_grad=None if res is None else res.cuda())
    torch.cuda.synchronize()
    return dx, dg, db


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", SHAPES + [(700, 2048), (1200, 72), (1003, 4096), (920, 520), (950, 8192), (2500, 1544)])
def test_backward(s, rows, cols, dtype, residual):
    x, gamma, beta, r = inputs(rows, cols, dtype)
    dy = r(rows, cols).to(DT[dtype])
    res = r(rows, cols).to(DT[dtype]) if residual else None
    _, wm, wr, _ = formula(x, gamma, beta, 1e-5)
    mean, rstd = wm.float(), wr.float()
    dx, dg, db = backward(s, dy, x, mean, rstd, gamma, res)
    wx, wg, wb, sx, sg, sb = formula_grad(x, dy, mean, rstd, gamma)
    # xh = (t - mean) rstd is off by a few E of (|t| + |mean|) rstd, not of xh
    amp = 1 + ((x.double().abs() + mean.double().abs()[:, None]) * rstd.double()[:, None]).amax()
    if residual:
        wx = wx + res.double()
        sx = sx + res.double().abs() / amp
    within(dx, wx, 128 * E * amp * sx + HALF[DT[dtype]] * (wx.abs() + 128 * E * amp * sx), "dx")
    within(dg, wg, (rows + 64) * E * amp * (sg + sb), "dgamma")
    within(db, wb, (rows + 64) * E * sb, "dbeta")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(37, 512), (37, 4096), (37, 1001), (37, 9000), (1301, 4096), (1301, 8192)])
def test_backward_of_constant_rows(s, rows, cols, dtype):
    """Rows of one value far from zero: xh is exactly 0 (the sum of `cols`
    times 1000 = 125 * 8 is exact below 2^24 * 8, so is its division, so is
    x - mean), and so is dgamma, however large rstd = 316 is."""
    x = torch.full((rows, cols), 1000.0).to(DT[dtype])
    _, gamma, beta, r = inputs(rows, cols, dtype)
    dy = r(rows, cols).to(DT[dtype])
    y, mean, rstd, _ = forward(s, x, gamma, beta)
    assert (mean == 1000.0).all() and torch.equal(y.cpu(), beta.to(DT[dtype]).expand(rows, cols))
    dx, dg, db = backward(s, dy.cuda(), x.cuda(), mean, rstd, gamma.cuda())
    assert (dg == 0).all()
    w, _, wb, scale, _, sb = formula_grad(x, dy, mean.cpu(), rstd.cpu(), gamma)
    within(dx, w, 128 * E * scale + HALF[DT[dtype]] * (w.abs() + 128 * E * scale), "dx")
    within(db, wb, E * (rows + 64) * sb, "dbeta")


@pytest.mark.gpu
def test_backward_without_rows_writes_zeros(s):
    e = torch.empty(0, 96, device="cuda")
    dg, db = (torch.full((96,), 7.0, device="cuda") for _ in range(2))
    st = torch.empty(0, device="cuda")
    s.shmm_layernorm_backward(e, e, st, st, torch.ones(96, device="cuda"), e, dg, db, None)
    torch.cuda.synchronize()
    assert (dg == 0).all() and (db == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(401, 96), (401, 4096), (401, 1001), (401, 9000), (1301, 4096)])
def test_backward_in_place(s, rows, cols):
    """dx over dy, over x and over the residual's gradient gives the same bits."""
    from partial_sum_reduction_gb300 import helpers as H
    x, gamma, beta, r = inputs(rows, cols, "bf16")
    dy, res = r(rows, cols).bfloat16(), r(rows, cols).bfloat16()
    _, wm, wr, _ = formula(x, gamma, beta, 1e-5)
    mean, rstd = wm.float(), wr.float()
    want = backward(s, dy, x, mean, rstd, gamma, res)
    for which in ("dy", "res", "x"):
        b = {"dy": dy.cuda(), "res": res.cuda(), "x": x.cuda()}
        dg, db = torch.empty_like(want[1]), torch.empty_like(want[2])
        s.shmm_layernorm_backward(b["dy"], b["x"], mean.cuda(), rstd.cuda(), gamma.cuda(), b[which], dg, db,
                                  H.layernorm_workspace(rows, cols), residual_grad=b["res"])
        torch.cuda.synchronize()
        assert torch.equal(b[which], want[0]) and torch.equal(dg, want[1]) and torch.equal(db, want[2])


@pytest.mark.gpu
def test_backward_against_differences(s):
    """The gradient of L = sum(y * c) by central differences in 64 bits of
    the formula, at every element of a small case.  The differences' own
    error: h^2/6 of the third derivative, below 1e-6 here with h = 1e-4."""
    rows, cols, eps, h = 3, 24, 1e-5, 1e-4
    x, gamma, beta, r = inputs(rows, cols, "f32")
    c = r(rows, cols)
    loss = lambda t, ga, be: (formula(t, ga, be, eps)[0] * c.double()).sum()
    _, wm, wr, _ = formula(x, gamma, beta, eps)
    dx, dg, db = backward(s, c, x, wm.float(), wr.float(), gamma)
    xd, gd, bd = x.double(), gamma.double(), beta.double()
    for got, var, args in ((dx, xd, 0), (dg, gd, 1), (db, bd, 2)):
        flat = got.double().cpu().flatten()
        for i in range(var.numel()):
            vals = []
            for sgn in (1, -1):
                v = var.clone()
                v.view(-1)[i] += sgn * h
                a = [xd, gd, bd]
                a[args] = v
                vals.append(loss(*a))
            assert abs((vals[0] - vals[1]) / (2 * h) - flat[i]) < 2e-5


@pytest.mark.gpu
def test_backward_repeats_its_bits(s):
    x, gamma, beta, r = inputs(3001, 1032, "bf16")
    dy = r(3001, 1032).bfloat16()
    _, wm, wr, _ = formula(x, gamma, beta, 1e-5)
    a = backward(s, dy, x, wm.float(), wr.float(), gamma)
    for _ in range(3):
        for p, q in zip(a, backward(s, dy, x, wm.float(), wr.float(), gamma)):
            assert torch.equal(p, q)


# ---- the gathered pair -------------------------------------------------------

GATHERS = [([("X", 2)], (("X",), ()), ((), ()), ((), ()), 1), ([("X", 8)], (("X",), ()), ((), ()), ((), ()), 1),
           # gathered over Y within each X block: 4 groups of 2
           ([("X", 4), ("Y", 2)], (("X", "Y"), ()), ((), ()), (("X",), ()), 4),
           # columns sharded over Y, replicas over Z: each normalises its own block
           ([("X", 2), ("Y", 2), ("Z", 2)], (("X",), ()), ((), ("Y",)), ((), ("Y",)), 4)]


@pytest.mark.gpu
@pytest.mark.parametrize("brows,cols,dtype,grad", [(5, 64, "bf16", "f32"), (33, 1001, "bf16", "bf16"),
                                                   (70, 4096, "bf16", "f32"), (9, 2048, "f32", "f32"),
                                                   (1, 8192, "bf16", "bf16"), (3, 8208, "f32", "f32"),
                                                   (479, 1032, "bf16", "f32"), (461, 4096, "bf16", "bf16"),
                                                   (470, 8192, "f32", "f32")])
@pytest.mark.parametrize("which", range(len(GATHERS)))
def test_gathered_pair(s, which, brows, cols, dtype, grad):
    from partial_sum_reduction_gb300 import helpers as H
    mesh, sA, sB, sC, groups = GATHERS[which]
    n = int(np.prod([k for _, k in mesh]))
    G = n // groups
    blocks = n // (4 if which == 3 else 1)  # row blocks of the global result
    kc = 2 if which == 3 else 1
    plan = s.Plan(mesh, sA, sB, sC, brows * blocks, 8, cols * kc, dtype, dtype)
    assert plan.info.gather_C_size == G
    g = torch.Generator().manual_seed(brows + cols + which)
    r = lambda *sh: torch.randn(*sh, generator=g)
    shards = [r(brows, cols).to(DT[dtype]) for _ in range(n)]
    gamma, beta = 1.0 + 0.2 * r(cols), 0.2 * r(cols)
    dev = [t.cuda() for t in shards]
    full = H.alloc(plan, s.TENSOR_C, fill=float("nan"))
    mean, rstd = ([torch.full((brows,), float("nan"), device="cuda") for _ in range(n)] for _ in range(2))
    plan.layernorm_all_gather_forward(dev, gamma.cuda(), beta.cuda(), full, mean, rstd)
    torch.cuda.synchronize()
    # what each member holds: the blocks of the ranks it gathers from, in row order
    where = [plan.rank_box(s.TENSOR_C_REDUCED, q) for q in range(n)]
    mine = [plan.rank_box(s.TENSOR_C, q) for q in range(n)]
    coords = [np.unravel_index(q, [k for _, k in mesh]) for q in range(n)]
    fixed = [i for i, (a, _) in enumerate(mesh) if a not in {0: "X", 1: "X", 2: "Y", 3: "X"}[which]]
    member = [[o for o in range(n) if all(coords[o][i] == coords[q][i] for i in fixed)] for q in range(n)]
    want_y = []
    for q in range(n):
        wy, wm, wr, sc = formula(shards[q], gamma, beta, 1e-5)
        want_y.append((wy, sc))
        within(mean[q], wm, 64 * E * (shards[q].double().abs().mean(1) + wm.abs()), "mean")
        within(rstd[q], wr, 64 * E * wr * (1 + shards[q].double().abs().amax(1) * wr), "rstd")
    for q in range(n):
        assert len(member[q]) == G
        for o in member[q]:
            r0 = where[o][0][0] - mine[q][0][0]
            wy, sc = want_y[o]
            within(full[q][r0:r0 + brows], wy, 64 * E * sc + HALF[DT[dtype]] * (wy.abs() + 64 * E * sc), "y")
    # gradient: members' gradients summed in rank order per owner
    dfull = [(0.1 * r(*mine[q][1])).to(DT[grad]) for q in range(n)]
    dsh = H.alloc(plan, s.TENSOR_C_REDUCED, fill=float("nan"))
    dg, db = (torch.full((cols,), float("nan"), device="cuda") for _ in range(2))
    ws = H.layernorm_workspace(brows * n, cols)
    ws.fill_(0xff)
    plan.layernorm_all_gather_backward([t.cuda() for t in dfull], dev, mean, rstd, gamma.cuda(), dsh, dg, db, ws)
    torch.cuda.synchronize()
    sums = [torch.zeros(cols, dtype=torch.float64) for _ in range(4)]
    amp = 1.0
    for q in range(n):
        mc, rc = mean[q].cpu(), rstd[q].cpu()
        amp = max(amp, 1 + ((shards[q].double().abs() + mc.double().abs()[:, None]) * rc.double()[:, None]).max().item())
    for o in range(n):
        dy, mag = torch.zeros(brows, cols, dtype=torch.float64), torch.zeros(brows, cols, dtype=torch.float64)
        for q in member[o]:
            r0 = where[o][0][0] - mine[q][0][0]
            dy += dfull[q][r0:r0 + brows].double()
            mag += dfull[q][r0:r0 + brows].double().abs()
        wx, wg, wb, _, _, _ = formula_grad(shards[o], dy, mean[o].cpu(), rstd[o].cpu(), gamma)
        _, _, _, sx, sg, sb = formula_grad(shards[o], mag, mean[o].cpu(), rstd[o].cpu(), gamma.abs())
        sx = sx + rstd[o].cpu().double()[:, None] * (mag * gamma.double().abs()).mean(1, keepdim=True) * amp
        within(dsh[o], wx, 128 * E * amp * sx + HALF[DT[dtype]] * (wx.abs() + 128 * E * amp * sx), "dx")
        for a, b in zip(sums, (wg, wb, sg, sb)):
            a += b
    within(dg, sums[0], (brows * n + 64) * E * amp * (sums[2] + sums[3]), "dgamma")
    within(db, sums[1], (brows * n + 64) * E * sums[3], "dbeta")


@pytest.mark.gpu
def test_training_pair_captured_and_replayed(s):
    """Forward and backward captured into one graph on a side stream replay
    with eager bits on new inputs, with a second graph on its own workspace
    between the replays."""
    from partial_sum_reduction_gb300 import helpers as H
    rows, cols = 260, 1024
    gamma, beta = torch.rand(cols, device="cuda") + 0.5, torch.rand(cols, device="cuda")

    def buffers():
        b = {k: torch.randn(rows, cols, device="cuda").bfloat16() for k in ("x", "res", "dy")}
        b.update({k: torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16) for k in ("t", "y", "dx")})
        b.update({k: torch.empty(rows, device="cuda") for k in ("mean", "rstd")})
        b.update({k: torch.empty(cols, device="cuda") for k in ("dg", "db")})
        b["ws"] = H.layernorm_workspace(rows, cols)
        return b

    def step(b):
        s.shmm_layernorm_forward(b["x"], gamma, beta, b["y"], b["mean"], b["rstd"], residual=b["res"], total=b["t"])
        s.shmm_layernorm_backward(b["dy"], b["t"], b["mean"], b["rstd"], gamma, b["dx"], b["dg"], b["db"], b["ws"],
                                  residual_grad=b["dy"])

    sets, graphs = [buffers(), buffers()], []
    for b in sets:
        step(b)
    torch.cuda.synchronize()
    for b in sets:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step(b)
        graphs.append(g)
    for b in sets:
        for k in ("x", "res", "dy"):
            b[k].copy_(torch.randn(rows, cols, device="cuda").bfloat16())
    for g in (graphs[0], graphs[1], graphs[0]):
        g.replay()
    torch.cuda.synchronize()
    for b in sets:
        got = {k: b[k].clone() for k in ("t", "y", "dx", "mean", "rstd", "dg", "db")}
        step(b)
        torch.cuda.synchronize()
        for k, v in got.items():
            assert torch.equal(v, b[k]), k


# ---- refusals (no GPU) ---------------------------------------------------------

def test_refusals(monkeypatch):
    import partial_sum_reduction_gb300 as s
    from partial_sum_reduction_gb300 import build
    build.build()
    L, m = s.lib(), s.shmm
    P = ctypes.c_void_p
    a, odd = P(0x10000), P(0x10008)
    big = 1 << 40
    f = lambda rows=4, cols=64, dt=1, x=a, res=None, g=a, b=a, eps=1e-5, tot=None, y=P(0x20000), mean=a, rstd=a: \
        L.shmm_layernorm_forward(rows, cols, dt, x, res, g, b, eps, tot, y, mean, rstd, None)
    assert f(rows=-1) == m.ERR_SHAPE and f(cols=1 << 31) == m.ERR_SHAPE and f(eps=-1.0) == m.ERR_SHAPE
    assert f(eps=float("nan")) == m.ERR_SHAPE and f(rows=big, cols=1 << 30) == m.ERR_SHAPE
    assert f(dt=5) == m.ERR_DTYPE
    assert f(x=None) == m.ERR_NULL and f(mean=None) == m.ERR_NULL and f(g=None) == m.ERR_NULL
    assert f(x=odd) == m.ERR_ALIGN and f(y=odd) == m.ERR_ALIGN and f(rstd=P(0x10002)) == m.ERR_ALIGN
    assert f(res=a) == m.ERR_NULL and f(res=odd, tot=a) == m.ERR_ALIGN
    assert f(tot=a) == m.ERR_UNSUPPORTED and f(res=a, tot=P(0x20000)) == m.ERR_UNSUPPORTED
    assert f(rows=0) == m.OK and f(cols=0) == m.OK
    w = lambda rows=4, cols=64, dt=1, dy=a, x=a, mean=a, rstd=a, g=a, r=None, dx=a, dg=a, db=a, ws=a, n=big: \
        L.shmm_layernorm_backward(rows, cols, dt, dy, x, mean, rstd, g, r, dx, dg, db, ws, n, None)
    assert w(ws=None) == m.ERR_NULL and w(ws=P(0x10080)) == m.ERR_ALIGN and w(n=4 * 2 * 64 * 4 - 1) == m.ERR_NOMEM
    assert w(dy=None) == m.ERR_NULL and w(dg=None) == m.ERR_NULL and w(dx=odd) == m.ERR_ALIGN
    assert w(r=odd) == m.ERR_ALIGN and w(dt=7) == m.ERR_DTYPE and w(rows=-2) == m.ERR_SHAPE and w(cols=0) == m.OK
    assert s.shmm_layernorm_backward_workspace_size(4, 64) == 4 * 2 * 64 * 4
    big = s.shmm_layernorm_backward_workspace_size(1 << 20, 64)
    assert big == s.shmm_layernorm_backward_workspace_size(1 << 30, 64) <= 1024 * 2 * 64 * 4
    assert L.shmm_layernorm_backward_workspace_size(1, 1, None) == m.ERR_NULL
    with pytest.raises(s.ShmmError):
        s.shmm_layernorm_backward_workspace_size(-1, 4)
    # the gathered pair
    p = s.Plan("{X:2}", "I_X,J", "J,K", "I,K", 8, 8, 64)
    q = s.Plan("{X:2}", "I_X,J", "J,K", "I_X,K", 8, 8, 64)
    cols_plan = s.Plan("{X:2}", "I,J", "J,K_X", "I,K", 8, 8, 64)
    PP = P * 2
    ok, nul, mis = PP(0x10000, 0x20000), PP(0, 0x20000), PP(0x10000, 0x20008)
    F = lambda plan=p, sh=ok, g=a, b=a, eps=1e-5, full=ok, mean=ok, rstd=ok: L.shmm_layernorm_all_gather_forward(
        plan.handle if plan else None, sh, g, b, eps, full, mean, rstd, None)
    assert F(plan=None) == m.ERR_NULL and F(plan=q) == m.ERR_UNSUPPORTED and F(plan=cols_plan) == m.ERR_UNSUPPORTED
    assert F(sh=nul) == m.ERR_NULL and F(full=mis) == m.ERR_ALIGN and F(mean=nul) == m.ERR_NULL
    assert F(rstd=None) == m.ERR_NULL and F(eps=-0.5) == m.ERR_SHAPE and F(g=None) == m.ERR_NULL
    B = lambda plan=p, dt=0, df=ok, sh=ok, mean=ok, rstd=ok, g=a, ds=ok, dg=a, db=a, ws=a, n=big: \
        L.shmm_layernorm_all_gather_backward(plan.handle, dt, df, sh, mean, rstd, g, ds, dg, db, ws, n, None)
    assert B(plan=q) == m.ERR_UNSUPPORTED and B(dt=3) == m.ERR_DTYPE and B(df=nul) == m.ERR_NULL
    assert B(ds=mis) == m.ERR_ALIGN and B(n=10) == m.ERR_NOMEM and B(db=None) == m.ERR_NULL
    pf = s.Plan("{X:2}", "I_X,J", "J,K", "I,K", 8, 8, 64, "f32", "f32")
    assert B(plan=pf, dt=1) == m.ERR_DTYPE
    names = ["shmm_layernorm_forward", "shmm_layernorm_backward", "shmm_layernorm_all_gather_forward",
             "shmm_layernorm_all_gather_backward"]
    monkeypatch.setenv("SHMM_INJECT_FAIL", ",".join(names))
    assert f() == w() == F() == B() == m.ERR_INJECTED
    # the binding refuses what is not a dense CUDA tensor of the right kind
    t = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        s.shmm_layernorm_forward(t, t[0], t[0], t, t[:, 0], t[:, 0])
    with pytest.raises(ValueError, match="expected torch.float32 or"):
        s.shmm_layernorm_backward(t.half(), t.half(), t, t, t, t, t, t, None)
    with pytest.raises(ValueError, match="2 ranks"):
        p.layernorm_all_gather_forward([t], t, t, [t], [t], [t])
