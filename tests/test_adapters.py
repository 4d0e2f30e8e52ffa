"""Low-rank adapters beside a sharded projection (Plan.adapters_forward,
Plan.adapters_backward) against the formulas in 64 bits, and the block they
are used in: normalise, gather, project, adapt, and the gradient back.

Tolerances, with E = 2^-24 an fp32 half step.  A tensor-core sum of n products
is at most n / 16 accumulations, each off by at most 2 E (truncation) of the
running magnitude, and the joining of warps and CTAs adds fewer than 64; an
fp32 chain on CUDA cores is at most n / 32 chunks of 32 additions of E each.
So any sum of n products is off by at most (n + 64) 2 E of the sum of their
magnitudes, and by (n / 16 + 64) 2 E on tensor cores.  The split of an fp32
operand into two bf16 parts loses 2^-16 of it, into three 2^-23.  On top come
half a step of the stored type and what an inexact low or dlow carries on."""
import ctypes

import numpy as np
import pytest
import torch

from parity_util import lib

E = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: E}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def s():
    return lib()


LAYOUTS = {
    "whole": ("{X:1}", "I,J", "J,K", "I,K"),
    "rows": ("{X:4}", "I_X,J", "J,K", "I_X,K"),
    "contracted": ("{X:2,Y:2}", "I_X,J_Y", "J_Y,K", "I_X,K"),       # C replicated over Y
    "scattered": ("{Y:2}", "I,J_Y", "J_Y,K", "I_Y,K"),              # row-owned C
    "columns": ("{X:4}", "I,J", "J,K_X", "I,K_X"),                  # A replicated, column-sharded C
    "gathered": ("{X:2}", "I_X,J", "J,K_X", "I_X,K"),               # case 4: B gathered
    "grid": ("{X:2,Y:2}", "I_X,J", "J,K_Y", "I_X,K_Y"),
}


def sum_tol(n, tensor_core):
    return ((n / 16 if tensor_core else n) + 64) * 2 * E


class Case:
    """A plan with inputs on the host (input types) and on the device."""

    def __init__(self, s, layout, I, J, K, R, n, in_dt="bf16", out_dt="bf16", seed=0, ids=None, scale=True):
        from partial_sum_reduction_gb300 import helpers as H
        self.s, self.H = s, H
        mesh, sa, sb, sc = LAYOUTS[layout]
        self.plan = s.Plan(mesh, sa, sb, sc, I, J, K, in_dt, out_dt)
        self.I, self.J, self.K, self.R, self.n = I, J, K, R, n
        self.ti, self.to = DT[in_dt], DT[out_dt]
        g = torch.Generator().manual_seed(seed + I + 3 * J + 7 * K + 11 * R)
        r = lambda *sh: torch.randn(*sh, generator=g)
        self.A, self.down, self.up = r(I, J).to(self.ti), (r(n, R, J) / J ** 0.5).to(self.ti), r(n, R, K).to(self.ti)
        self.scale = torch.rand(n, generator=g) + 0.5 if scale else None
        self.base, self.dC, self.dbase = r(I, K).to(self.to), r(I, K).to(self.to), r(I, J).to(self.ti)
        self.ids = torch.randint(-1, n, (I,), generator=g, dtype=torch.int32) if ids is None else ids.to(torch.int32)
        self.dev = {k: getattr(self, k).cuda() for k in ("down", "up", "ids")}
        self.dev["scale"] = None if self.scale is None else self.scale.cuda()
        self.A_r = H.shard(self.plan, s.TENSOR_A, self.A)

    def cut(self, tensor, full):
        return self.H.shard(self.plan, tensor, full)

    def forward(self, base="other"):
        p, s = self.plan, self.s
        C = self.H.alloc(p, s.TENSOR_C, fill=float("nan"))
        b = None
        if base == "other":
            b = self.cut(s.TENSOR_C, self.base)
        elif base == "same":
            b = C = self.cut(s.TENSOR_C, self.base)
        low = torch.full((self.I, self.R), float("nan"), device="cuda")
        p.adapters_forward(self.A_r, self.dev["ids"], self.dev["down"], self.dev["up"], self.dev["scale"], b, C, low)
        s.shmm_sync_status()
        return C, low

    def backward(self, low, base="other"):
        p, s, H = self.plan, self.s, self.H
        dA = H.alloc(p, s.TENSOR_A, fill=float("nan"))
        b = None
        if base == "other":
            b = self.cut(s.TENSOR_A, self.dbase)
        elif base == "same":
            b = dA = self.cut(s.TENSOR_A, self.dbase)
        dd, du = (torch.full((self.n, self.R, w), float("nan"), device="cuda") for w in (self.J, self.K))
        ws = H.adapters_workspace(p, self.n, self.R)
        if ws is not None:
            ws.fill_(0xff)
        p.adapters_backward(self.cut(s.TENSOR_C, self.dC), self.A_r, self.dev["ids"], self.dev["down"],
                            self.dev["up"], self.dev["scale"], low, b, dA, dd, du, ws)
        s.shmm_sync_status()
        return dA, dd, du

    # ---- the formulas in 64 bits, with the magnitudes their bounds need
    def rows_of(self):
        return [(a, (self.ids == a).nonzero().flatten()) for a in range(self.n)]

    def sc(self, a):
        return 1.0 if self.scale is None else self.scale[a].double()

    def check_forward(self, C, low, base=True):
        tc = self.ti == torch.bfloat16
        want = torch.zeros(self.I, self.R, dtype=torch.float64)
        mag = torch.zeros_like(want)
        c = self.base.double() if base else torch.zeros(self.I, self.K, dtype=torch.float64)
        cm, err = c.abs() * E, torch.zeros_like(c)
        split = 2.0 ** -16 if self.to == torch.bfloat16 else 2.0 ** -23
        for a, idx in self.rows_of():
            x, d, u = self.A[idx].double(), self.down[a].double(), self.up[a].double()
            want[idx], mag[idx] = x @ d.T, x.abs() @ d.abs().T
            e_low = sum_tol(self.J, tc) * mag[idx]
            add = self.sc(a) * (want[idx] @ u)
            m = self.sc(a) * ((want[idx].abs() + e_low) @ u.abs())
            c[idx] += add
            err[idx] = self.sc(a) * (e_low @ u.abs()) + m * ((split if tc else 0) + sum_tol(self.R, False)) + m * E
        close(low, want, sum_tol(self.J, tc) * mag, "low")
        err = err + cm
        none = ((self.ids < 0) | (self.ids >= self.n)).nonzero().flatten()
        assert (low.cpu()[none] == 0).all()
        for r, t in enumerate(C):
            (o0, o1), (e0, e1) = self.plan.rank_box(self.s.TENSOR_C, r)
            w, b = c[o0:o0 + e0, o1:o1 + e1], err[o0:o0 + e0, o1:o1 + e1]
            close(t, w, b + HALF[self.to] * (w.abs() + b), "C[%d]" % r)
            keep = none[(none >= o0) & (none < o0 + e0)]
            src = self.base if base else torch.zeros(self.I, self.K, dtype=self.to)
            assert torch.equal(t.cpu()[keep - o0], src[keep, o1:o1 + e1])

    def check_backward(self, low, dA, dd, du, base=True):
        tc = self.ti == torch.bfloat16
        mixed = self.to == torch.bfloat16 and tc
        low = low.double().cpu()
        want = self.dbase.double() if base else torch.zeros(self.I, self.J, dtype=torch.float64)
        err = want.abs() * E
        wd, wu = torch.zeros(self.n, self.R, self.J, dtype=torch.float64), torch.zeros(self.n, self.R, self.K,
                                                                                      dtype=torch.float64)
        ed, eu = torch.zeros_like(wd), torch.zeros_like(wu)
        split = 2.0 ** -16 if self.ti == torch.bfloat16 else 0.0
        for a, idx in self.rows_of():
            g, x, d, u = self.dC[idx].double(), self.A[idx].double(), self.down[a].double(), self.up[a].double()
            ds, m = self.sc(a) * (g @ u.T), self.sc(a) * (g.abs() @ u.abs().T)
            e_ds = (sum_tol(self.K, mixed) + E) * m
            want[idx] += ds @ d
            mm = (ds.abs() + e_ds) @ d.abs()
            err[idx] += e_ds @ d.abs() + mm * (split + sum_tol(self.R, False))
            n = len(idx)
            wd[a], wu[a] = ds.T @ x, self.sc(a) * (low[idx].T @ g)
            ed[a] = (ds.abs() + e_ds).T @ x.abs() * (sum_tol(n, False) + 2.0 ** -23) + e_ds.T @ x.abs()
            eu[a] = self.sc(a) * (low[idx].abs().T @ g.abs()) * (sum_tol(n, False) + 2.0 ** -22)
        close(dd, wd, ed + E * wd.abs(), "ddown")
        close(du, wu, eu + E * wu.abs(), "dup")
        none = ((self.ids < 0) | (self.ids >= self.n)).nonzero().flatten()
        for r, t in enumerate(dA):
            (o0, o1), (e0, e1) = self.plan.rank_box(self.s.TENSOR_A, r)
            w, b = want[o0:o0 + e0, o1:o1 + e1], err[o0:o0 + e0, o1:o1 + e1]
            close(t, w, b + HALF[self.ti] * (w.abs() + b), "dA[%d]" % r)
            keep = none[(none >= o0) & (none < o0 + e0)]
            src = self.dbase if base else torch.zeros(self.I, self.J, dtype=self.ti)
            assert torch.equal(t.cpu()[keep - o0], src[keep, o1:o1 + e1])

    def check(self, base="other"):
        C, low = self.forward(base)
        self.check_forward(C, low, base is not None)
        dA, dd, du = self.backward(low, base)
        self.check_backward(low, dA, dd, du, base is not None)


def close(got, want, bound, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    if got.numel():
        over = ((got - want).abs() - bound).max().item()
        assert over <= 0, "%s: %.3g over its bound" % (what, over)


# ---- CPU: refusals -----------------------------------------------------------

def test_refusals(monkeypatch):
    import partial_sum_reduction_gb300 as s
    from partial_sum_reduction_gb300 import build
    build.build()
    L, m, P = s.lib(), s.shmm, ctypes.c_void_p
    p = s.Plan("{X:2}", "I_X,J", "J,K", "I_X,K", 8, 16, 24)
    gelu = s.Plan("{X:2}", "I_X,J", "J,K", "I_X,K", 8, 16, 24, flags=s.FLAG_GELU)
    PP = P * 2
    ok, nul, mis = PP(0x10000, 0x20000), PP(0x10000, 0), PP(0x10008, 0x20000)
    a, odd4, odd16 = P(0x30000), P(0x30002), P(0x30008)
    F = lambda plan=p, n=3, R=8, A=ok, ids=a, d=a, u=a, sc=a, b=ok, C=ok, low=a: L.shmm_adapters_forward(
        plan.handle if plan else None, n, R, A, ids, d, u, sc, b, C, low, None)
    B = lambda plan=p, n=3, R=8, dC=ok, A=ok, ids=a, d=a, u=a, sc=a, low=a, b=ok, dA=ok, dd=a, du=a, ws=P(0x40000), \
        nb=1 << 40: L.shmm_adapters_backward(plan.handle if plan else None, n, R, dC, A, ids, d, u, sc, low, b, dA, dd,
                                             du, ws, nb, None)
    for f in (F, B):
        assert f(plan=None) == m.ERR_NULL and f(plan=gelu) == m.ERR_UNSUPPORTED
        assert f(n=0) == m.ERR_SHAPE and f(n=65536) == m.ERR_SHAPE and f(R=0) == m.ERR_SHAPE
        assert f(R=65) == m.ERR_UNSUPPORTED
        assert f(ids=None) == m.ERR_NULL and f(ids=odd4) == m.ERR_ALIGN
        assert f(d=None) == m.ERR_NULL and f(u=odd16) == m.ERR_ALIGN and f(sc=odd4) == m.ERR_ALIGN
        assert f(A=None) == m.ERR_NULL and f(A=nul) == m.ERR_NULL and f(A=mis) == m.ERR_ALIGN
        assert f(b=nul) == m.ERR_NULL and f(b=mis) == m.ERR_ALIGN and f(low=None) == m.ERR_NULL
    assert F(C=nul) == m.ERR_NULL and F(C=mis) == m.ERR_ALIGN
    assert B(dC=nul) == m.ERR_NULL and B(dA=mis) == m.ERR_ALIGN and B(dd=None) == m.ERR_NULL
    assert B(du=odd4) == m.ERR_ALIGN and B(ws=None) == m.ERR_NULL and B(ws=P(0x40010)) == m.ERR_ALIGN
    need = p.adapters_workspace_size(3, 8)
    assert need >= 8 * 8 * 4 and need % 256 == 0 and B(nb=need - 1) == m.ERR_NOMEM
    with pytest.raises(s.ShmmError) as e:
        p.adapters_workspace_size(3, 65)
    assert e.value.status == m.ERR_UNSUPPORTED
    for n, R in ((0, 8), (3, 0), (-1, 1)):
        with pytest.raises(s.ShmmError):
            p.adapters_workspace_size(n, R)
    assert L.shmm_adapters_workspace_size(None, 1, 8, ctypes.byref(ctypes.c_size_t())) == m.ERR_NULL
    monkeypatch.setenv("SHMM_INJECT_FAIL", "shmm_adapters_forward,shmm_adapters_backward")
    assert F() == B() == m.ERR_INJECTED
    t = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="CUDA"):
        p.adapters_forward([t, t], t, t[None], t[None], None, None, [t, t], t)
    with pytest.raises(ValueError, match="down"):
        p.adapters_forward([t, t], t, t, t, None, None, [t, t], t)


# ---- GPU -----------------------------------------------------------------------


def test_refusal_of_a_gradient_over_its_inputs():
    import partial_sum_reduction_gb300 as s
    from partial_sum_reduction_gb300 import build
    build.build()
    L, m, P = s.lib(), s.shmm, ctypes.c_void_p
    p = s.Plan("{X:2}", "I_X,J", "J,K", "I_X,K", 8, 16, 16)
    PP, a = P * 2, P(0x30000)
    for A, dC, dA in (((1, 2), (3, 4), (5, 2)), ((1, 2), (3, 4), (3, 5)), ((1, 2), (3, 4), (1, 2))):
        A, dC, dA = (PP(*(0x10000 * v for v in t)) for t in (A, dC, dA))
        assert L.shmm_adapters_backward(p.handle, 3, 8, dC, A, a, a, a, None, a, None, dA, a, a, P(0x40000), 1 << 40,
                                        None) == m.ERR_UNSUPPORTED


def test_refusals_of_sizes():
    import partial_sum_reduction_gb300 as s
    from partial_sum_reduction_gb300 import build
    build.build()
    L, m, P = s.lib(), s.shmm, ctypes.c_void_p
    one, a, n = (P * 1)(0x10000), P(0x30000), ctypes.c_size_t()
    for I, J, K, ok in ((1 << 31, 8, 8, False), (8, 1 << 23, 8, False), (8, 8, 1 << 23, False),
                        ((1 << 31) - 1, 8, 8, True), (8, (1 << 23) - 8, (1 << 23) - 8, True)):
        p = s.Plan("{X:1}", "I,J", "J,K", "I,K", I, J, K)
        st = L.shmm_adapters_workspace_size(p.handle, 2, 8, ctypes.byref(n))
        assert st == (m.OK if ok else m.ERR_SHAPE)
        if ok:
            assert n.value >= I * 8 * 4
            continue
        assert L.shmm_adapters_forward(p.handle, 2, 8, one, a, a, a, None, None, one, a, None) == m.ERR_SHAPE
        assert L.shmm_adapters_backward(p.handle, 2, 8, one, one, a, a, a, None, a, None, one, a, a, a, 1 << 40,
                                        None) == m.ERR_SHAPE


@pytest.mark.gpu
@pytest.mark.parametrize("layout", list(LAYOUTS))
@pytest.mark.parametrize("in_dt,out_dt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
def test_layouts_and_types(s, layout, in_dt, out_dt):
    Case(s, layout, 72, 160, 192, 16, 5, in_dt, out_dt).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("I,J,K,R,n", [(1, 8, 8, 1, 1), (1, 4096, 1000, 16, 3), (3, 1, 1, 2, 2), (17, 7, 13, 5, 4),
                                       (64, 520, 72, 64, 70), (33, 1001, 515, 33, 2), (200, 64, 1032, 8, 1),
                                       (5, 2056, 4104, 32, 9), (130, 96, 96, 12, 300)])
def test_sizes(s, I, J, K, R, n, dt):
    Case(s, "whole", I, J, K, R, n, dt, dt).check()


@pytest.mark.gpu
@pytest.mark.parametrize("layout,J,K", [("contracted", 1000, 136), ("contracted", 18, 40), ("columns", 40, 36),
                                        ("grid", 24, 1036)])
def test_shards_that_are_no_whole_vectors(s, layout, J, K):
    """J and K are multiples of 8 or 4 while a shard's width is not: rows of
    a shard start off 16-byte boundaries."""
    Case(s, layout, 44, J, K, 16, 3).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["none", "one", "runs", "every", "outside"])
def test_row_adapters(s, kind, dt):
    I, n = 150, 7
    ids = {"none": torch.full((I,), -1), "one": torch.full((I,), 3),
           "runs": torch.arange(I) // 23 % (n + 1) - 1, "every": torch.arange(I) % n,
           "outside": torch.tensor([-2 ** 31, 2 ** 31 - 1, n, -1, 2] * 30)}[kind]
    Case(s, "rows", 4 * 37 if kind == "runs" else 152, 264, 136, 16, n, dt, dt,
         ids=(ids[:148] if kind == "runs" else torch.cat([ids, torch.tensor([-1, -1])]))).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("base", [None, "same"])
def test_without_base_and_in_place(s, base, dt):
    c = Case(s, "contracted", 70, 176, 120, 16, 4, dt, dt)
    c.check(base)
    c = Case(s, "whole", 70, 177, 121, 9, 4, dt, dt, scale=False)
    c.check(base)


@pytest.mark.gpu
@pytest.mark.parametrize("I,R", [(9800, 16), (9730, 64), (12000, 8), (9900, 32)])
def test_many_rows(s, I, R):
    """Enough rows for the tall row tiles, in runs as requests leave them."""
    ids = torch.arange(I) // 613 % 6 - 1
    Case(s, "whole", I, 192, 136, R, 5, ids=ids).check()


@pytest.mark.gpu
@pytest.mark.parametrize("layout,I,J,K,R,n,kind", [
    ("whole", 2048, 512, 512, 16, 3, "runs"), ("whole", 2500, 520, 1000, 5, 40, "random"),
    ("contracted", 2600, 1200, 640, 33, 4, "runs"), ("columns", 2100, 576, 4096, 64, 9, "random"),
    ("rows", 4 * 700, 640, 520, 32, 6, "runs"), ("grid", 2 * 1100, 1160, 1040, 64, 2, "random"),
    ("whole", 4300, 2056, 2104, 8, 300, "random"), ("scattered", 2304, 1024, 768, 16, 1, "random")])
def test_tall_batches(s, layout, I, J, K, R, n, kind):
    """Batches of 2048 rows and more: row tiles of 128 with one adapter and
    with dozens (several passes over a tile), shards whose rows and columns
    are no whole tiles."""
    g = torch.Generator().manual_seed(I)
    ids = torch.arange(I) // 211 % (n + 1) - 1 if kind == "runs" else torch.randint(-1, n, (I,), generator=g)
    Case(s, layout, I, J, K, R, n, ids=ids).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("I,R,n,kind", [(33000, 8, 3, "any"), (40001, 20, 2, "any"), (5000, 16, 400, "one"),
                                        (17000, 40, 305, "one")])
def test_long_and_lopsided_batches(s, I, R, n, kind, dt):
    """More rows than one pass over the row adapters marks, and one adapter
    with nearly all rows among many without any."""
    ids = None
    if kind == "one":
        ids = torch.full((I,), 7)
        ids[::611] = n - 1
        ids[5::977] = -1
    c = Case(s, "whole", I, 72, 40, R, n, dt, dt, ids=ids)
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("layout,I,J,K,R,n,few", [("columns", 6540, 160, 272, 32, 17, 0), ("whole", 9000, 264, 520, 16, 3, 200),
                                                  ("rows", 4100, 136, 72, 64, 9, 1300), ("whole", 2600, 40, 24, 5, 2, 65)])
def test_an_adapter_with_most_rows(s, layout, I, J, K, R, n, few, dt):
    """One adapter's rows shared by many CTAs; `few` rows among the others."""
    g = torch.Generator().manual_seed(I)
    ids = torch.full((I,), n - 1)
    at = torch.randperm(I, generator=g)[:few]
    ids[at] = torch.randint(0, n - 1, (few,), generator=g)
    Case(s, layout, I, J, K, R, n, dt, dt, ids=ids).check()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_an_adapter_without_rows_has_zero_gradients_whatever_its_scale(s, dt):
    c = Case(s, "whole", 70, 136, 72, 12, 4, dt, dt, ids=torch.arange(70) % 2)
    c.scale[2], c.scale[3] = float("nan"), float("inf")
    c.dev["scale"] = c.scale.cuda()
    C, low = c.forward()
    dA, dd, du = c.backward(low)
    assert all(torch.isfinite(t.float()).all() for t in C + dA + [low, dd, du])
    assert (dd[2:] == 0).all() and (du[2:] == 0).all()
    assert (dd[:2] != 0).any() and (du[:2] != 0).any()


@pytest.mark.gpu
def test_infinities_and_nan_stay_in_their_rows_of_a_tall_batch(s):
    I, n = 2304, 5
    ids = torch.arange(I, dtype=torch.int32) % (n + 1) - 1
    c = Case(s, "whole", I, 512, 520, 16, n, ids=ids)
    C0, low0 = c.forward()
    dA0, dd0, du0 = c.backward(low0)
    c.down[2, 3, 5], c.up[2, 1, 7] = float("inf"), float("nan")
    c.A[7], c.dC[7], c.A[13] = float("nan"), float("nan"), float("inf")  # adapter 0
    c.A[6], c.dC[6] = float("nan"), float("inf")                         # none
    assert ids[7] == 0 and ids[13] == 0 and ids[6] == -1
    for k in ("down", "up"):
        c.dev[k] = getattr(c, k).cuda()
    c.A_r = c.H.shard(c.plan, s.TENSOR_A, c.A)
    C1, low1 = c.forward()
    dA1, dd1, du1 = c.backward(low1)
    clean = [i for i in range(I) if ids[i] != 2 and i not in (6, 7, 13)]
    assert torch.equal(C0[0][clean], C1[0][clean]) and torch.equal(low0[clean], low1[clean])
    assert torch.equal(dA0[0][clean], dA1[0][clean])
    for a in (1, 3, 4):
        assert torch.equal(dd0[a], dd1[a]) and torch.equal(du0[a], du1[a])
    assert torch.equal(C1[0][6].cpu(), c.base[6]) and (low1[6] == 0).all()


@pytest.mark.gpu
def test_rows_past_2_to_the_32_bytes(s):
    """Offsets past 32 bits: the last rows of operands of more than 4 GiB."""
    I, J, K, R = 1 << 17, 16640, 16, 4
    plan = s.Plan("{X:1}", "I,J", "J,K", "I,K", I, J, K)
    A = torch.zeros(I, J, dtype=torch.bfloat16, device="cuda")
    A[-3:] = torch.randn(3, J, device="cuda").bfloat16()
    down, up = torch.randn(2, R, J, device="cuda").bfloat16(), torch.randn(2, R, K, device="cuda").bfloat16()
    ids = torch.full((I,), -1, dtype=torch.int32, device="cuda")
    ids[-3:] = torch.tensor([1, -1, 0], dtype=torch.int32)
    C, low = torch.empty(I, K, dtype=torch.bfloat16, device="cuda"), torch.empty(I, R, device="cuda")
    plan.adapters_forward([A], ids, down, up, None, None, [C], low)
    dA = torch.empty_like(A)
    dd, du = torch.empty(2, R, J, device="cuda"), torch.empty(2, R, K, device="cuda")
    plan.adapters_backward([C], [A], ids, down, up, None, low, None, [dA], dd, du,
                           __import__("partial_sum_reduction_gb300").helpers.adapters_workspace(plan, 2, R))
    s.shmm_sync_status()
    x, d, u = A[-3:].double(), down.double(), up.double()
    for row, a in ((0, 1), (2, 0)):
        want = d[a] @ x[row]
        tol = sum_tol(J, True) * (d[a].abs() @ x[row].abs())
        assert ((low[I - 3 + row].double() - want).abs() <= tol).all()
        g = C[I - 3 + row].double()
        ds = u[a] @ g
        m = (u[a].abs() @ g.abs()) @ d[a].abs()
        assert ((dA[I - 3 + row].double() - ds @ d[a]).abs() <= 2 ** -8 * (ds @ d[a]).abs() + 2 ** -14 * m).all()
        assert ((dd[a].double() - ds[:, None] * x[row]).abs() <= 2 ** -14 * (u[a].abs() @ g.abs())[:, None]
                * x[row].abs()).all()
    assert (low[:-3] == 0).all() and (dA[-2] == 0).all() and (dA[: I - 3: 4097] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_infinities_and_nan_stay_in_their_rows(s, dt):
    """An adapter of infinities, a row of NaN, and rows without an adapter
    that hold both: every other row's and adapter's results are unchanged."""
    I, n = 90, 4
    ids = torch.arange(I, dtype=torch.int32) % (n + 1) - 1
    c = Case(s, "whole", I, 200, 104, 16, n, dt, dt, ids=ids)
    C0, low0 = c.forward()
    dA0, dd0, du0 = c.backward(low0)
    c.down[2, 3, 5], c.up[2, 1, 7] = float("inf"), float("nan")
    c.A[11] = float("nan")            # adapter 0
    c.A[10], c.base[10], c.dC[10] = float("inf"), float("nan"), float("nan")  # no adapter
    c.dC[11] = float("-inf")
    assert ids[11] == 0 and ids[10] == -1
    for k in ("down", "up"):
        c.dev[k] = getattr(c, k).cuda()
    c.A_r = c.H.shard(c.plan, s.TENSOR_A, c.A)
    C1, low1 = c.forward()
    dA1, dd1, du1 = c.backward(low1)
    clean = [i for i in range(I) if ids[i] != 2 and i not in (10, 11)]
    assert torch.equal(C0[0][clean], C1[0][clean]) and torch.equal(low0[clean], low1[clean])
    assert torch.equal(dA0[0][clean], dA1[0][clean])
    for a in (1, 3):
        assert torch.equal(dd0[a], dd1[a]) and torch.equal(du0[a], du1[a])
    assert torch.equal(C1[0][10].cpu().isnan(), c.base[10].isnan()) and (low1[10] == 0).all()
    assert torch.equal(dA1[0][10].cpu(), c.dbase[10])
    assert low1[11].isnan().all() and C1[0][11].isnan().all()


@pytest.mark.gpu
def test_no_rows(s):
    """An empty batch: nothing to write forward, zero gradients backward."""
    for dt in ("bf16", "f32"):
        plan = s.Plan("{X:1}", "I,J", "J,K", "I,K", 0, 40, 200, dt, dt)
        e = lambda *sh: torch.empty(*sh, device="cuda", dtype=DT[dt])
        low = torch.empty(0, 4, device="cuda")
        ids = torch.empty(0, dtype=torch.int32, device="cuda")
        d, u = e(3, 4, 40), e(3, 4, 200)
        plan.adapters_forward([e(0, 40)], ids, d, u, None, None, [e(0, 200)], low)
        dd, du = torch.ones(3, 4, 40, device="cuda"), torch.ones(3, 4, 200, device="cuda")
        plan.adapters_backward([e(0, 200)], [e(0, 40)], ids, d, u, None, low, None, [e(0, 40)], dd, du, None)
        s.shmm_sync_status()
        assert (dd == 0).all() and (du == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [64900, 65535])
def test_as_many_adapters_as_there_may_be(s, n, dt):
    """The launches' second grid dimension is one adapter each; few of them
    have rows, one has most."""
    ids = torch.full((900,), n - 1)
    ids[::3] = torch.arange(300) * 211
    c = Case(s, "whole", 900, 24, 16, 2, n, dt, dt, ids=ids)
    used = torch.unique(c.ids).tolist()
    c.rows_of = lambda: [(a, (c.ids == a).nonzero().flatten()) for a in used]
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("I,J,K,R,n,dt", [(130, 96, 96, 12, 300, "f32"), (97, 40, 36, 3, 2, "f32"), (191, 24, 8, 64, 7, "f32"),
                                          (257, 136, 72, 16, 2, "bf16"), (900, 264, 136, 32, 5, "bf16"),
                                          (2600, 72, 520, 64, 3, "bf16"), (2, 8, 8, 1, 9, "bf16")])
def test_nothing_outside_its_buffers(s, I, J, K, R, n, dt):
    """Every buffer, the workspace to the byte, lies between guard bytes."""
    c = Case(s, "whole", I, J, K, R, n, dt, dt, ids=(torch.arange(I) % 29 == 3).int() * (n - 1))
    pool = torch.full((64 << 20,), 0x5a, dtype=torch.uint8, device="cuda")
    guard = torch.ones(pool.numel(), dtype=torch.bool, device="cuda")
    end = [4096]

    def take(nbytes):
        lo, end[0] = end[0], end[0] + (nbytes + 8191) // 256 * 256
        guard[lo:lo + nbytes] = False
        return pool[lo:lo + nbytes]

    def put(t, fill=None):
        d = take(t.numel() * t.element_size()).view(t.dtype).view(t.shape)
        return d.copy_(t) if fill is None else d.fill_(fill)

    nan = float("nan")
    A, dC, base, dbase, down, up, scale, ids = (put(t) for t in (c.A, c.dC, c.base, c.dbase, c.down, c.up, c.scale, c.ids))
    C, dA, low = put(c.base, nan), put(c.dbase, nan), put(torch.empty(I, R), nan)
    dd, du = put(torch.empty(n, R, J), nan), put(torch.empty(n, R, K), nan)
    ws = take(c.plan.adapters_workspace_size(n, R))
    assert end[0] < pool.numel()
    c.plan.adapters_forward([A], ids, down, up, scale, [base], [C], low)
    c.plan.adapters_backward([dC], [A], ids, down, up, scale, low, [dbase], [dA], dd, du, ws)
    s.shmm_sync_status()
    assert (pool[guard] == 0x5a).all()
    c.check_forward([C], low)
    c.check_backward(low, [dA], dd, du)


@pytest.mark.gpu
def test_order_of_requests_does_not_matter(s):
    """Rows of one adapter scattered over the batch give the bits of the same
    rows in runs, row by row; the gradients of the factors agree too, their
    rows being added in ascending order in both."""
    I, n = 320, 5
    runs = torch.arange(I, dtype=torch.int32) // 64
    c = Case(s, "whole", I, 512, 264, 16, n, ids=runs)
    C, low = c.forward()
    perm = torch.arange(I).reshape(5, 64).T.reshape(-1)  # round robin; ascending within each adapter
    d = Case(s, "whole", I, 512, 264, 16, n, ids=runs[perm])
    for k in ("A", "base", "dC", "dbase"):
        setattr(d, k, getattr(c, k)[perm])
    d.A_r = d.H.shard(d.plan, s.TENSOR_A, d.A)
    Cp, lowp = d.forward()
    assert torch.equal(C[0][perm.cuda()], Cp[0]) and torch.equal(low[perm.cuda()], lowp)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_repeats_its_bits(s, dt):
    c = Case(s, "contracted", 300, 1024, 520, 16, 6, dt, dt)
    C, low = c.forward()
    g = c.backward(low)
    for _ in range(3):
        C2, low2 = c.forward()
        g2 = c.backward(low2)
        assert torch.equal(low, low2) and all(torch.equal(a, b) for a, b in zip(C, C2))
        assert all(torch.equal(a, b) for a, b in zip(g[0], g2[0]))
        assert torch.equal(g[1], g2[1]) and torch.equal(g[2], g2[2])


@pytest.mark.gpu
def test_gradient_against_differences(s):
    """L = sum(C * dC) by central differences in 64 bits of the formula in
    every input of a small fp32 case; the formula is at most bilinear in each,
    so the differences are exact up to rounding."""
    c = Case(s, "whole", 6, 10, 9, 3, 2, "f32", "f32")
    C, low = c.forward()
    dA, dd, du = c.backward(low, None)
    v = {"A": c.A.double(), "down": c.down.double(), "up": c.up.double()}

    def loss(v):
        out = 0.0
        for a, idx in c.rows_of():
            out = out + (c.sc(a) * (v["A"][idx] @ v["down"][a].T @ v["up"][a]) * c.dC[idx].double()).sum()
        return out

    h = 1e-3
    for name, got in (("A", dA[0]), ("down", dd), ("up", du)):
        flat = got.double().cpu().flatten()
        for i in range(v[name].numel()):
            w = []
            for sg in (1, -1):
                t = dict(v)
                t[name] = v[name].clone()
                t[name].view(-1)[i] += sg * h
                w.append(loss(t))
            assert abs((w[0] - w[1]) / (2 * h) - flat[i]) < 1e-4


@pytest.mark.gpu
def test_captured_and_replayed(s):
    """Two graphs, each with its own workspace, of a decode step and its
    gradient replay in turn with eager bits on new inputs and new adapters
    per row."""
    cases = [Case(s, "rows", 24, 512, 512, 16, 8, seed=q) for q in range(2)]
    sets, graphs = [], []
    for c in cases:
        H = c.H
        b = {"C": H.alloc(c.plan, s.TENSOR_C), "base": c.cut(s.TENSOR_C, c.base), "dC": c.cut(s.TENSOR_C, c.dC),
             "dA": H.alloc(c.plan, s.TENSOR_A), "low": torch.empty(24, 16, device="cuda"),
             "dd": torch.empty(8, 16, 512, device="cuda"), "du": torch.empty(8, 16, 512, device="cuda"),
             "ws": H.adapters_workspace(c.plan, 8, 16)}
        sets.append(b)

    def step(c, b):
        d = c.dev
        c.plan.adapters_forward(c.A_r, d["ids"], d["down"], d["up"], d["scale"], b["base"], b["C"], b["low"])
        c.plan.adapters_backward(b["dC"], c.A_r, d["ids"], d["down"], d["up"], d["scale"], b["low"], None, b["dA"],
                                 b["dd"], b["du"], b["ws"])

    for c, b in zip(cases, sets):
        step(c, b)
    torch.cuda.synchronize()
    for c, b in zip(cases, sets):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step(c, b)
        graphs.append(g)
    for c in cases:
        c.dev["ids"].copy_(torch.randint(-1, 8, (24,), dtype=torch.int32))
        for t in c.A_r:
            t.copy_(torch.randn(t.shape).bfloat16())
    for g in (graphs[0], graphs[1], graphs[0]):
        g.replay()
    torch.cuda.synchronize()
    for c, b in zip(cases, sets):
        keep = {k: [t.clone() for t in (v if isinstance(v, list) else [v])] for k, v in b.items() if k != "ws"}
        step(c, b)
        torch.cuda.synchronize()
        for k, v in keep.items():
            for x, y in zip(v, b[k] if isinstance(b[k], list) else [b[k]]):
                assert torch.equal(x, y), k


@pytest.mark.gpu
def test_sequence_parallel_block_with_adapters(s):
    """The calls together, as a block of a sequence-parallel model on {X:4}
    uses them: LayerNorm + all-gather with statistics, the column-sharded
    projection, adapters beside it; then back: the adapters' gradient on top of
    the shared projection's, and LayerNorm's gradient with the reduce-scatter.
    Every rank's gradient of the gathered rows is a partial one: its own
    columns' (the adapters' part joins rank 0's).  Compared with the same
    chain in 64 bits: bf16 intermediates are off by 2^-8 each (half a step of
    the gathered rows, of C, of dA), so the end is within 2^-6 of the largest
    value of its own kind."""
    from partial_sum_reduction_gb300 import helpers as H
    T, D, F, R, n, G = 256, 512, 1024, 16, 6, 4
    g = torch.Generator().manual_seed(5)
    r = lambda *sh: torch.randn(*sh, generator=g)
    x = r(T, D).bfloat16()
    gamma, beta = 1 + 0.1 * r(D), 0.1 * r(D)
    W, down, up = (r(D, F) / D ** 0.5).bfloat16(), (r(n, R, D) / D ** 0.5).bfloat16(), (0.1 * r(n, R, F)).bfloat16()
    scale, ids = torch.rand(n, generator=g) + 0.5, torch.randint(-1, n, (T,), generator=g, dtype=torch.int32)
    dC = r(T, F).bfloat16()
    X4 = "{X:4}"
    gather = s.Plan(X4, "I_X,J", "J,K", "I,K", T, 8, D)
    proj = s.Plan(X4, "I,J", "J,K_X", "I,K_X", T, D, F)
    shards = H.shard(gather, s.TENSOR_C_REDUCED, x)
    full = H.alloc(gather, s.TENSOR_C)
    mean, rstd = ([torch.empty(T // G, device="cuda") for _ in range(G)] for _ in range(2))
    ga, be = gamma.cuda(), beta.cuda()
    gather.layernorm_all_gather_forward(shards, ga, be, full, mean, rstd)
    C = H.alloc(proj, s.TENSOR_C)
    proj.run(full, H.shard(proj, s.TENSOR_B, W), C, H.workspace(proj))
    low = torch.empty(T, R, device="cuda")
    ad = (ids.cuda(), down.cuda(), up.cuda(), scale.cuda())
    proj.adapters_forward(full, *ad, C, C, low)
    # back: rank q's dX = dC[:, q] . W[:, q]^T, fp32 partials of a plan that reduces over X
    back = s.Plan(X4, "I,J_X", "J_X,K", "I_X,K", T, F, D)
    dX = H.alloc(back, s.TENSOR_P)
    back.local_matmul(H.shard(back, s.TENSOR_A, dC), H.shard(back, s.TENSOR_B, W.T.contiguous()), dX)
    dd, du = torch.empty(n, R, D, device="cuda"), torch.empty(n, R, F, device="cuda")
    dA = H.alloc(proj, s.TENSOR_A)
    proj.adapters_backward(H.shard(proj, s.TENSOR_C, dC), full, *ad, low, None, dA, dd, du,
                           H.adapters_workspace(proj, n, R))
    dX[0] += dA[0].float()
    dx = H.alloc(gather, s.TENSOR_C_REDUCED)
    dg, db = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    gather.layernorm_all_gather_backward(dX, shards, mean, rstd, ga, dx, dg, db, H.layernorm_workspace(T, D))
    s.shmm_sync_status()
    # the same in 64 bits
    v = {k: t.double().requires_grad_() for k, t in (("x", x), ("gamma", gamma), ("beta", beta), ("down", down),
                                                     ("up", up))}
    mu = v["x"].mean(1, keepdim=True)
    var = ((v["x"] - mu) ** 2).mean(1, keepdim=True)
    y = (v["x"] - mu) / torch.sqrt(var + 1e-5) * v["gamma"] + v["beta"]
    out = y @ W.double()
    pick = ids.clamp(min=0).long()
    s_eff = torch.where(ids >= 0, scale.double()[pick], torch.zeros((), dtype=torch.float64))
    out = out + s_eff[:, None] * torch.einsum("tr,trk->tk", torch.einsum("tj,trj->tr", y, v["down"][pick]),
                                              v["up"][pick])
    (out * dC.double()).sum().backward()
    got = torch.cat([c.double().cpu() for c in C], 1)
    for a, b in ((got, out.detach()), (torch.cat([t.double().cpu() for t in dx]), v["x"].grad),
                 (dg.double().cpu(), v["gamma"].grad), (db.double().cpu(), v["beta"].grad),
                 (dd.double().cpu(), v["down"].grad), (du.double().cpu(), v["up"].grad)):
        assert (a - b).abs().max() <= 2.0 ** -6 * b.abs().max()
