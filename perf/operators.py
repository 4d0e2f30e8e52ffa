"""Cases of the row-normalisation and low-rank-adapter operators: inputs, one
pass through each (in plain torch, or through the library), and the result
from the definition in 64 bits.

Operators (``case["op"]``):
  ln_forward    layer normalisation of token rows with saved statistics, with
                a residual added on the way, or gathered to every rank
  ln_backward   its gradient: rows, gain and bias; with the members' gradients
                of a gathered result summed on the way
  adapt         a low-rank adapter per token row beside a shared projection
  adapt_grad    the gradient of that: rows, and every adapter's two factors
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # four token rows of one decoding step, residual added before the norm
        {"name": "ln_forward_decode", "op": "ln_forward", "rows": 4, "cols": 4096, "dtype": "bf16", "ranks": 1,
         "residual": True},
        # the MLP block's 8192 tokens, residual added before the norm
        {"name": "ln_forward_tokens", "op": "ln_forward", "rows": 8192, "cols": 4096, "dtype": "bf16", "ranks": 1,
         "residual": True},
        # sequence parallelism: 8 owners of 1024 tokens, gathered to all 8
        {"name": "ln_forward_gather", "op": "ln_forward", "rows": 8192, "cols": 4096, "dtype": "bf16", "ranks": 8,
         "residual": False},
        # a training step's norm with the gradient of the residual branch joined
        {"name": "ln_backward_tokens", "op": "ln_backward", "rows": 8192, "cols": 4096, "dtype": "bf16", "ranks": 1,
         "grad": "bf16", "residual": True},
        # a small fp32 step whose rows are no whole 16-byte vectors
        {"name": "ln_backward_odd", "op": "ln_backward", "rows": 1031, "cols": 1157, "dtype": "f32", "ranks": 1,
         "grad": "f32", "residual": False},
        # sequence parallelism's backward: 8 ranks' fp32 partial gradients
        {"name": "ln_backward_scatter", "op": "ln_backward", "rows": 8192, "cols": 4096, "dtype": "bf16", "ranks": 8,
         "grad": "f32", "residual": False},
        # one token of one request
        {"name": "adapt_one_token", "op": "adapt", "layout": "whole", "rows": 1, "J": 4096, "K": 4096, "rank": 16,
         "adapters": 8, "requests": 1, "dtype": "bf16"},
        # a decoding batch: 96 requests of one token each, 64 adapters
        {"name": "adapt_decode", "op": "adapt", "layout": "rows", "rows": 96, "J": 8192, "K": 8192, "rank": 16,
         "adapters": 64, "requests": 96, "dtype": "bf16"},
        # prompts of 24 requests through the down-projection on {X:4,Y:2}
        {"name": "adapt_prompts", "op": "adapt", "layout": "contracted", "rows": 8192, "J": 28672, "K": 8192,
         "rank": 16, "adapters": 12, "requests": 24, "dtype": "bf16"},
        # a small fp32 fine-tuning step of odd sizes
        {"name": "adapt_grad_odd", "op": "adapt_grad", "layout": "whole", "rows": 301, "J": 1000, "K": 1157,
         "rank": 12, "adapters": 3, "requests": 7, "dtype": "f32"},
        # four adapters tuned at once on a square projection
        {"name": "adapt_grad_square", "op": "adapt_grad", "layout": "whole", "rows": 4096, "J": 4096, "K": 4096,
         "rank": 16, "adapters": 4, "requests": 16, "dtype": "bf16"},
        # eight adapters of rank 32 on the column-sharded first MLP matmul, {X:8}
        {"name": "adapt_grad_columns", "op": "adapt_grad", "layout": "columns", "rows": 8192, "J": 4096, "K": 16384,
         "rank": 32, "adapters": 8, "requests": 32, "dtype": "bf16"},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_forward", "ln_backward", "adapt", "adapt_grad"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("ln_forward", "ln_backward"):
        ranks = rng.choice([1, 1, 2, 4, 8])
        rows = _spread(rng, 1, 8192 // ranks) * ranks
        cols = _spread(rng, 64, 8192 if rows <= 4096 else 4096)
        if rng.random() < 0.6:
            cols = (cols + 7) // 8 * 8
        case = {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "ranks": ranks,
                "residual": ranks == 1 and rng.random() < 0.5}
        if op == "ln_backward":
            case["grad"] = rng.choice([dtype, "f32"]) if ranks > 1 else dtype
        return case
    layout = rng.choice(["whole", "rows", "contracted", "columns"])
    split = {"whole": 1, "rows": 4, "contracted": 4, "columns": 1}[layout]
    rows = _spread(rng, 1, (8192 if dtype == "bf16" else 1024) // split) * split
    top = 8192 if rows <= 2048 else 4096
    J, K = _spread(rng, 128, top), _spread(rng, 128, top)
    if rng.random() < 0.75:
        J, K = (J + 7) // 8 * 8, (K + 7) // 8 * 8
    if layout == "contracted":
        J += J % 2
    if layout == "columns":
        K = (K + 7) // 8 * 8
    adapters = _spread(rng, 1, 32)
    return {"op": op, "layout": layout, "rows": rows, "J": J, "K": K, "rank": rng.choice([4, 8, 12, 16, 16, 32, 64]),
            "adapters": adapters, "requests": min(rows, _spread(rng, 1, 96)), "dtype": dtype}


# ------------------------------------------------- sharding of the rows

# mesh, specs of A[I,J], B[J,K], C[I,K], and per rank (i part, of; j part,
# of; k part, of): which slice of A (i, j) and of C (i, k) the rank holds.
LAYOUTS = {
    "whole": ("{X:1}", "I,J", "J,K", "I,K", [((0, 1), (0, 1), (0, 1))]),
    "rows": ("{X:4}", "I_X,J", "J,K", "I_X,K", [((r, 4), (0, 1), (0, 1)) for r in range(4)]),
    "contracted": ("{X:4,Y:2}", "I_X,J_Y", "J_Y,K", "I_X,K", [((r // 2, 4), (r % 2, 2), (0, 1)) for r in range(8)]),
    "columns": ("{X:8}", "I,J", "J,K_X", "I,K_X", [((0, 1), (0, 1), (r, 8)) for r in range(8)]),
}


def _part(n, part):
    q, of = part
    return slice(q * n // of, (q + 1) * n // of)


def _cut_A(case, full):
    return [full[_part(case["rows"], i), _part(case["J"], j)].contiguous() if len(LAYOUTS[case["layout"]][4]) > 1
            else full for i, j, k in LAYOUTS[case["layout"]][4]]


def _cut_C(case, full):
    return [full[_part(case["rows"], i), _part(case["K"], k)].contiguous() if len(LAYOUTS[case["layout"]][4]) > 1
            else full for i, j, k in LAYOUTS[case["layout"]][4]]


def _whole(case, shards, width, which):
    """The global array from the ranks' slices (each slice from the first
    rank that holds it)."""
    parts = LAYOUTS[case["layout"]][4]
    if len(parts) == 1:
        return shards[0]
    out = torch.empty(case["rows"], width, dtype=shards[0].dtype, device=shards[0].device)
    seen = set()
    for (i, j, k), t in zip(parts, shards):
        c = j if which == "A" else k
        if (i, c) not in seen:
            seen.add((i, c))
            out[_part(case["rows"], i), _part(width, c)] = t
    return out


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rows_like_activations(g, rows, cols):
    """Token rows: a scale per token, an offset per feature, a few features
    far larger than the rest."""
    x = _normal(g, rows, cols)
    x *= torch.exp(0.3 * _normal(g, rows, 1))
    x += 0.2 * _normal(g, 1, cols)
    x[:, :: max(1, cols // 5)] *= 12.0
    return x


def _ln_inputs(case, seed):
    g = _gen(seed)
    rows, cols, G = case["rows"], case["cols"], case["ranks"]
    dt = DTYPES[case["dtype"]]
    st = {"x": _rows_like_activations(g, rows, cols).to(dt), "gamma": 1.0 + 0.1 * _normal(g, cols),
          "beta": 0.1 * _normal(g, cols)}
    if case["op"] == "ln_forward":
        if case["residual"]:
            st["residual"] = _rows_like_activations(g, rows, cols).to(dt)
        return st
    xd = st["x"].double()
    mean = xd.mean(1)
    st["mean"] = mean.float()
    st["rstd"] = ((xd - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
    gdt = DTYPES[case["grad"]]
    st["dy"] = [(_normal(g, rows, cols) * 0.02).to(gdt) for _ in range(G)]
    if case["residual"]:
        st["dres"] = (_normal(g, rows, cols) * 0.02).to(dt)
    return st


def _row_adapters(case, g):
    """Rows of one request are together and share its adapter; every tenth
    request has none, and the last rows of a batch that is not full have no
    request.  Each adapter is used when there are requests enough."""
    rows, q, n = case["rows"], case["requests"], case["adapters"]
    host = torch.Generator().manual_seed(int(torch.randint(1 << 30, (1,), generator=g, device="cuda")))
    used = rows - rows // 50
    cuts = torch.randperm(max(used - 1, 1), generator=host)[:q - 1] + 1 if q < used else torch.arange(1, used)
    bounds = sorted(set([0, used] + [int(c) for c in cuts if 0 < int(c) < used]))
    order = torch.randperm(n, generator=host).tolist()
    ids = torch.full((rows,), -1, dtype=torch.int32)
    left = 0
    for i, (a, b) in enumerate(zip(bounds[:-1], bounds[1:])):
        if i % 10 == 9:
            continue
        ids[a:b] = order[left % n]
        left += 1
    return ids


def _adapt_inputs(case, seed):
    g = _gen(seed)
    T, J, K, R, n = case["rows"], case["J"], case["K"], case["rank"], case["adapters"]
    dt = DTYPES[case["dtype"]]
    st = {"A": _normal(g, T, J).to(dt), "down": (_normal(g, n, R, J) / math.sqrt(J)).to(dt),
          "up": (0.05 * _normal(g, n, R, K)).to(dt), "scale": 0.5 + torch.rand(n, generator=g, device="cuda")}
    ids = _row_adapters(case, g)
    st["ids"], st["ids_host"] = ids.cuda(), ids
    if case["op"] == "adapt":
        st["base"] = _normal(g, T, K).to(dt)
        return st
    st["dC"] = (0.02 * _normal(g, T, K)).to(dt)
    st["base"] = (0.02 * _normal(g, T, J)).to(dt)
    low = torch.zeros(T, R, dtype=torch.float32, device="cuda")
    for a in range(n):
        idx = (ids == a).nonzero().flatten().cuda()
        if len(idx):
            low[idx] = st["A"][idx].float() @ st["down"][a].float().T
    st["low"] = low
    return st


def prepare(case, seed):
    st = {"case": case}
    if case["op"] in ("ln_forward", "ln_backward"):
        st.update(_ln_inputs(case, seed))
        rows, cols, G = case["rows"], case["cols"], case["ranks"]
        if G > 1:
            b = rows // G
            st["x"] = [st["x"][p * b:(p + 1) * b].clone() for p in range(G)]
            if case["op"] == "ln_backward":
                for k in ("mean", "rstd"):
                    st[k] = [st[k][p * b:(p + 1) * b].clone() for p in range(G)]
        if own:
            import partial_sum_reduction_gb300 as s
            dev = {"device": "cuda"}
            dt = DTYPES[case["dtype"]]
            if G > 1:
                st["plan"] = s.Plan([("X", G)], "I_X,J", "J,K", "I,K", rows, 8, cols, case["dtype"], case["dtype"])
            b = rows // G
            if case["op"] == "ln_forward":
                st["y"] = [torch.empty(rows, cols, dtype=dt, **dev) for _ in range(G)]
                st["total"] = torch.empty(rows, cols, dtype=dt, **dev) if case["residual"] else None
                st["mean"] = [torch.empty(b, **dev) for _ in range(G)]
                st["rstd"] = [torch.empty(b, **dev) for _ in range(G)]
            else:
                st["dx"] = [torch.empty(b, cols, dtype=dt, **dev) for _ in range(G)]
                st["dgamma"], st["dbeta"] = torch.empty(cols, **dev), torch.empty(cols, **dev)
                st["workspace"] = s.helpers.layernorm_workspace(rows, cols)
        return st
    inp = _adapt_inputs(case, seed)
    T, J, K, R, n = case["rows"], case["J"], case["K"], case["rank"], case["adapters"]
    grad = case["op"] == "adapt_grad"
    for k in ("down", "up", "scale", "ids"):
        st[k] = inp[k]
    st["A"] = _cut_A(case, inp["A"])
    st["base"] = _cut_A(case, inp["base"]) if grad else _cut_C(case, inp["base"])
    if grad:
        st["dC"], st["low"] = _cut_C(case, inp["dC"]), inp["low"]
    if own:
        import partial_sum_reduction_gb300 as s
        mesh, sa, sb, sc, _ = LAYOUTS[case["layout"]]
        st["plan"] = s.Plan(mesh, sa, sb, sc, T, J, K, case["dtype"], case["dtype"])
        # a rank's shard is a buffer of its own, which a view of the whole at an odd offset is not
        for k in ("A", "base", "dC"):
            if k in st:
                st[k] = [t.clone() if t.data_ptr() % 16 else t for t in st[k]]
        st["out"] = [torch.empty_like(t) for t in st["base"]]
        if grad:
            st["ddown"] = torch.empty(n, R, J, device="cuda")
            st["dup"] = torch.empty(n, R, K, device="cuda")
            st["workspace"] = s.helpers.adapters_workspace(st["plan"], n, R)
        else:
            st["low"] = torch.empty(T, R, device="cuda")
    else:
        # the rows of each adapter, as the program that placed the requests knows them
        st["rows_of"] = [(a, (inp["ids_host"] == a).nonzero().flatten().cuda()) for a in range(n)
                         if bool((inp["ids_host"] == a).any())]
    return st


# -------------------------------------------------------------- plain forms

def _plain_ln_forward(case, st):
    dt = DTYPES[case["dtype"]]
    x = torch.cat(st["x"]) if case["ranks"] > 1 else st["x"]
    t = x.float()
    out = {}
    if case["residual"]:
        out["total"] = (t + st["residual"].float()).to(dt)
        t = out["total"].float()
    mean = t.sum(1) / case["cols"]
    d = t - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).sum(1) / case["cols"] + EPS)
    y = (d * rstd[:, None] * st["gamma"] + st["beta"]).to(dt)
    out["y"] = [y] + [y.clone() for _ in range(case["ranks"] - 1)]
    out["mean"], out["rstd"] = mean, rstd
    return out


def _plain_ln_backward(case, st):
    dt = DTYPES[case["dtype"]]
    G, cols = case["ranks"], case["cols"]
    cat = torch.cat if G > 1 else (lambda t: t)
    dy = st["dy"][0].float()
    for m in range(1, G):
        dy = dy + st["dy"][m].float()
    mean, rstd = cat(st["mean"]), cat(st["rstd"])
    xh = (cat(st["x"]).float() - mean[:, None]) * rstd[:, None]
    g = dy * st["gamma"]
    dx = rstd[:, None] * (g - g.sum(1, keepdim=True) / cols - xh * ((g * xh).sum(1, keepdim=True) / cols))
    if case["residual"]:
        dx = dx + st["dres"].float()
    return {"dx": dx.to(dt), "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0)}


def _plain_adapt(case, st):
    T, K, R = case["rows"], case["K"], case["rank"]
    A = _whole(case, st["A"], case["J"], "A")
    low = torch.zeros(T, R, dtype=torch.float32, device="cuda")
    delta = torch.zeros(T, K, dtype=torch.float32, device="cuda")
    for a, idx in st["rows_of"]:
        s = A[idx].float() @ st["down"][a].float().T
        low[idx] = s
        delta[idx] = (s @ st["up"][a].float()) * st["scale"][a]
    parts = LAYOUTS[case["layout"]][4]
    return {"C": [(b.float() + delta[_part(T, i), _part(K, k)]).to(b.dtype)
                  for (i, j, k), b in zip(parts, st["base"])], "low": low}


def _plain_adapt_grad(case, st):
    T, J, K, R, n = case["rows"], case["J"], case["K"], case["rank"], case["adapters"]
    A, dC = _whole(case, st["A"], J, "A"), _whole(case, st["dC"], K, "C")
    dA = torch.zeros(T, J, dtype=torch.float32, device="cuda")
    ddown = torch.zeros(n, R, J, dtype=torch.float32, device="cuda")
    dup = torch.zeros(n, R, K, dtype=torch.float32, device="cuda")
    for a, idx in st["rows_of"]:
        d = dC[idx].float()
        ds = (d @ st["up"][a].float().T) * st["scale"][a]
        dA[idx] = ds @ st["down"][a].float()
        ddown[a] = ds.T @ A[idx].float()
        dup[a] = (st["low"][idx].T @ d) * st["scale"][a]
    parts = LAYOUTS[case["layout"]][4]
    return {"dA": [(b.float() + dA[_part(T, i), _part(J, j)]).to(b.dtype)
                   for (i, j, k), b in zip(parts, st["base"])], "ddown": ddown, "dup": dup}


# -------------------------------------------------------- the library's calls

def _own_ln_forward(case, st):
    import partial_sum_reduction_gb300 as s
    if case["ranks"] > 1:
        st["plan"].layernorm_all_gather_forward(st["x"], st["gamma"], st["beta"], st["y"], st["mean"], st["rstd"],
                                                eps=EPS)
        return {"y": st["y"], "mean": torch.cat(st["mean"]), "rstd": torch.cat(st["rstd"])}
    s.shmm_layernorm_forward(st["x"], st["gamma"], st["beta"], st["y"][0], st["mean"][0], st["rstd"][0],
                             residual=st.get("residual"), total=st["total"], eps=EPS)
    out = {"total": st["total"]} if case["residual"] else {}
    out.update({"y": st["y"], "mean": st["mean"][0], "rstd": st["rstd"][0]})
    return out


def _own_ln_backward(case, st):
    import partial_sum_reduction_gb300 as s
    if case["ranks"] > 1:
        st["plan"].layernorm_all_gather_backward(st["dy"], st["x"], st["mean"], st["rstd"], st["gamma"], st["dx"],
                                                 st["dgamma"], st["dbeta"], st["workspace"])
        return {"dx": st["dx"], "dgamma": st["dgamma"], "dbeta": st["dbeta"]}
    s.shmm_layernorm_backward(st["dy"][0], st["x"], st["mean"], st["rstd"], st["gamma"], st["dx"][0], st["dgamma"],
                              st["dbeta"], st["workspace"], residual_grad=st.get("dres"))
    return {"dx": st["dx"], "dgamma": st["dgamma"], "dbeta": st["dbeta"]}


def _own_adapt(case, st):
    st["plan"].adapters_forward(st["A"], st["ids"], st["down"], st["up"], st["scale"], st["base"], st["out"],
                                st["low"])
    return {"C": st["out"], "low": st["low"]}


def _own_adapt_grad(case, st):
    st["plan"].adapters_backward(st["dC"], st["A"], st["ids"], st["down"], st["up"], st["scale"], st["low"],
                                 st["base"], st["out"], st["ddown"], st["dup"], st["workspace"])
    return {"dA": st["out"], "ddown": st["ddown"], "dup": st["dup"]}


def run(state):
    case = state["case"]
    if own:
        return {"ln_forward": _own_ln_forward, "ln_backward": _own_ln_backward, "adapt": _own_adapt,
                "adapt_grad": _own_adapt_grad}[case["op"]](case, state)
    out = {"ln_forward": _plain_ln_forward, "ln_backward": _plain_ln_backward, "adapt": _plain_adapt,
           "adapt_grad": _plain_adapt_grad}[case["op"]](case, state)
    if case["op"] == "ln_backward":
        b = case["rows"] // case["ranks"]
        out["dx"] = [out["dx"][p * b:(p + 1) * b] for p in range(case["ranks"])]
    return out


# --------------------------------------------------------------------- work

def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] in ("ln_forward", "ln_backward"):
        n, G = case["rows"] * case["cols"], case["ranks"]
        if case["op"] == "ln_forward":
            b = n * es * (1 + G + (2 if case["residual"] else 0)) + 8 * case["rows"] + 8 * case["cols"]
            return {"bytes": b, "flops": n * 8}
        ge = 4 if case["grad"] == "f32" else 2
        b = n * (es * (2 + (1 if case["residual"] else 0)) + G * ge) + 8 * case["rows"] + 12 * case["cols"]
        return {"bytes": b, "flops": n * (14 + G)}
    T, J, K, R = case["rows"], case["J"], case["K"], case["rank"]
    parts = LAYOUTS[case["layout"]][4]
    held_A = sum((T // i[1]) * (J // j[1]) for i, j, k in parts)   # elements over all ranks
    held_C = sum((T // i[1]) * (K // k[1]) for i, j, k in parts)
    used = min(case["adapters"], max(1, case["requests"] - case["requests"] // 10))
    factors = used * R * (J + K) * es + 4 * T * R + 4 * T
    if case["op"] == "adapt":
        return {"bytes": T * J * es + 2 * held_C * es + factors, "flops": 2 * T * R * (J + K)}
    grads = 4 * case["adapters"] * R * (J + K)
    return {"bytes": T * (J + K) * es + 2 * held_A * es + factors + grads, "flops": 4 * T * R * (J + K)}


# -------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    if case["op"] == "ln_forward":
        st = _ln_inputs(case, seed)
        t = st["x"].double()
        out = {}
        if case["residual"]:
            # the statistics are those of the stored sum, so it is rounded here too
            out["total"] = t + st["residual"].double()
            t = (st["x"].float() + st["residual"].float()).to(DTYPES[case["dtype"]]).double()
        var, mean = torch.var_mean(t, dim=1, correction=0)
        rstd = torch.rsqrt(var + EPS)
        y = torch.addcmul(st["beta"].double(), (t - mean.unsqueeze(1)) * rstd.unsqueeze(1), st["gamma"].double())
        out.update({"y": [y] * case["ranks"], "mean": mean, "rstd": rstd})
        return out
    if case["op"] == "ln_backward":
        # the adjoint applied directly: dx = J^T dy with J's projections written as means over the row
        st = _ln_inputs(case, seed)
        dy = torch.zeros_like(st["dy"][0], dtype=torch.float64)
        for d in st["dy"]:
            dy += d.double()
        r = st["rstd"].double().unsqueeze(1)
        xh = r * (st["x"].double() - st["mean"].double().unsqueeze(1))
        w = dy * st["gamma"].double()
        dx = w - w.mean(1, keepdim=True)
        dx -= xh * torch.einsum("ij,ij->i", w, xh).unsqueeze(1) / case["cols"]
        dx *= r
        if case["residual"]:
            dx += st["dres"].double()
        return {"dx": list(dx.split(case["rows"] // case["ranks"])), "dgamma": torch.einsum("ij,ij->j", dy, xh),
                "dbeta": dy.sum(0)}
    st = _adapt_inputs(case, seed)
    T, J, K, R = case["rows"], case["J"], case["K"], case["rank"]
    ids = st["ids_host"].numpy()
    one_hot = {a: torch.from_numpy(np.flatnonzero(ids == a)).cuda() for a in np.unique(ids) if a >= 0}
    parts = LAYOUTS[case["layout"]][4]
    f64 = {"dtype": torch.float64, "device": "cuda"}
    if case["op"] == "adapt":
        low, C = torch.zeros(T, R, **f64), st["base"].double()
        for a, rows in one_hot.items():
            low[rows] = torch.einsum("tj,rj->tr", st["A"][rows].double(), st["down"][a].double())
            C[rows] += st["scale"][a].double() * torch.einsum("tr,rk->tk", low[rows], st["up"][a].double())
        return {"C": [C[_part(T, i), _part(K, k)] for i, j, k in parts], "low": low}
    dA = st["base"].double()
    ddown, dup = torch.zeros(case["adapters"], R, J, **f64), torch.zeros(case["adapters"], R, K, **f64)
    for a, rows in one_hot.items():
        a = int(a)
        g = st["dC"][rows].double() * st["scale"][a].double()
        ds = torch.einsum("tk,rk->tr", g, st["up"][a].double())
        dA[rows] += torch.einsum("tr,rj->tj", ds, st["down"][a].double())
        ddown[a] = torch.einsum("tr,tj->rj", ds, st["A"][rows].double())
        dup[a] = torch.einsum("tr,tk->rk", st["low"][rows].double(), g)
    return {"dA": [dA[_part(T, i), _part(J, j)] for i, j, k in parts], "ddown": ddown, "dup": dup}
