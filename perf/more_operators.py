"""Cases of the 8-bit and gated operators: inputs, one pass through each (in
plain torch, or through the library), and the result from the definition in
64 bits.

Operators (``case["op"]``):
  quantize     8-bit values (e4m3) with a power-of-two scale for each block of
               128 (of a row, or 128 x 128), and the way back
  scaled       the sharded matmul of such operands
  scaled_grad  its gradient: A's rows, and B from the 8-bit A that was kept
  gated        the gated first half of an MLP block, act(A.gate) * (A.up), with
               the two pre-activations kept for the gradient
  gated_grad   its gradient: A's rows and both projections
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
BLOCK = 128


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the activations of a decoding batch before an 8-bit matmul
        {"name": "quantize_decode", "op": "quantize", "way": "to", "rows": 16, "cols": 4096, "block_rows": 1,
         "dtype": "bf16"},
        # the MLP block's hidden activations, kept in 8 bits for the backward pass
        {"name": "quantize_tokens", "op": "quantize", "way": "to", "rows": 8192, "cols": 16384, "block_rows": 1,
         "dtype": "bf16"},
        # 8192 tokens of a block's input back in bf16
        {"name": "restore_tokens", "op": "quantize", "way": "back", "rows": 8192, "cols": 4096, "block_rows": 1,
         "dtype": "bf16"},
        # a decoding step of 16 requests through the first MLP matmul's weights in 8 bits
        {"name": "scaled_decode", "op": "scaled", "layout": "columns", "rows": 16, "J": 4096, "K": 16384,
         "out": "bf16"},
        # the down-projection on {X:4,Y:2}, both operands in 8 bits
        {"name": "scaled_down_projection", "op": "scaled", "layout": "contracted", "rows": 8192, "J": 28672, "K": 8192,
         "out": "bf16"},
        # a small step of sizes that end inside blocks and tiles
        {"name": "scaled_grad_odd", "op": "scaled_grad", "layout": "whole", "rows": 1000, "J": 1040, "K": 2032},
        # the training step of the column-sharded first MLP matmul, {X:8}
        {"name": "scaled_grad_columns", "op": "scaled_grad", "layout": "columns", "rows": 8192, "J": 4096, "K": 16384},
        # four token rows of one decoding step, nothing kept
        {"name": "gated_decode", "op": "gated", "layout": "columns", "rows": 4, "J": 4096, "K": 16384, "dtype": "bf16",
         "act": "silu", "saved": "none"},
        # a small fp32 step of odd sizes
        {"name": "gated_odd", "op": "gated", "layout": "whole", "rows": 301, "J": 1000, "K": 1157, "dtype": "f32",
         "act": "gelu", "saved": "f32"},
        # the MLP block's 8192 tokens, {X:8}, pre-activations kept in 8 bits
        {"name": "gated_tokens", "op": "gated", "layout": "columns", "rows": 8192, "J": 4096, "K": 16384,
         "dtype": "bf16", "act": "silu", "saved": "e4m3"},
        # a fine-tuning step of a few hundred tokens, pre-activations kept as they were
        {"name": "gated_grad_small", "op": "gated_grad", "layout": "whole", "rows": 515, "J": 1024, "K": 2816,
         "dtype": "bf16", "act": "gelu", "saved": "bf16"},
        # the backward pass of the block's 8192 tokens, from 8 bits
        {"name": "gated_grad_columns", "op": "gated_grad", "layout": "columns", "rows": 8192, "J": 4096, "K": 16384,
         "dtype": "bf16", "act": "silu", "saved": "e4m3"},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "scaled", "scaled_grad", "gated", "gated_grad"])
    if op == "quantize":
        rows = _spread(rng, 1, 8192)
        cols = _spread(rng, 64, 16384)
        if rng.random() < 0.7:
            cols = (cols + 15) // 16 * 16
        return {"op": op, "way": rng.choice(["to", "to", "back"]), "rows": rows, "cols": cols,
                "block_rows": rng.choice([1, 1, 1, 128]), "dtype": rng.choice(["bf16", "bf16", "bf16", "f32"])}
    f32 = op in ("gated", "gated_grad") and rng.random() < 0.15
    layout = "whole" if f32 else rng.choice(["whole", "rows", "contracted", "columns"])
    top = 8192 if layout != "columns" else 16384
    rows = _spread(rng, 1, 1024 if f32 else 8192)
    J, K = _spread(rng, 128, 1024 if f32 else 4096), _spread(rng, 128, 1500 if f32 else top)
    if not f32:
        # what the shards of a real model are: whole 16-byte rows, edges on whole blocks
        J, K = (J + 15) // 16 * 16, (K + 15) // 16 * 16
        if layout == "rows":
            rows = max(512, rows // 512 * 512)
        if layout == "contracted":
            rows, J = max(512, rows // 512 * 512), (J + 255) // 256 * 256
        if layout == "columns":
            K = (K + 1023) // 1024 * 1024
    case = {"op": op, "layout": layout, "rows": rows, "J": J, "K": K}
    if op == "scaled":
        case["out"] = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("gated", "gated_grad"):
        case["dtype"] = "f32" if f32 else "bf16"
        case["act"] = rng.choice(["silu", "silu", "gelu"])
        case["saved"] = rng.choice(["e4m3", "e4m3", case["dtype"]] + (["none"] if op == "gated" else []))
    return case


# ------------------------------------------------------- sharding and blocks

# mesh, specs of A[I,J], B[J,K], C[I,K], and per rank (i part, of; j part,
# of; k part, of): which slice of A (i, j), B (j, k) and C (i, k) it holds.
LAYOUTS = {
    "whole": ("{X:1}", "I,J", "J,K", "I,K", [((0, 1), (0, 1), (0, 1))]),
    "rows": ("{X:4}", "I_X,J", "J,K", "I_X,K", [((r, 4), (0, 1), (0, 1)) for r in range(4)]),
    "contracted": ("{X:4,Y:2}", "I_X,J_Y", "J_Y,K", "I_X,K", [((r // 2, 4), (r % 2, 2), (0, 1)) for r in range(8)]),
    "columns": ("{X:8}", "I,J", "J,K_X", "I,K_X", [((0, 1), (0, 1), (r, 8)) for r in range(8)]),
}
DIMS = {"A": (0, 1), "B": (1, 2), "C": (0, 2)}


def _parts(case, which):
    """Per rank: (row part, column part) of its slice of A, B or C."""
    d0, d1 = DIMS[which]
    return [(p[d0], p[d1]) for p in LAYOUTS[case["layout"]][4]]


def _part(n, part):
    q, of = part
    return slice(q * n // of, (q + 1) * n // of)


def _cut(case, full, which):
    """A buffer per rank with its slice of a whole array."""
    return [full[_part(full.shape[0], r), _part(full.shape[1], c)].clone() for r, c in _parts(case, which)]


def _distinct(case, which):
    """(row part, column part, first rank that holds it) of every slice."""
    seen = {}
    for rank, key in enumerate(_parts(case, which)):
        seen.setdefault(key, rank)
    return [(r, c, rank) for (r, c), rank in seen.items()]


def _whole(case, shards, which, rows, cols):
    """The whole array from the ranks' slices (each from the first that holds it)."""
    out = torch.empty(rows, cols, dtype=shards[0].dtype, device=shards[0].device)
    for r, c, rank in _distinct(case, which):
        out[_part(rows, r), _part(cols, c)] = shards[rank]
    return out


def _blocks(x, block_rows):
    """x [rows, cols], padded with zeros to whole blocks, as [row blocks,
    block_rows, column blocks, 128]."""
    rows, cols = x.shape
    rb, cb = -(-rows // block_rows), -(-cols // BLOCK)
    if (rb * block_rows, cb * BLOCK) != (rows, cols):
        p = torch.zeros(rb * block_rows, cb * BLOCK, dtype=x.dtype, device=x.device)
        p[:rows, :cols] = x
        x = p
    return x.reshape(rb, block_rows, cb, BLOCK)


def _to_8bit(x, block_rows):
    """(e4m3 values, fp32 scales) of x: a block's scale is the smallest power
    of two 2^e with 448 2^e >= its largest magnitude (1 for a block of zeros),
    its values are x 2^-e rounded to nearest even."""
    v = _blocks(x, block_rows)
    amax = v.abs().amax(dim=(1, 3)).float()
    m, p = torch.frexp(amax)
    e = torch.clamp(p - 9 + (m > 0.875).to(torch.int32), min=-126)
    # 2^e by its bits: a power function may be off by a unit in the last place
    scale = torch.where(amax > 0, ((e + 127) << 23).view(torch.float32), torch.ones_like(amax))
    codes = (v / scale[:, None, :, None].to(v.dtype)).to(torch.float32).to(E4M3)
    return codes.reshape(v.shape[0] * block_rows, -1)[:x.shape[0], :x.shape[1]].contiguous(), scale


def _from_8bit(codes, scale, block_rows, dtype=torch.float32):
    v = _blocks(codes.to(dtype), block_rows) * scale[:, None, :, None].to(dtype)
    return v.reshape(v.shape[0] * block_rows, -1)[:codes.shape[0], :codes.shape[1]]


def _act(name, x):
    """(value, derivative) of the gate's activation."""
    if name == "silu":
        s = torch.sigmoid(x)
        return x * s, s * (1 + x * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (x + 0.044715 * x * x * x))
    return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)


# ------------------------------------------------------------------ inputs

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, rows, cols):
    """Token rows: a scale per token, a few features far larger than the rest."""
    x = _normal(g, rows, cols)
    x *= torch.exp(0.3 * _normal(g, rows, 1))
    x[:, :: max(1, cols // 5)] *= 12.0
    return x


def _inputs(case, seed):
    """The whole arrays, as the definition takes them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "quantize":
        x = _activations(g, case["rows"], case["cols"]).to(DTYPES[case["dtype"]])
        if case["way"] == "to":
            return {"x": x}
        codes, scale = _to_8bit(x, case["block_rows"])
        return {"codes": codes, "scale": scale}
    T, J, K = case["rows"], case["J"], case["K"]
    st = {}
    if case["op"] in ("scaled", "scaled_grad"):
        # every rank quantises its own slices; their edges fall on whole blocks
        st["A"], st["A_scale"] = _to_8bit(_activations(g, T, J).to(torch.bfloat16), 1)
        st["B"], st["B_scale"] = _to_8bit((_normal(g, J, K) / math.sqrt(J)).to(torch.bfloat16), BLOCK)
        if case["op"] == "scaled_grad":
            st["dC"] = (0.02 * _activations(g, T, K)).to(torch.bfloat16)
        return st
    dt = DTYPES[case["dtype"]]
    st["A"] = _normal(g, T, J).to(dt)
    for name in ("gate", "up"):
        st[name] = (_normal(g, J, K) * (1.3 / math.sqrt(J))).to(dt)
    if case["op"] == "gated_grad":
        st["dC"] = (0.02 * _normal(g, T, K)).to(dt)
        for name in ("gate", "up"):
            h = 1.3 * _activations(g, T, K)
            if case["saved"] == "e4m3":
                st["saved_" + name], st["saved_" + name + "_scale"] = _to_8bit(h, 1)
            else:
                st["saved_" + name] = h.to(dt)
    return st


def prepare(case, seed):
    inp = _inputs(case, seed)
    st = {"case": case}
    dev = {"device": "cuda"}
    if case["op"] == "quantize":
        st.update(inp)
        rows, cols, br = case["rows"], case["cols"], case["block_rows"]
        if case["way"] == "to":
            st["codes"] = torch.empty(rows, cols, dtype=E4M3, **dev)
            st["scale"] = torch.empty(-(-rows // br), -(-cols // BLOCK), **dev)
        else:
            st["y"] = torch.empty(rows, cols, dtype=DTYPES[case["dtype"]], **dev)
        return st
    for k, which in (("A", "A"), ("A_scale", "A"), ("B", "B"), ("B_scale", "B"), ("gate", "B"), ("up", "B"), ("dC", "C"),
                     ("saved_gate", "C"), ("saved_up", "C"), ("saved_gate_scale", "C"), ("saved_up_scale", "C")):
        if k in inp:
            st[k] = _cut(case, inp[k], which)
    if own:
        import partial_sum_reduction_gb300 as s
        H = s.helpers
        mesh, sa, sb, sc, _ = LAYOUTS[case["layout"]]
        scaled = case["op"] in ("scaled", "scaled_grad")
        dt = "e4m3" if scaled else case["dtype"]
        out = case.get("out", "bf16") if scaled else dt
        st["plan"] = p = s.Plan(mesh, sa, sb, sc, case["rows"], case["J"], case["K"], dt, out)
        if case["op"] in ("scaled", "gated"):
            st["C"] = H.alloc(p, s.TENSOR_C)
        if case["op"] == "gated" and case["saved"] != "none":
            st["saved"] = H.gated_saved(p, case["saved"])
            if case["saved"] == "e4m3":
                st["values"] = [[torch.empty_like(c) for c in st["C"]] for _ in range(2)]
        if case["op"] == "scaled_grad":
            st["dA"], st["dB"] = (H.alloc(p, t, dtype=torch.bfloat16) for t in (s.TENSOR_A, s.TENSOR_B))
            st["workspace"] = H.scaled_workspace(p)
        if case["op"] == "gated_grad":
            e = case["saved"] == "e4m3"
            st["saved"] = s.GatedSaved(case["saved"], st["saved_gate"], st["saved_up"],
                                       st["saved_gate_scale"] if e else None, st["saved_up_scale"] if e else None)
            st["dA"] = H.alloc(p, s.TENSOR_A)
            st["dgate"], st["dup"] = H.alloc(p, s.TENSOR_B), H.alloc(p, s.TENSOR_B)
            st["workspace"] = H.gated_workspace(p)
    return st


# -------------------------------------------------------------- plain forms

def _plain_quantize(case, st):
    if case["way"] == "to":
        codes, scale = _to_8bit(st["x"].float(), case["block_rows"])
        return {"codes": codes, "scale": scale}
    return {"y": _from_8bit(st["codes"], st["scale"], case["block_rows"]).to(DTYPES[case["dtype"]])}


def _blocks_of(n, part=BLOCK):
    return -(-n // part)


def _plain_scaled_operands(case, st):
    T, J, K = case["rows"], case["J"], case["K"]
    A = _whole(case, st["A"], "A", T, J)
    As = _whole(case, st["A_scale"], "A", T, _blocks_of(J))
    B = _whole(case, st["B"], "B", J, K)
    Bs = _whole(case, st["B_scale"], "B", _blocks_of(J), _blocks_of(K))
    return _from_8bit(A, As, 1), _from_8bit(B, Bs, BLOCK)


def _plain_scaled(case, st):
    A, B = _plain_scaled_operands(case, st)
    return {"C": _cut(case, (A @ B).to(DTYPES[case["out"]]), "C")}


def _plain_scaled_grad(case, st):
    A, B = _plain_scaled_operands(case, st)
    dC = _whole(case, st["dC"], "C", case["rows"], case["K"]).float()
    q = _from_8bit(*_to_8bit(dC, 1), 1)  # dC in 8 bits, too, for the product with B
    return {"dA": _cut(case, (q @ B.T).to(torch.bfloat16), "A"), "dB": _cut(case, (A.T @ dC).to(torch.bfloat16), "B")}


def _plain_gated(case, st):
    T, J, K, dt = case["rows"], case["J"], case["K"], DTYPES[case["dtype"]]
    A = _whole(case, st["A"], "A", T, J).float()
    g = A @ _whole(case, st["gate"], "B", J, K).float()
    u = A @ _whole(case, st["up"], "B", J, K).float()
    out = {"C": _cut(case, (_act(case["act"], g)[0] * u).to(dt), "C")}
    if case["saved"] == "e4m3":
        g, u = _from_8bit(*_to_8bit(g, 1), 1), _from_8bit(*_to_8bit(u, 1), 1)
    if case["saved"] != "none":
        out["gate"], out["up"] = _cut(case, g.to(dt), "C"), _cut(case, u.to(dt), "C")
    return out


def _plain_gated_grad(case, st):
    T, J, K, dt = case["rows"], case["J"], case["K"], DTYPES[case["dtype"]]
    A = _whole(case, st["A"], "A", T, J).float()
    dC = _whole(case, st["dC"], "C", T, K).float()
    h = []
    for name in ("gate", "up"):
        v = _whole(case, st["saved_" + name], "C", T, K)
        if case["saved"] == "e4m3":
            h.append(_from_8bit(v, _whole(case, st["saved_" + name + "_scale"], "C", T, _blocks_of(K)), 1))
        else:
            h.append(v.float())
    a, slope = _act(case["act"], h[0])
    dg, du = dC * h[1] * slope, dC * a
    dA = dg @ _whole(case, st["gate"], "B", J, K).float().T + du @ _whole(case, st["up"], "B", J, K).float().T
    return {"dA": _cut(case, dA.to(dt), "A"), "dgate": _cut(case, (A.T @ dg).to(dt), "B"),
            "dup": _cut(case, (A.T @ du).to(dt), "B")}


# -------------------------------------------------------- the library's calls

def _own_quantize(case, st):
    import partial_sum_reduction_gb300 as s
    if case["way"] == "to":
        s.shmm_quantize(st["x"], st["codes"], st["scale"], block_rows=case["block_rows"])
        return {"codes": st["codes"], "scale": st["scale"]}
    s.shmm_dequantize(st["codes"], st["scale"], st["y"], block_rows=case["block_rows"])
    return {"y": st["y"]}


def _own_scaled(case, st):
    st["plan"].run_scaled(st["A"], st["A_scale"], st["B"], st["B_scale"], st["C"])
    return {"C": st["C"]}


def _own_scaled_grad(case, st):
    st["plan"].scaled_backward(st["dC"], st["A"], st["A_scale"], st["B"], st["B_scale"], st["dA"], st["dB"],
                               st["workspace"])
    return {"dA": st["dA"], "dB": st["dB"]}


def _own_gated(case, st):
    import partial_sum_reduction_gb300 as s
    saved = st.get("saved")
    st["plan"].gated_forward(st["A"], st["gate"], st["up"], st["C"], activation=case["act"], saved=saved)
    out = {"C": st["C"]}
    if case["saved"] == "e4m3":  # the values that the kept bytes stand for
        for codes, scales, values in ((saved.gate, saved.gate_scale, st["values"][0]),
                                      (saved.up, saved.up_scale, st["values"][1])):
            for c, sc, v in zip(codes, scales, values):
                s.shmm_dequantize(c, sc, v)
        out["gate"], out["up"] = st["values"]
    elif case["saved"] != "none":
        out["gate"], out["up"] = saved.gate, saved.up
    return out


def _own_gated_grad(case, st):
    st["plan"].gated_backward(st["dC"], st["A"], st["gate"], st["up"], st["saved"], st["dA"], st["dgate"], st["dup"],
                              st["workspace"], activation=case["act"])
    return {"dA": st["dA"], "dgate": st["dgate"], "dup": st["dup"]}


def run(state):
    case = state["case"]
    if own:
        return {"quantize": _own_quantize, "scaled": _own_scaled, "scaled_grad": _own_scaled_grad, "gated": _own_gated,
                "gated_grad": _own_gated_grad}[case["op"]](case, state)
    return {"quantize": _plain_quantize, "scaled": _plain_scaled, "scaled_grad": _plain_scaled_grad,
            "gated": _plain_gated, "gated_grad": _plain_gated_grad}[case["op"]](case, state)


# --------------------------------------------------------------------- work

def work(case):
    if case["op"] == "quantize":
        n, es = case["rows"] * case["cols"], 4 if case["dtype"] == "f32" else 2
        scales = 4 * _blocks_of(case["rows"], case["block_rows"]) * _blocks_of(case["cols"])
        return {"bytes": n * (es + 1) + scales, "flops": n * (3 if case["way"] == "to" else 1)}
    T, J, K = case["rows"], case["J"], case["K"]

    def held(which, rows, cols):  # elements over all ranks
        return sum((rows // r[1]) * (cols // c[1]) for r, c in _parts(case, which))

    a, b, c = T * J, J * K, T * K
    if case["op"] == "scaled":
        es = 4 if case["out"] == "f32" else 2
        return {"bytes": a + b + 4 * T * _blocks_of(J) + held("C", T, K) * es, "flops": 2 * T * J * K}
    if case["op"] == "scaled_grad":
        return {"bytes": a + b + 4 * T * _blocks_of(J) + 2 * c + 2 * held("A", T, J) + 2 * held("B", J, K),
                "flops": 4 * T * J * K}
    es = 4 if case["dtype"] == "f32" else 2
    saved = {"none": 0, "e4m3": 1 + 4 / BLOCK}.get(case["saved"], es)
    if case["op"] == "gated":
        return {"bytes": (a + 2 * b) * es + held("C", T, K) * (es + 2 * saved), "flops": 4 * T * J * K}
    return {"bytes": (a + 2 * b + c) * es + 2 * c * saved + (held("A", T, J) + 2 * held("B", J, K)) * es,
            "flops": 8 * T * J * K}


# -------------------------------------------------- the definition in 64 bits

def _round_e4m3(x):
    """Nearest e4m3 values of x (64 bits, magnitudes up to 448), ties to even:
    three fraction bits, exponents from -6."""
    e = torch.clamp(torch.frexp(x)[1] - 1, min=-6)
    step = _pow2(e - 3)
    return torch.round(x / step) * step


def _pow2(e):
    """2^e in 64 bits, by its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_8bit(x, block_rows):
    """(values with their scale, values without, scales) of the 8-bit form of x."""
    rows, cols = x.shape
    r = torch.arange(rows, device=x.device) // block_rows
    c = torch.arange(cols, device=x.device) // BLOCK
    rb, cb = int(r[-1]) + 1, int(c[-1]) + 1
    by_cols = torch.zeros(rows, cb, dtype=x.dtype, device=x.device)
    by_cols.scatter_reduce_(1, c.expand(rows, cols), x.abs(), "amax")
    amax = torch.zeros(rb, cb, dtype=x.dtype, device=x.device)
    amax.scatter_reduce_(0, r[:, None].expand(rows, cb), by_cols, "amax")
    e = torch.ceil(torch.log2(torch.clamp(amax, min=1e-300) / 448))
    e = torch.where(448 * _pow2(e - 1) >= amax, e - 1, e)  # log2 may be off at the borders
    e = torch.where(448 * _pow2(e) < amax, e + 1, e)
    scale = torch.where(amax > 0, _pow2(torch.clamp(e, min=-126)), torch.ones_like(amax))
    per = scale[r][:, c]
    plain = _round_e4m3(x / per)
    return plain * per, plain, scale


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "quantize":
        if case["way"] == "to":
            _, plain, scale = _exact_8bit(st["x"].double(), case["block_rows"])
            return {"codes": plain, "scale": scale}
        scale = st["scale"].double().repeat_interleave(case["block_rows"], 0)[:case["rows"]]
        return {"y": st["codes"].double() * scale.repeat_interleave(BLOCK, 1)[:, :case["cols"]]}
    if case["op"] in ("scaled", "scaled_grad"):
        A = st["A"].double() * st["A_scale"].double().repeat_interleave(BLOCK, 1)[:, :case["J"]]
        bs = st["B_scale"].double().repeat_interleave(BLOCK, 0)[:case["J"]]
        B = st["B"].double() * bs.repeat_interleave(BLOCK, 1)[:, :case["K"]]
        if case["op"] == "scaled":
            return {"C": _cut(case, torch.einsum("ij,jk->ik", A, B), "C")}
        dC = st["dC"].double()
        dA = torch.einsum("ik,jk->ij", _exact_8bit(dC, 1)[0], B)
        return {"dA": _cut(case, dA, "A"), "dB": _cut(case, torch.einsum("ij,ik->jk", A, dC), "B")}
    A, Wg, Wu = st["A"].double(), st["gate"].double(), st["up"].double()
    silu = case["act"] == "silu"
    # both activations are x times the logistic function of z(x)
    k0, k1 = (1.0, 0.0) if silu else (2 * math.sqrt(2 / math.pi), 2 * math.sqrt(2 / math.pi) * 0.044715)
    if case["op"] == "gated":
        g, u = torch.einsum("ij,jk->ik", A, Wg), torch.einsum("ij,jk->ik", A, Wu)
        out = {"C": _cut(case, g / (1 + torch.exp(-(k0 * g + k1 * g ** 3))) * u, "C")}
        if case["saved"] == "e4m3":
            g, u = _exact_8bit(g, 1)[0], _exact_8bit(u, 1)[0]
        if case["saved"] != "none":
            out["gate"], out["up"] = _cut(case, g, "C"), _cut(case, u, "C")
        return out
    g, u = st["saved_gate"].double(), st["saved_up"].double()
    if case["saved"] == "e4m3":
        g *= st["saved_gate_scale"].double().repeat_interleave(BLOCK, 1)[:, :case["K"]]
        u *= st["saved_up_scale"].double().repeat_interleave(BLOCK, 1)[:, :case["K"]]
    z = k0 * g + k1 * g ** 3
    s, t = 1 / (1 + torch.exp(-z)), 1 / (1 + torch.exp(z))
    dC = st["dC"].double()
    dg = dC * u * (s + g * s * t * (k0 + 3 * k1 * g * g))
    du = dC * g * s
    dA = torch.einsum("ik,jk->ij", dg, Wg) + torch.einsum("ik,jk->ij", du, Wu)
    return {"dA": _cut(case, dA, "A"), "dgate": _cut(case, torch.einsum("ij,ik->jk", A, dg), "B"),
            "dup": _cut(case, torch.einsum("ij,ik->jk", A, du), "B")}
