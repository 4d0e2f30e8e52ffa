"""Plain 64-bit forms of the 8-bit and gated operators, layouts and inputs,
shared by their tests.  Nothing here calls the library's kernels."""
import math

import torch

BLOCK = 128
E4M3 = torch.float8_e4m3fn
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # of a value rounded to nearest, relative

# name -> (mesh, spec of A, of B, of C): all four cases, one rank, copies
LAYOUTS = {
    "whole": ("{X:1}", "I,J", "J,K", "I,K"),
    "rows": ("{X:4}", "I_X,J", "J,K", "I_X,K"),
    "columns": ("{X:4}", "I,J", "J,K_X", "I,K_X"),
    "grid": ("{X:2,Y:2}", "I_X,J", "J,K_Y", "I_X,K_Y"),
    "gather_A": ("{X:4}", "I,J_X", "J,K", "I,K"),
    "gather_B": ("{X:2,Y:2}", "I_X,J", "J_Y,K", "I_X,K"),
    "all_reduce": ("{X:2,Y:2}", "I_X,J_Y", "J_Y,K", "I_X,K"),
    "scatter_rows": ("{X:2,Y:2}", "I_X,J_Y", "J_Y,K", "I_XY,K"),
    "scatter_columns": ("{X:2,Y:2}", "I_X,J_Y", "J_Y,K", "I_X,K_Y"),
    "case_4": ("{X:2}", "I_X,J", "J,K_X", "I_X,K"),
    "copies": ("{X:2,Y:2}", "I_X,J", "J,K", "I_X,K"),
}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def blocks(x, block_rows):
    rows, cols = x.shape
    rb, cb = -(-rows // block_rows), -(-cols // BLOCK)
    p = torch.zeros(rb * block_rows, cb * BLOCK, dtype=x.dtype, device=x.device)
    p[:rows, :cols] = x
    return p.reshape(rb, block_rows, cb, BLOCK)


def quantized(x, block_rows=1):
    """(values as e4m3, fp32 scales) of x by the definition, in 64 bits."""
    v = blocks(x.double(), block_rows)
    finite = torch.isfinite(v)
    amax = torch.where(finite, v, torch.zeros_like(v)).abs().amax(dim=(1, 3))
    m, p = torch.frexp(amax)
    e = torch.clamp(p.long() - 9 + (m > 0.875).long(), min=-126)
    scale = torch.where(amax > 0, ((e + 1023) << 52).view(torch.float64), torch.ones_like(amax))
    q = v / scale[:, None, :, None]
    step = ((torch.clamp(torch.frexp(q)[1].long() - 1, min=-6) - 3 + 1023) << 52).view(torch.float64)
    q = torch.where(finite, torch.round(q / step) * step, torch.full_like(q, math.nan))
    codes = q.reshape(v.shape[0] * block_rows, -1)[:x.shape[0], :x.shape[1]].contiguous().float().to(E4M3)
    return codes, scale.float()


def restored(codes, scale, block_rows=1):
    """What the blocks stand for, in 64 bits."""
    s = scale.double().repeat_interleave(block_rows, 0)[:codes.shape[0]]
    return codes.double() * s.repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def gate_act(name, x):
    """(value, slope) of the activation in 64 bits."""
    if name == "silu":
        s = torch.sigmoid(x)
        return x * s, s + x * s * (1 - s)
    # (1 + tanh v) / 2 is the logistic function of 2 v, which does not cancel where v is far below zero
    c = 2 * math.sqrt(2 / math.pi)
    p = torch.sigmoid(c * (x + 0.044715 * x ** 3))
    q = torch.sigmoid(-c * (x + 0.044715 * x ** 3))
    return x * p, p + x * p * q * c * (1 + 3 * 0.044715 * x * x)


def box(plan, tensor, rank, full):
    (o0, o1), (e0, e1) = plan.rank_box(tensor, rank)
    return full[o0:o0 + e0, o1:o1 + e1]


def cut(plan, tensor, full):
    return [box(plan, tensor, r, full).clone(memory_format=torch.contiguous_format) for r in range(plan.nranks)]


def gathered(plan, tensor, parts, rows, cols, dtype=torch.float64):
    """The whole array from the ranks' boxes."""
    out = torch.full((rows, cols), math.nan, dtype=dtype, device="cuda")
    for r, t in enumerate(parts):
        box(plan, tensor, r, out).copy_(t.to(dtype))
    return out


def assert_ranks(plan, tensor, parts, want, bound, what):
    """Every rank's box is within `bound` (elementwise) of the whole array."""
    for r, t in enumerate(parts):
        w, b = box(plan, tensor, r, want), box(plan, tensor, r, bound)
        off = (t.double() - w).abs()
        ok = off <= b
        assert bool(ok.all()), "%s[%d]: %d of %d values off, worst by %.3g (allowed %.3g)" % (
            what, r, int((~ok).sum()), off.numel(), float((off - b).max()), float(b.flatten()[(off - b).argmax()]))


def sum_error(terms, size):
    """Bound on the rounding of a sum of `terms` products in fp32 whose
    magnitudes add up to `size`: every addition rounds (or, in the tensor
    cores, truncates) a partial sum no larger than `size` by at most 2^-23 of
    it.  A matrix instruction adds at least 16 products at once; the CUDA
    cores add 256 one by one and then those sums."""
    per = min(terms, 256) + terms / 16 + 4
    return per * 2.0 ** -23 * size
