"""8-bit blocks: shmm_quantize and shmm_dequantize against the definition in
64 bits.  Values and scales are powers of two apart, so both are compared bit
for bit."""
import ctypes
import math

import pytest
import torch

import partial_sum_reduction_gb300 as s
from partial_sum_reduction_gb300 import shmm as m
from block_util import DTYPES, E4M3, gen, normal, quantized, restored

SIZES = [(1, 1), (1, 128), (3, 129), (16, 4096), (127, 257), (128, 1024), (129, 1031), (301, 96), (5, 8200), (1030, 8),
         (2, 70000)]


def values(seed, rows, cols, dtype):
    """Activations with features far larger than the rest, zeros and a block of nothing."""
    g = gen(seed)
    x = normal(g, rows, cols) * torch.exp(3 * normal(g, rows, 1))
    x[:, ::7] *= 40.0
    x[rows // 2] = 0.0
    return x.to(DTYPES[dtype])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_to_8_bits_and_back(rows, cols, block_rows, dtype):
    x = values(rows * 7 + cols, rows, cols, dtype)
    codes, scales = s.helpers.quantize(x, block_rows)
    want, want_scales = quantized(x, block_rows)
    assert torch.equal(scales, want_scales)
    assert torch.equal(codes.view(torch.uint8), want.view(torch.uint8))
    y = torch.empty_like(x)
    s.shmm_dequantize(codes, scales, y, block_rows)
    assert torch.equal(y.double(), restored(want, want_scales, block_rows))  # exact: a power of two
    # half a step of e4m3, 2^-4, or half of its smallest step, 2^-10 times the scale
    small = restored(torch.ones_like(codes.float()).to(E4M3), scales, block_rows) * 2.0 ** -10
    assert bool(((y.double() - x.double()).abs() <= torch.maximum(x.double().abs() * 2.0 ** -4, small)).all())


@pytest.mark.gpu
@pytest.mark.parametrize("block_rows", [1, 128])
def test_any_scale_is_taken_back(block_rows):
    g = gen(3)
    codes = normal(g, 200, 300).mul(50).to(E4M3)
    scales = torch.rand(*s.scale_shape(200, 300, block_rows), generator=g, device="cuda") * 3
    for dt in (torch.float32, torch.bfloat16):
        y = torch.empty(200, 300, dtype=dt, device="cuda")
        s.shmm_dequantize(codes, scales, y, block_rows)
        per = scales.repeat_interleave(block_rows, 0)[:200].repeat_interleave(128, 1)[:, :300]
        assert torch.equal(y, (codes.float() * per).to(dt))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_extremes(dtype, block_rows):
    """Infinities and NaN stay in their places, as NaN; the type's largest and
    smallest values, and borders of the scale."""
    dt = DTYPES[dtype]
    x = torch.zeros(140, 400, device="cuda", dtype=dt)
    x[0, 3], x[0, 5], x[0, 7], x[0, 9] = math.inf, -math.inf, math.nan, 2.5
    x[1, :4] = torch.finfo(dt).max
    x[2, 0], x[2, 1] = torch.finfo(dt).tiny, -torch.finfo(dt).tiny
    x[3, 130] = torch.finfo(dt).smallest_normal / 4  # below the smallest scale's values
    for i, e in enumerate(range(-20, 20)):
        x[4 + i, 0], x[4 + i, 1] = 448.0 * 2.0 ** e, 1.0
        x[60 + i, 200], x[60 + i, 201] = 450.0 * 2.0 ** e, -447.0 * 2.0 ** e
    x[129, 399] = math.inf  # a block with nothing finite but zeros
    codes, scales = s.helpers.quantize(x, block_rows)
    want, want_scales = quantized(x, block_rows)
    assert torch.equal(scales, want_scales) and bool(torch.isfinite(scales).all())
    a, b = codes.float(), want.float()
    assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.isnan(a), ~torch.isfinite(x.float()))
    assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


@pytest.mark.gpu
def test_nothing_to_do_and_what_is_left_alone():
    whole = torch.full((64, 256), 7.0, device="cuda").to(E4M3)
    x = normal(gen(1), 40, 256)
    s.shmm_quantize(x, whole[:40], torch.empty(40, 2, device="cuda"))
    assert bool((whole[40:].float() == 7.0).all())
    for shape in ((0, 5), (5, 0)):
        e = torch.empty(shape, device="cuda")
        s.shmm_quantize(e, e.to(E4M3), torch.empty(*s.scale_shape(*shape), device="cuda"))
        s.shmm_dequantize(e.to(E4M3), torch.empty(*s.scale_shape(*shape), device="cuda"), e)


@pytest.mark.gpu
def test_on_another_stream_and_in_a_graph():
    x = normal(gen(5), 256, 512).bfloat16()
    codes, scales = s.helpers.quantize(x)
    c2, s2, y = torch.empty_like(codes), torch.empty_like(scales), torch.empty_like(x)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        s.shmm_quantize(x, c2, s2)
    torch.cuda.synchronize()
    assert torch.equal(c2.view(torch.uint8), codes.view(torch.uint8)) and torch.equal(s2, scales)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.shmm_quantize(x, c2, s2)
        s.shmm_dequantize(c2, s2, y)
    x.copy_(normal(gen(6), 256, 512).bfloat16())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y.double(), restored(*quantized(x)))


# ---- refusals: no GPU is reached ------------------------------------------

def _call(name, rows=4, cols=256, dtype=m.BF16, block_rows=1, a=4096, codes=1 << 20, scales=1 << 24):
    lib = s.lib()
    if name == "shmm_quantize":
        return lib.shmm_quantize(rows, cols, dtype, block_rows, a, codes, scales, None)
    return lib.shmm_dequantize(rows, cols, dtype, block_rows, codes, scales, a, None)


@pytest.mark.parametrize("name", ["shmm_quantize", "shmm_dequantize"])
@pytest.mark.parametrize("args,status", [
    (dict(rows=-1), m.ERR_SHAPE), (dict(cols=-1), m.ERR_SHAPE), (dict(rows=1 << 31), m.ERR_SHAPE),
    (dict(cols=1 << 26), m.ERR_SHAPE), (dict(block_rows=64), m.ERR_SHAPE), (dict(block_rows=0), m.ERR_SHAPE),
    (dict(dtype=m.E4M3), m.ERR_DTYPE), (dict(dtype=9), m.ERR_DTYPE), (dict(a=None), m.ERR_NULL),
    (dict(codes=None), m.ERR_NULL), (dict(scales=None), m.ERR_NULL), (dict(a=4104), m.ERR_ALIGN),
    (dict(codes=(1 << 20) + 8), m.ERR_ALIGN), (dict(scales=(1 << 24) + 2), m.ERR_ALIGN),
    (dict(codes=4096 + 16), m.ERR_UNSUPPORTED), (dict(rows=0, a=None, codes=None, scales=None), m.OK),
    (dict(cols=0, a=None, codes=None, scales=None), m.OK)])
def test_refusals(name, args, status):
    assert _call(name, **args) == status


def test_scales_over_the_values_are_refused():
    assert _call("shmm_quantize", scales=4096 + 64) == m.ERR_UNSUPPORTED
    assert _call("shmm_dequantize", scales=4096 + 64) == m.ERR_UNSUPPORTED
    assert _call("shmm_quantize", scales=(1 << 20) + 1020) == m.ERR_UNSUPPORTED


def test_injected_failure(monkeypatch):
    monkeypatch.setenv("SHMM_INJECT_FAIL", "shmm_quantize,shmm_dequantize")
    assert _call("shmm_quantize") == m.ERR_INJECTED and _call("shmm_dequantize") == m.ERR_INJECTED


def test_the_binding_checks_tensors():
    x = torch.zeros(4, 256)
    with pytest.raises(ValueError):
        s.shmm_quantize(x, x.to(E4M3), torch.zeros(4, 2))
    with pytest.raises(ValueError):
        s.shmm_quantize(x, x.to(E4M3), torch.zeros(4, 2), block_rows=64)
    with pytest.raises(ValueError):
        s.shmm_dequantize(x.to(E4M3), torch.zeros(4, 2), torch.zeros(4, 256, dtype=torch.float16))
    assert ctypes.sizeof(ctypes.c_void_p) == 8
