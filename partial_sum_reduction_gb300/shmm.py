"""ctypes binding of libshmm (include/shmm.h): the same entry points, with
argument marshalling only.  Every step of the sharded matmul runs in the
library's CUDA kernels; there is no CPU or PyTorch fallback, and importing a
missing library raises.

Meshes and shardings may be given as Python values or as strings:
  mesh   [("X", 4), ("Y", 2)]  or  "{X:4,Y:2}"
  spec   (("X",), ("Y",))  or  "P('X','Y')"  or  "P(('X','Y'),None)"  or
         the subscript form "I_X,J_Y" ("Sharded matmuls and collectives on a
         torus", Notation: A[I_X, J_Y] is P('X', 'Y'); A[I_XY, J] is
         P(('X', 'Y'), None)).
Tensors are lists of per-rank CUDA tensors, indexed by rank id, each a dense
row-major buffer holding exactly that rank's box (Plan.rank_box).
"""
from __future__ import annotations

import ctypes
import os
import re
from array import array
from typing import List, Optional, Sequence, Tuple

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
# SHMM_CHECKED=1 selects the bounds-checked build (build.build(checked=True)):
# the same kernels with every global index compared with its buffer's extent.
LIB_PATH = os.path.join(HERE, "libshmm_checked.so" if os.environ.get("SHMM_CHECKED") == "1" else "libshmm.so")

MAX_AXES = 8
MAX_RANKS = 256

# status codes
OK, ERR_INVALID_SPEC, ERR_ILLEGAL_OUTPUT, ERR_SHAPE, ERR_DTYPE, ERR_NULL, ERR_ALIGN, ERR_CUDA, \
    ERR_TIMEOUT, ERR_NOMEM, ERR_UNSUPPORTED, ERR_INJECTED, ERR_BOUNDS = range(13)
F32, BF16, E4M3 = 0, 1, 2
SCALE_BLOCK = 128
SILU, GELU_TANH = 0, 1
FLAG_FUSED, FLAG_GELU, FLAG_TREE, FLAG_PARTIAL_OUT_DTYPE, FLAG_SIMT = 0x1, 0x2, 0x4, 0x8, 0x10
FLAG_RANK_ORDER = 0x20
TENSOR_A, TENSOR_B, TENSOR_C, TENSOR_P, TENSOR_A_LOCAL, TENSOR_B_LOCAL, TENSOR_C_REDUCED = range(7)
COLL_NONE, COLL_REDUCE_SCATTER, COLL_ALL_REDUCE = range(3)
COLLECTIVE_NAMES = {COLL_NONE: "none", COLL_REDUCE_SCATTER: "reduce_scatter",
                    COLL_ALL_REDUCE: "all_reduce"}
DTYPE_CODES = {"f32": F32, "bf16": BF16, "e4m3": E4M3}
ACTIVATIONS = {"silu": SILU, "gelu": GELU_TANH}


class shmm_mesh_t(ctypes.Structure):
    _fields_ = [("naxes", ctypes.c_int), ("name", (ctypes.c_char * 8) * MAX_AXES),
                ("size", ctypes.c_int * MAX_AXES)]


class shmm_spec_t(ctypes.Structure):
    _fields_ = [("naxes", ctypes.c_int * 2), ("axes", (ctypes.c_int * MAX_AXES) * 2)]


class shmm_plan_info_t(ctypes.Structure):
    _fields_ = [("case_id", ctypes.c_int), ("collective", ctypes.c_int),
                ("scatter_dim", ctypes.c_int), ("nranks", ctypes.c_int),
                ("group_size", ctypes.c_int), ("ngroups", ctypes.c_int),
                ("gather_A_size", ctypes.c_int), ("gather_B_size", ctypes.c_int),
                ("gather_C_size", ctypes.c_int), ("in_dtype", ctypes.c_int),
                ("out_dtype", ctypes.c_int), ("partial_dtype", ctypes.c_int),
                ("flags", ctypes.c_uint32), ("tensor_core", ctypes.c_int), ("fused", ctypes.c_int),
                ("local_I", ctypes.c_int64), ("local_J", ctypes.c_int64), ("local_K", ctypes.c_int64),
                ("flops_per_rank", ctypes.c_int64), ("payload_operand_ag", ctypes.c_int64),
                ("payload_reduce_scatter", ctypes.c_int64), ("payload_result_ag", ctypes.c_int64),
                ("workspace_bytes", ctypes.c_size_t), ("fused_gather", ctypes.c_int)]


class shmm_device_model_t(ctypes.Structure):
    _fields_ = [("flops_per_s", ctypes.c_double), ("bytes_per_s", ctypes.c_double)]


class shmm_operand_choice_t(ctypes.Structure):
    _fields_ = [("choice", ctypes.c_int), ("gather_compute_bound", ctypes.c_int),
                ("bytes_gather", ctypes.c_double), ("bytes_reduce", ctypes.c_double),
                ("t_gather", ctypes.c_double), ("t_reduce", ctypes.c_double)]


class shmm_gated_saved_t(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("gate", ctypes.c_void_p), ("up", ctypes.c_void_p),
                ("gate_scale", ctypes.c_void_p), ("up_scale", ctypes.c_void_p)]


class ShmmError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("%s: %s" % (_status_name(status), message))
        self.status = status


EXPORTS = ["shmm_plan", "shmm_plan_destroy", "shmm_plan_query", "shmm_plan_rank_box",
           "shmm_plan_set_sm_limit", "shmm_plan_group", "shmm_workspace_size", "shmm_local_matmul", "shmm_reduce_scatter",
           "shmm_all_reduce", "shmm_all_gather", "shmm_run", "shmm_sync_status", "shmm_last_error",
           "shmm_status_string", "shmm_version", "shmm_kernel_launches", "shmm_run_static_workspace",
           "shmm_selftest_wait_timeout", "shmm_choose_operand", "shmm_reshard", "shmm_layernorm",
           "shmm_layernorm_all_gather", "shmm_run_host", "shmm_bounds_checked", "shmm_run_batch",
           "shmm_layernorm_forward", "shmm_layernorm_backward_workspace_size", "shmm_layernorm_backward",
           "shmm_layernorm_all_gather_forward", "shmm_layernorm_all_gather_backward",
           "shmm_adapters_forward", "shmm_adapters_workspace_size", "shmm_adapters_backward",
           "shmm_quantize", "shmm_dequantize", "shmm_run_scaled", "shmm_scaled_backward_workspace_size",
           "shmm_scaled_backward", "shmm_gated_forward", "shmm_gated_backward_workspace_size",
           "shmm_gated_backward"]

_lib = None


def lib():
    """The loaded libshmm.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("%s is not built (%s); run partial_sum_reduction_gb300.build.build(%s)"
                               % (os.path.basename(LIB_PATH), LIB_PATH,
                                  "checked=True" if LIB_PATH.endswith("_checked.so") else ""))
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        PP = ctypes.POINTER(ctypes.c_void_p)
        st = ctypes.c_int
        L.shmm_plan.argtypes = [ctypes.POINTER(shmm_mesh_t), ctypes.POINTER(shmm_spec_t),
                                ctypes.POINTER(shmm_spec_t), ctypes.POINTER(shmm_spec_t),
                                ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                                ctypes.c_int, ctypes.c_uint32, ctypes.POINTER(P)]
        L.shmm_plan_destroy.argtypes = [P]
        L.shmm_plan_set_sm_limit.argtypes = [P, ctypes.c_int]
        L.shmm_plan_query.argtypes = [P, ctypes.POINTER(shmm_plan_info_t)]
        L.shmm_plan_rank_box.argtypes = [P, ctypes.c_int, ctypes.c_int,
                                         ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int64)]
        L.shmm_plan_group.argtypes = [P, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
        L.shmm_workspace_size.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
        L.shmm_local_matmul.argtypes = [P, PP, PP, PP, P]
        L.shmm_reduce_scatter.argtypes = [P, PP, PP, P]
        L.shmm_all_reduce.argtypes = [P, PP, PP, P]
        L.shmm_all_gather.argtypes = [P, ctypes.c_int, PP, PP, P]
        L.shmm_run.argtypes = [P, PP, PP, PP, P, ctypes.c_size_t, P]
        L.shmm_run_static_workspace.argtypes = [P, PP, PP, PP, P]
        L.shmm_run_batch.argtypes = [ctypes.c_int, PP, ctypes.POINTER(PP), ctypes.POINTER(PP), ctypes.POINTER(PP),
                                     PP, ctypes.POINTER(ctypes.c_size_t), P]
        L.shmm_run_host.argtypes = [P, P, P, P, PP, PP, PP, P, ctypes.c_size_t, P]
        L.shmm_sync_status.argtypes = [P]
        L.shmm_selftest_wait_timeout.argtypes = [ctypes.c_uint64, P]
        L.shmm_layernorm.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, P, P, P, ctypes.c_float, P, P]
        L.shmm_layernorm_all_gather.argtypes = [P, PP, P, P, ctypes.c_float, PP, P]
        L.shmm_layernorm_forward.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, P, P, P, P, ctypes.c_float,
                                             P, P, P, P, P]
        L.shmm_layernorm_backward_workspace_size.argtypes = [ctypes.c_int64, ctypes.c_int64,
                                                             ctypes.POINTER(ctypes.c_size_t)]
        L.shmm_layernorm_backward.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, P, P, P, P, P, P, P, P, P,
                                              P, ctypes.c_size_t, P]
        L.shmm_layernorm_all_gather_forward.argtypes = [P, P, P, P, ctypes.c_float, P, P, P, P]
        L.shmm_layernorm_all_gather_backward.argtypes = [P, ctypes.c_int, P, P, P, P, P, P, P, P, P, ctypes.c_size_t,
                                                         P]
        L.shmm_adapters_forward.argtypes = [P, ctypes.c_int, ctypes.c_int, P, P, P, P, P, P, P, P, P]
        L.shmm_adapters_workspace_size.argtypes = [P, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)]
        L.shmm_adapters_backward.argtypes = [P, ctypes.c_int, ctypes.c_int, P, P, P, P, P, P, P, P, P, P, P, P,
                                             ctypes.c_size_t, P]
        L.shmm_quantize.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int, P, P, P, P]
        L.shmm_dequantize.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int, P, P, P, P]
        L.shmm_run_scaled.argtypes = [P, P, P, P, P, P, P]
        L.shmm_scaled_backward_workspace_size.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
        L.shmm_scaled_backward.argtypes = [P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        L.shmm_gated_forward.argtypes = [P, ctypes.c_int, P, P, P, P, ctypes.POINTER(shmm_gated_saved_t), P]
        L.shmm_gated_backward_workspace_size.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
        L.shmm_gated_backward.argtypes = [P, ctypes.c_int, P, P, P, P, ctypes.POINTER(shmm_gated_saved_t), P, P, P, P, P,
                                          ctypes.c_size_t, P]
        L.shmm_reshard.argtypes = [ctypes.POINTER(shmm_mesh_t), ctypes.POINTER(shmm_spec_t),
                                   ctypes.POINTER(shmm_spec_t), ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                                   PP, PP, P]
        L.shmm_choose_operand.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                                          ctypes.c_int, ctypes.POINTER(shmm_device_model_t),
                                          ctypes.POINTER(shmm_operand_choice_t)]
        L.shmm_last_error.restype = ctypes.c_char_p
        L.shmm_status_string.argtypes = [ctypes.c_int]
        L.shmm_status_string.restype = ctypes.c_char_p
        L.shmm_kernel_launches.restype = ctypes.c_uint64
        for f in EXPORTS:
            if f not in ("shmm_last_error", "shmm_status_string", "shmm_kernel_launches"):
                getattr(L, f).restype = st
        _lib = L
    return _lib


def _status_name(s: int) -> str:
    try:
        return lib().shmm_status_string(s).decode()
    except Exception:  # library unavailable while formatting an error
        return "status %d" % s


def _check(status: int) -> None:
    if status != OK:
        raise ShmmError(status, lib().shmm_last_error().decode())


# ------------------------------------------------------------- parsing (D6)

def parse_mesh(mesh) -> List[Tuple[str, int]]:
    """'{X:4,Y:2}' or [('X',4),('Y',2)] -> [('X',4),('Y',2)]."""
    if isinstance(mesh, str):
        body = mesh.strip().strip("{}")
        out = []
        for part in body.split(","):
            if part.strip():
                name, size = part.split(":")
                out.append((name.strip().strip("'\""), int(size)))
        return out
    return [(str(n), int(s)) for n, s in mesh]


def parse_spec(spec) -> Tuple[Tuple[str, ...], Tuple[str, ...]]:
    """Sharding of a 2-D array in any of the accepted forms -> per-dim axis
    tuples, first axis major."""
    if isinstance(spec, str):
        s = spec.strip()
        if s.startswith("P(") and s.endswith(")"):
            inner = s[2:-1].strip()
            if not inner:
                return ((), ())
            dims = []
            depth, cur = 0, ""
            for ch in inner + ",":
                if ch == "," and depth == 0:
                    dims.append(cur.strip())
                    cur = ""
                    continue
                depth += ch == "("
                depth -= ch == ")"
                cur += ch
            parsed = []
            for d in dims:
                if d in ("None", ""):
                    parsed.append(())
                else:
                    parsed.append(tuple(re.findall(r"['\"]([^'\"]+)['\"]", d)))
            while len(parsed) < 2:
                parsed.append(())
            if len(parsed) != 2:
                raise ValueError("a 2-D PartitionSpec has at most two entries: %r" % spec)
            return parsed[0], parsed[1]
        dims = [d.strip() for d in s.strip("[]").split(",")]
        if len(dims) != 2:
            raise ValueError("expected two dims in %r" % spec)
        return tuple(tuple(d.split("_", 1)[1]) if "_" in d else () for d in dims)
    a, b = spec
    return tuple(a), tuple(b)


def _mesh_struct(mesh) -> shmm_mesh_t:
    m = shmm_mesh_t()
    axes = parse_mesh(mesh)
    if len(axes) > MAX_AXES:
        raise ValueError("at most %d mesh axes" % MAX_AXES)
    m.naxes = len(axes)
    for i, (n, s) in enumerate(axes):
        enc = n.encode()
        if len(enc) >= 8:
            raise ValueError("axis name %r longer than 7 bytes" % n)
        m.name[i].value = enc
        m.size[i] = s
    return m


def _spec_struct(mesh, spec) -> shmm_spec_t:
    names = [n for n, _ in parse_mesh(mesh)]
    s = shmm_spec_t()
    for d, axes in enumerate(parse_spec(spec)):
        if len(axes) > MAX_AXES:
            raise ValueError("too many axes on one dim")
        s.naxes[d] = len(axes)
        for i, a in enumerate(axes):
            s.axes[d][i] = names.index(a) if a in names else 99  # 99: rejected by the planner
    return s


# --------------------------------------------------------------- marshalling

def _ptr_array(tensors: Sequence, what: str) -> ctypes.Array:
    arr = (ctypes.c_void_p * len(tensors))()
    for i, t in enumerate(tensors):
        if t is None:
            arr[i] = None
        elif isinstance(t, int):
            arr[i] = t
        else:
            arr[i] = t.data_ptr()
    return arr


# The current stream's handle without a Stream object around it (3 us less per
# call where this torch has it).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(stream, dev: Optional[int] = None) -> Optional[int]:
    """dev: the current device, where the caller has asked for it."""
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device() if dev is None else dev)
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


TORCH_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def _refuse(t, what: str, shape, dtype):
    """Raises ValueError with what is wrong with tensor t (see _tensor)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % what)
    if t.dtype is not dtype:
        raise ValueError("%s is %s, expected %s" % (what, t.dtype, dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (what, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be dense (row-major contiguous)" % what)
    raise ValueError("%s is on %s, the current device is cuda:%d" % (what, t.device, torch.cuda.current_device()))


def _device() -> int:
    """The current device; without a GPU, a number that no tensor is on (a CPU
    tensor is on -1)."""
    try:
        return torch.cuda.current_device()
    except (RuntimeError, AssertionError):
        return -2


def _tensor(t, what: str, shape, dtype, dev: int) -> int:
    """Address of a dense CUDA tensor of device `dev` (the current one) with
    the given shape and dtype; anything else is refused before the library
    sees it."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _refuse(t, what, shape, dtype)


def _tensors(ts, what: str, shapes, dtype, dev: int) -> array:
    """Addresses of dense tensors (see _tensor), one per shape, as an array of
    pointers; its _at() goes to the library (a ctypes array costs ten times
    as much to make)."""
    if len(ts) != len(shapes):
        raise ValueError("%s: %d tensors, the plan has %d ranks" % (what, len(ts), len(shapes)))
    ptrs = array("Q")
    for t, shape in zip(ts, shapes):
        try:
            if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
                ptrs.append(t.data_ptr())
                continue
        except AttributeError:
            pass
        _refuse(t, "%s[%d]" % (what, len(ptrs)), shape, dtype)
    return ptrs


def _at(ptrs: Optional[array]) -> Optional[int]:
    return None if ptrs is None else ptrs.buffer_info()[0]


def _rows_dtype(x, what: str = "x"):
    """(rows, cols, torch dtype, dtype code) of a 2-D fp32 or bf16 tensor."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("%s must be a 2-D CUDA tensor" % what)
    (rows, cols), dtype = x.shape, x.dtype
    if dtype is torch.bfloat16:
        return rows, cols, dtype, BF16
    if dtype is torch.float32:
        return rows, cols, dtype, F32
    raise ValueError("%s is %s, expected torch.float32 or torch.bfloat16" % (what, dtype))


def _dense(x, what: str, dev: int) -> int:
    """Address of a tensor of known shape and type: dense, on device `dev`."""
    if x.get_device() == dev and x.is_contiguous():
        return x.data_ptr()
    return _refuse(x, what, x.shape, x.dtype)


def _workspace(ws, dev: int):
    """(address, bytes) of a workspace tensor, or of none."""
    if ws is None:
        return None, 0
    if not isinstance(ws, torch.Tensor) or ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("workspace must be a dense CUDA tensor of the current device")
    return ws.data_ptr(), ws.nbytes


def scale_shape(rows: int, cols: int, block_rows: int = 1) -> Tuple[int, int]:
    """Shape of the scales of a [rows, cols] array in 8 bits."""
    return (-(-rows // block_rows), -(-cols // SCALE_BLOCK))


def _activation(name: str) -> int:
    if name not in ACTIVATIONS:
        raise ValueError("activation %r, expected one of %s" % (name, sorted(ACTIVATIONS)))
    return ACTIVATIONS[name]


class GatedSaved:
    """What gated_forward keeps for gated_backward: per-rank lists of the two
    projections' values before the activation, in the plan's type or (dtype
    "e4m3") in 8 bits with a scale for each 128 columns of a row."""

    def __init__(self, dtype: str, gate, up, gate_scale=None, up_scale=None):
        self.dtype, self.gate, self.up, self.gate_scale, self.up_scale = dtype, gate, up, gate_scale, up_scale


class Plan:
    """A shmm_plan_t handle (freed on garbage collection or close())."""

    def __init__(self, mesh, spec_A, spec_B, spec_C, I: int, J: int, K: int, in_dtype: str = "bf16",
                 out_dtype: str = "bf16", flags: int = 0):
        self.mesh = parse_mesh(mesh)
        self.spec_A, self.spec_B, self.spec_C = parse_spec(spec_A), parse_spec(spec_B), parse_spec(spec_C)
        self.shape = (int(I), int(J), int(K))
        self.in_dtype, self.out_dtype, self.flags = in_dtype, out_dtype, int(flags)
        h = ctypes.c_void_p()
        m = _mesh_struct(self.mesh)
        sa, sb, sc = (_spec_struct(self.mesh, s) for s in (self.spec_A, self.spec_B, self.spec_C))
        _check(lib().shmm_plan(ctypes.byref(m), ctypes.byref(sa), ctypes.byref(sb), ctypes.byref(sc),
                               int(I), int(J), int(K), DTYPE_CODES[in_dtype], DTYPE_CODES[out_dtype],
                               int(flags), ctypes.byref(h)))
        self._h = h
        self._box_shapes = {}
        self.info = self.query()
        self.nranks = self.info.nranks

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            lib().shmm_plan_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    def set_sm_limit(self, max_sms: int):
        """Caps the SMs this plan's tensor-core GEMM launches occupy (0: all)."""
        _check(lib().shmm_plan_set_sm_limit(self._h, int(max_sms)))

    def query(self) -> shmm_plan_info_t:
        info = shmm_plan_info_t()
        _check(lib().shmm_plan_query(self._h, ctypes.byref(info)))
        return info

    def rank_box(self, tensor: int, rank: int):
        off = (ctypes.c_int64 * 2)()
        ext = (ctypes.c_int64 * 2)()
        _check(lib().shmm_plan_rank_box(self._h, tensor, rank, off, ext))
        return (off[0], off[1]), (ext[0], ext[1])

    def group(self, rank: int) -> List[int]:
        out = (ctypes.c_int * self.info.group_size)()
        _check(lib().shmm_plan_group(self._h, rank, out))
        return list(out)

    def workspace_size(self) -> int:
        n = ctypes.c_size_t()
        _check(lib().shmm_workspace_size(self._h, ctypes.byref(n)))
        return n.value

    # ---- device work ----
    def local_matmul(self, A_r, B_r, P_r, stream=None):
        _check(lib().shmm_local_matmul(self._h, _ptr_array(A_r, "A"), _ptr_array(B_r, "B"),
                                       _ptr_array(P_r, "P"), _stream_handle(stream)))

    def reduce_scatter(self, P_r, C_r, stream=None):
        _check(lib().shmm_reduce_scatter(self._h, _ptr_array(P_r, "P"), _ptr_array(C_r, "C"),
                                         _stream_handle(stream)))

    def all_reduce(self, P_r, C_r, stream=None):
        _check(lib().shmm_all_reduce(self._h, _ptr_array(P_r, "P"), _ptr_array(C_r, "C"),
                                     _stream_handle(stream)))

    def all_gather(self, tensor: int, shard_r, full_r, stream=None):
        _check(lib().shmm_all_gather(self._h, tensor, _ptr_array(shard_r, "shard"),
                                     _ptr_array(full_r, "full"), _stream_handle(stream)))

    def run(self, A_r, B_r, C_r, workspace=None, stream=None):
        ws_ptr = None if workspace is None else (workspace if isinstance(workspace, int) else workspace.data_ptr())
        ws_bytes = 0 if workspace is None else (
            self.workspace_size() if isinstance(workspace, int) else workspace.numel() * workspace.element_size())
        _check(lib().shmm_run(self._h, _ptr_array(A_r, "A"), _ptr_array(B_r, "B"), _ptr_array(C_r, "C"),
                              ws_ptr, ws_bytes, _stream_handle(stream)))

    def layernorm_all_gather(self, shard_r, gamma, beta, full_r, eps: float = 1e-5, stream=None):
        """Layer-normalise the row-owned result blocks and all-gather them
        (sequence parallelism's LayerNorm then AllGather, in one pass)."""
        _check(lib().shmm_layernorm_all_gather(self._h, _ptr_array(shard_r, "shard"), gamma.data_ptr(),
                                               beta.data_ptr(), float(eps), _ptr_array(full_r, "full"),
                                               _stream_handle(stream)))

    def _shapes(self, tensor: int):
        """Per-rank box extents of `tensor` (kept: they never change)."""
        got = self._box_shapes.get(tensor)
        if got is None:
            got = self._box_shapes[tensor] = [self.rank_box(tensor, r)[1] for r in range(self.nranks)]
        return got

    def _gathered(self):
        """(owner blocks' shapes, their row counts as shapes, (columns,))."""
        got = self._box_shapes.get("rows")
        if got is None:
            block = self._shapes(TENSOR_C_REDUCED)
            got = self._box_shapes["rows"] = (block, [(e[0],) for e in block], (block[0][1],))
        return got

    def layernorm_all_gather_forward(self, shard_r, gamma, beta, full_r, mean_r, rstd_r, eps: float = 1e-5,
                                     stream=None):
        """layernorm_all_gather that also leaves each owner block's row
        statistics in mean_r, rstd_r (one fp32 [block rows] tensor per rank),
        for layernorm_all_gather_backward."""
        dt, f32, dev = TORCH_DTYPES[self.out_dtype], torch.float32, _device()
        block, rows, cols = self._gathered()
        shard = _tensors(shard_r, "shard", block, dt, dev)
        full = _tensors(full_r, "full", self._shapes(TENSOR_C), dt, dev)
        mean, rstd = _tensors(mean_r, "mean", rows, f32, dev), _tensors(rstd_r, "rstd", rows, f32, dev)
        _check(lib().shmm_layernorm_all_gather_forward(
            self._h, _at(shard), _tensor(gamma, "gamma", cols, f32, dev), _tensor(beta, "beta", cols, f32, dev), eps,
            _at(full), _at(mean), _at(rstd), _stream_handle(stream)))

    def layernorm_all_gather_backward(self, dfull_r, shard_r, mean_r, rstd_r, gamma, dshard_r, dgamma, dbeta,
                                      workspace, stream=None):
        """Gradient of layernorm_all_gather_forward: every member's gradient
        of the gathered rows (fp32, or the plan's output dtype), reduced to
        the rows' owners and taken through the normalisation in one pass
        (see include/shmm.h).  workspace: helpers.layernorm_workspace of the
        rows of every rank's block."""
        dt, f32, dev = TORCH_DTYPES[self.out_dtype], torch.float32, _device()
        block, rows, cols = self._gathered()
        gdt = f32 if len(dfull_r) and getattr(dfull_r[0], "dtype", None) is f32 else dt
        ws, ws_bytes = _workspace(workspace, dev)
        dfull = _tensors(dfull_r, "dfull", self._shapes(TENSOR_C), gdt, dev)
        shard, dshard = _tensors(shard_r, "shard", block, dt, dev), _tensors(dshard_r, "dshard", block, dt, dev)
        mean, rstd = _tensors(mean_r, "mean", rows, f32, dev), _tensors(rstd_r, "rstd", rows, f32, dev)
        _check(lib().shmm_layernorm_all_gather_backward(
            self._h, F32 if gdt is f32 else BF16, _at(dfull), _at(shard), _at(mean), _at(rstd),
            _tensor(gamma, "gamma", cols, f32, dev), _at(dshard), _tensor(dgamma, "dgamma", cols, f32, dev),
            _tensor(dbeta, "dbeta", cols, f32, dev), ws, ws_bytes, _stream_handle(stream)))

    def adapters_workspace_size(self, n_adapters: int, rank: int) -> int:
        n = ctypes.c_size_t()
        _check(lib().shmm_adapters_workspace_size(self._h, int(n_adapters), int(rank), ctypes.byref(n)))
        return n.value

    def _adapters(self, row_adapter, down, up, scale, dev):
        """(n, rank, addresses) of the adapters' factors, checked."""
        dt, (I, J, K) = TORCH_DTYPES[self.in_dtype], self.shape
        if not isinstance(down, torch.Tensor) or down.dim() != 3:
            raise ValueError("down must be a CUDA tensor [adapters, rank, J]")
        n, rank, _ = down.shape
        return n, rank, (_tensor(row_adapter, "row_adapter", (I,), torch.int32, dev),
                         _tensor(down, "down", (n, rank, J), dt, dev), _tensor(up, "up", (n, rank, K), dt, dev),
                         None if scale is None else _tensor(scale, "scale", (n,), torch.float32, dev))

    def adapters_forward(self, A_r, row_adapter, down, up, scale, base_r, C_r, low, stream=None):
        """Low-rank adapters beside the plan's product: C = base + scale[a]
        (A . down[a]^T) . up[a] for the rows of adapter a (see
        include/shmm.h).  down [n, rank, J], up [n, rank, K]; scale [n] or
        None; base_r: per-rank tensors (C_r itself included) or None."""
        dev = _device()
        n, rank, ptrs = self._adapters(row_adapter, down, up, scale, dev)
        dt, box = TORCH_DTYPES[self.out_dtype], self._shapes(TENSOR_C)
        A = _tensors(A_r, "A", self._shapes(TENSOR_A), TORCH_DTYPES[self.in_dtype], dev)
        base = None if base_r is None else _tensors(base_r, "base", box, dt, dev)
        C = _tensors(C_r, "C", box, dt, dev)
        _check(lib().shmm_adapters_forward(
            self._h, n, rank, _at(A), *ptrs, _at(base), _at(C),
            _tensor(low, "low", (self.shape[0], rank), torch.float32, dev), _stream_handle(stream)))

    def adapters_backward(self, dC_r, A_r, row_adapter, down, up, scale, low, base_r, dA_r, ddown, dup, workspace,
                          stream=None):
        """Gradient of adapters_forward: dA (+ base), and every adapter's
        ddown, dup in fp32 (see include/shmm.h).  workspace:
        helpers.adapters_workspace."""
        dev = _device()
        n, rank, ptrs = self._adapters(row_adapter, down, up, scale, dev)
        dt, box, f32 = TORCH_DTYPES[self.in_dtype], self._shapes(TENSOR_A), torch.float32
        I, J, K = self.shape
        ws, ws_bytes = _workspace(workspace, dev)
        dC = _tensors(dC_r, "dC", self._shapes(TENSOR_C), TORCH_DTYPES[self.out_dtype], dev)
        A, dA = _tensors(A_r, "A", box, dt, dev), _tensors(dA_r, "dA", box, dt, dev)
        base = None if base_r is None else _tensors(base_r, "base", box, dt, dev)
        _check(lib().shmm_adapters_backward(
            self._h, n, rank, _at(dC), _at(A), *ptrs, _tensor(low, "low", (I, rank), f32, dev), _at(base), _at(dA),
            _tensor(ddown, "ddown", (n, rank, J), f32, dev), _tensor(dup, "dup", (n, rank, K), f32, dev), ws, ws_bytes,
            _stream_handle(stream)))

    def _scale_shapes(self, tensor: int, block_rows: int = 1):
        """Per-rank shapes of the scales of `tensor`'s boxes in 8 bits (kept)."""
        key = (tensor, block_rows)
        got = self._box_shapes.get(key)
        if got is None:
            got = self._box_shapes[key] = [scale_shape(e[0], e[1], block_rows) for e in self._shapes(tensor)]
        return got

    def _scaled(self, A_r, A_scale_r, B_r, B_scale_r, dev):
        f32, e4m3 = torch.float32, TORCH_DTYPES[self.in_dtype]
        return (_tensors(A_r, "A", self._shapes(TENSOR_A), e4m3, dev),
                _tensors(A_scale_r, "A_scale", self._scale_shapes(TENSOR_A), f32, dev),
                _tensors(B_r, "B", self._shapes(TENSOR_B), e4m3, dev),
                _tensors(B_scale_r, "B_scale", self._scale_shapes(TENSOR_B, SCALE_BLOCK), f32, dev))

    def run_scaled(self, A_r, A_scale_r, B_r, B_scale_r, C_r, stream=None):
        """The sharded matmul of 8-bit operands (a plan of in_dtype "e4m3"):
        A with a scale for each 128 columns of a row, B one for each 128 x
        128 values, every rank's box quantised on its own (see
        include/shmm.h)."""
        dev = _device()
        ops = self._scaled(A_r, A_scale_r, B_r, B_scale_r, dev)
        C = _tensors(C_r, "C", self._shapes(TENSOR_C), TORCH_DTYPES[self.out_dtype], dev)
        _check(lib().shmm_run_scaled(self._h, *map(_at, ops), _at(C), _stream_handle(stream)))

    def scaled_workspace_size(self) -> int:
        n = ctypes.c_size_t()
        _check(lib().shmm_scaled_backward_workspace_size(self._h, ctypes.byref(n)))
        return n.value

    def scaled_backward(self, dC_r, A_r, A_scale_r, B_r, B_scale_r, dA_r, dB_r, workspace, stream=None):
        """Gradient of run_scaled: dA = Q(dC) . B^T with dC in 8 bits too,
        dB = A^T . dC from the 8-bit A that was kept (see include/shmm.h);
        dA_r or dB_r may be None.  workspace: helpers.scaled_workspace."""
        dev, bf16 = _device(), torch.bfloat16
        ops = self._scaled(A_r, A_scale_r, B_r, B_scale_r, dev)
        ws, ws_bytes = _workspace(workspace, dev)
        dC = _tensors(dC_r, "dC", self._shapes(TENSOR_C), TORCH_DTYPES[self.out_dtype], dev)
        dA = None if dA_r is None else _tensors(dA_r, "dA", self._shapes(TENSOR_A), bf16, dev)
        dB = None if dB_r is None else _tensors(dB_r, "dB", self._shapes(TENSOR_B), bf16, dev)
        _check(lib().shmm_scaled_backward(self._h, _at(dC), *map(_at, ops), _at(dA), _at(dB), ws, ws_bytes,
                                          _stream_handle(stream)))

    def _saved(self, saved, dev):
        """(structure, what it points to) of a GatedSaved, checked."""
        if saved is None:
            return None, None
        box, f32 = self._shapes(TENSOR_C), torch.float32
        if saved.dtype not in TORCH_DTYPES:
            raise ValueError("saved.dtype is %r, expected one of %s" % (saved.dtype, sorted(TORCH_DTYPES)))
        dt = TORCH_DTYPES[saved.dtype]
        keep = [_tensors(saved.gate, "saved.gate", box, dt, dev), _tensors(saved.up, "saved.up", box, dt, dev)]
        if saved.dtype == "e4m3":
            if saved.gate_scale is None or saved.up_scale is None:
                raise ValueError("saved values in 8 bits need gate_scale and up_scale")
            scales = self._scale_shapes(TENSOR_C)
            keep += [_tensors(saved.gate_scale, "saved.gate_scale", scales, f32, dev),
                     _tensors(saved.up_scale, "saved.up_scale", scales, f32, dev)]
        return shmm_gated_saved_t(DTYPE_CODES[saved.dtype], *[_at(k) for k in keep]), keep

    def _gated(self, A_r, gate_r, up_r, dev):
        dt, box = TORCH_DTYPES[self.in_dtype], self._shapes(TENSOR_B)
        return (_tensors(A_r, "A", self._shapes(TENSOR_A), dt, dev), _tensors(gate_r, "gate", box, dt, dev),
                _tensors(up_r, "up", box, dt, dev))

    def gated_forward(self, A_r, gate_r, up_r, C_r, activation: str = "silu", saved: "Optional[GatedSaved]" = None,
                      stream=None):
        """The gated first half of an MLP block, C = act(A . gate) * (A .
        up), in one pass; `saved` (helpers.gated_saved) receives both
        projections for gated_backward (see include/shmm.h).  activation:
        "silu" or "gelu" (tanh form)."""
        dev = _device()
        ops = self._gated(A_r, gate_r, up_r, dev)
        C = _tensors(C_r, "C", self._shapes(TENSOR_C), TORCH_DTYPES[self.out_dtype], dev)
        st, keep = self._saved(saved, dev)
        _check(lib().shmm_gated_forward(self._h, _activation(activation), *map(_at, ops), _at(C),
                                        None if st is None else ctypes.byref(st), _stream_handle(stream)))

    def gated_workspace_size(self) -> int:
        n = ctypes.c_size_t()
        _check(lib().shmm_gated_backward_workspace_size(self._h, ctypes.byref(n)))
        return n.value

    def gated_backward(self, dC_r, A_r, gate_r, up_r, saved, dA_r, dgate_r, dup_r, workspace, activation: str = "silu",
                       C_r=None, stream=None):
        """Gradient of gated_forward from what it saved: dA, dgate, dup, and C
        again where C_r is given (see include/shmm.h).  dA_r, or dgate_r and
        dup_r, may be None.  workspace: helpers.gated_workspace."""
        dev = _device()
        dt, B = TORCH_DTYPES[self.in_dtype], self._shapes(TENSOR_B)
        ops = self._gated(A_r, gate_r, up_r, dev)
        st, keep = self._saved(saved, dev)
        ws, ws_bytes = _workspace(workspace, dev)
        dC = _tensors(dC_r, "dC", self._shapes(TENSOR_C), TORCH_DTYPES[self.out_dtype], dev)
        outs = [None if t is None else _tensors(t, what, box, dt, dev)
                for t, what, box in ((dA_r, "dA", self._shapes(TENSOR_A)), (dgate_r, "dgate", B), (dup_r, "dup", B),
                                     (C_r, "C", self._shapes(TENSOR_C)))]
        _check(lib().shmm_gated_backward(self._h, _activation(activation), _at(dC), *map(_at, ops),
                                         None if st is None else ctypes.byref(st), *map(_at, outs), ws, ws_bytes,
                                         _stream_handle(stream)))

    def run_host(self, A_host, B_host, C_host, A_r, B_r, C_r, workspace=None, stream=None):
        """shmm_run_host: global A [I,J], B [J,K] (CPU tensors, pinned for
        overlap, or None when A_r / B_r already hold the shards) in, global C
        [I,K] (a CPU tensor, or None) out, through the ranks' device buffers."""
        def host_ptr(t, shape, what):
            if t is None:
                return None
            if (not hasattr(t, "data_ptr") or t.device.type != "cpu" or not t.is_contiguous()
                    or tuple(t.shape) != shape):
                raise ValueError("%s_host must be a contiguous CPU tensor of shape %s" % (what, shape))
            return t.data_ptr()
        ws_ptr = None if workspace is None else (workspace if isinstance(workspace, int) else workspace.data_ptr())
        ws_bytes = 0 if workspace is None else (
            self.workspace_size() if isinstance(workspace, int) else workspace.numel() * workspace.element_size())
        I, J, K = self.shape
        _check(lib().shmm_run_host(self._h, host_ptr(A_host, (I, J), "A"), host_ptr(B_host, (J, K), "B"),
                                   host_ptr(C_host, (I, K), "C"),
                                   _ptr_array(A_r, "A"), _ptr_array(B_r, "B"), _ptr_array(C_r, "C"),
                                   ws_ptr, ws_bytes, _stream_handle(stream)))

    def run_static_workspace(self, A_r, B_r, C_r, stream=None):
        """shmm_run on the library's fixed 64 MiB device workspace, for
        callers that cannot allocate device memory (see include/shmm.h)."""
        _check(lib().shmm_run_static_workspace(self._h, _ptr_array(A_r, "A"), _ptr_array(B_r, "B"),
                                               _ptr_array(C_r, "C"), _stream_handle(stream)))


# Same names as the C-ABI, for callers that prefer the flat interface.
def shmm_plan(mesh, spec_A, spec_B, spec_C, I, J, K, in_dtype="bf16", out_dtype="bf16", flags=0) -> Plan:
    return Plan(mesh, spec_A, spec_B, spec_C, I, J, K, in_dtype, out_dtype, flags)


def shmm_plan_destroy(plan: Plan) -> None:
    plan.close()


def shmm_plan_set_sm_limit(plan: Plan, max_sms: int) -> None:
    plan.set_sm_limit(max_sms)


def shmm_plan_query(plan: Plan) -> shmm_plan_info_t:
    return plan.query()


def shmm_plan_rank_box(plan: Plan, tensor: int, rank: int):
    return plan.rank_box(tensor, rank)


def shmm_workspace_size(plan: Plan) -> int:
    return plan.workspace_size()


def shmm_local_matmul(plan: Plan, A_r, B_r, P_r, stream=None):
    plan.local_matmul(A_r, B_r, P_r, stream)


def shmm_reduce_scatter(plan: Plan, P_r, C_r, stream=None):
    plan.reduce_scatter(P_r, C_r, stream)


def shmm_all_reduce(plan: Plan, P_r, C_r, stream=None):
    plan.all_reduce(P_r, C_r, stream)


def shmm_all_gather(plan: Plan, tensor: int, shard_r, full_r, stream=None):
    plan.all_gather(tensor, shard_r, full_r, stream)


def shmm_run(plan: Plan, A_r, B_r, C_r, workspace=None, stream=None):
    plan.run(A_r, B_r, C_r, workspace, stream)


def shmm_run_batch(plans: Sequence[Plan], A_r, B_r, C_r, workspaces=None, stream=None):
    """Independent sharded matmuls whose local GEMMs share launches (see
    include/shmm.h).  A_r, B_r, C_r: per plan, its list of per-rank tensors;
    workspaces: per plan, a workspace tensor or None."""
    n = len(plans)
    keep = [[_ptr_array(t, w) for t in lists] for lists, w in ((A_r, "A"), (B_r, "B"), (C_r, "C"))]
    PP = ctypes.POINTER(ctypes.c_void_p)
    tables = [(PP * n)(*[ctypes.cast(a, PP) for a in arrs]) for arrs in keep]
    ws = list(workspaces) if workspaces is not None else [None] * n
    ws_ptr = (ctypes.c_void_p * n)(*[None if w is None else w.data_ptr() for w in ws])
    ws_bytes = (ctypes.c_size_t * n)(*[0 if w is None else w.numel() * w.element_size() for w in ws])
    handles = (ctypes.c_void_p * n)(*[p.handle.value for p in plans])
    _check(lib().shmm_run_batch(n, handles, tables[0], tables[1], tables[2], ws_ptr, ws_bytes,
                                _stream_handle(stream)))


def shmm_run_host(plan: Plan, A_host, B_host, C_host, A_r, B_r, C_r, workspace=None, stream=None):
    plan.run_host(A_host, B_host, C_host, A_r, B_r, C_r, workspace, stream)


def shmm_run_static_workspace(plan: Plan, A_r, B_r, C_r, stream=None):
    plan.run_static_workspace(A_r, B_r, C_r, stream)


STATIC_WORKSPACE_BYTES = 64 << 20


def shmm_sync_status(stream=None) -> None:
    _check(lib().shmm_sync_status(_stream_handle(stream)))


def shmm_layernorm(x, gamma, beta, y, eps: float = 1e-5, stream=None):
    """Row-wise layer normalisation of a 2-D CUDA tensor x into y."""
    rows, cols = x.shape
    dt = {"torch.float32": "f32", "torch.bfloat16": "bf16"}[str(x.dtype)]
    _check(lib().shmm_layernorm(int(rows), int(cols), DTYPE_CODES[dt], x.data_ptr(), gamma.data_ptr(),
                                beta.data_ptr(), float(eps), y.data_ptr(), _stream_handle(stream)))


def shmm_layernorm_forward(x, gamma, beta, y, mean, rstd, residual=None, total=None, eps: float = 1e-5, stream=None):
    """Row-wise layer normalisation of x (+ residual, the rounded sum kept in
    total) into y, with the rows' statistics for shmm_layernorm_backward
    (see include/shmm.h)."""
    rows, cols, dt, code = _rows_dtype(x)
    f32, shape, dev = torch.float32, (rows, cols), _device()
    _check(lib().shmm_layernorm_forward(
        rows, cols, code, _tensor(x, "x", shape, dt, dev),
        None if residual is None else _tensor(residual, "residual", shape, dt, dev),
        _tensor(gamma, "gamma", (cols,), f32, dev), _tensor(beta, "beta", (cols,), f32, dev), eps,
        None if total is None else _tensor(total, "total", shape, dt, dev), _tensor(y, "y", shape, dt, dev),
        _tensor(mean, "mean", (rows,), f32, dev), _tensor(rstd, "rstd", (rows,), f32, dev), _stream_handle(stream)))


def shmm_layernorm_backward_workspace_size(rows: int, cols: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().shmm_layernorm_backward_workspace_size(int(rows), int(cols), ctypes.byref(n)))
    return n.value


def shmm_layernorm_backward(dy, x, mean, rstd, gamma, dx, dgamma, dbeta, workspace, residual_grad=None, stream=None):
    """Gradient of shmm_layernorm_forward: dx (+ residual_grad), dgamma,
    dbeta (see include/shmm.h).  workspace: helpers.layernorm_workspace."""
    rows, cols, dt, code = _rows_dtype(x)
    f32, shape, dev = torch.float32, (rows, cols), _device()
    ws, ws_bytes = _workspace(workspace, dev)
    _check(lib().shmm_layernorm_backward(
        rows, cols, code, _tensor(dy, "dy", shape, dt, dev), _tensor(x, "x", shape, dt, dev),
        _tensor(mean, "mean", (rows,), f32, dev), _tensor(rstd, "rstd", (rows,), f32, dev),
        _tensor(gamma, "gamma", (cols,), f32, dev),
        None if residual_grad is None else _tensor(residual_grad, "residual_grad", shape, dt, dev),
        _tensor(dx, "dx", shape, dt, dev), _tensor(dgamma, "dgamma", (cols,), f32, dev),
        _tensor(dbeta, "dbeta", (cols,), f32, dev), ws, ws_bytes, _stream_handle(stream)))


def shmm_quantize(x, codes, scales, block_rows: int = 1, stream=None):
    """x [rows, cols] in 8 bits: codes (float8_e4m3fn) and fp32 scales, one for
    each 128 columns of a row (block_rows=1) or 128 x 128 values (128); see
    include/shmm.h.  scale_shape gives the scales' shape."""
    rows, cols, dt, code = _rows_dtype(x)
    dev = _device()
    if block_rows not in (1, SCALE_BLOCK):
        raise ValueError("block_rows must be 1 or %d" % SCALE_BLOCK)
    _check(lib().shmm_quantize(
        rows, cols, code, block_rows, _dense(x, "x", dev),
        _tensor(codes, "codes", (rows, cols), TORCH_DTYPES["e4m3"], dev),
        _tensor(scales, "scales", scale_shape(rows, cols, block_rows), torch.float32, dev),
        _stream_handle(stream, dev)))


def shmm_dequantize(codes, scales, y, block_rows: int = 1, stream=None):
    """The way back: y (fp32 or bf16) = codes * scales."""
    rows, cols, dt, code = _rows_dtype(y, "y")
    dev = _device()
    if block_rows not in (1, SCALE_BLOCK):
        raise ValueError("block_rows must be 1 or %d" % SCALE_BLOCK)
    _check(lib().shmm_dequantize(
        rows, cols, code, block_rows, _tensor(codes, "codes", (rows, cols), TORCH_DTYPES["e4m3"], dev),
        _tensor(scales, "scales", scale_shape(rows, cols, block_rows), torch.float32, dev),
        _dense(y, "y", dev), _stream_handle(stream, dev)))


def shmm_reshard(mesh, spec_from, spec_to, rows: int, cols: int, dtype: str, src_r, dst_r, stream=None):
    """All-to-all / reshard of a [rows, cols] array between two shardings
    (see include/shmm.h); src_r, dst_r are per-rank tensors (or pointers)."""
    m = _mesh_struct(mesh)
    a, b = _spec_struct(mesh, spec_from), _spec_struct(mesh, spec_to)
    _check(lib().shmm_reshard(ctypes.byref(m), ctypes.byref(a), ctypes.byref(b), int(rows), int(cols),
                              DTYPE_CODES[dtype], _ptr_array(src_r, "src"), _ptr_array(dst_r, "dst"),
                              _stream_handle(stream)))


def shmm_choose_operand(B: int, D: int, F: int, axis_size: int, flops_per_s: float, bytes_per_s: float,
                        elem_bytes: int = 2) -> shmm_operand_choice_t:
    """Which operand of X[B,D].W[D_X,F] to move: 1 = all-gather W, 2 = keep W
    sharded and all-reduce the [B,F] partials (see include/shmm.h)."""
    dev = shmm_device_model_t(float(flops_per_s), float(bytes_per_s))
    out = shmm_operand_choice_t()
    _check(lib().shmm_choose_operand(int(B), int(D), int(F), int(axis_size), int(elem_bytes),
                                     ctypes.byref(dev), ctypes.byref(out)))
    return out


def shmm_selftest_wait_timeout(limit_cycles: int, stream=None) -> None:
    _check(lib().shmm_selftest_wait_timeout(int(limit_cycles), _stream_handle(stream)))


def shmm_version() -> int:
    return lib().shmm_version()


def shmm_bounds_checked() -> bool:
    """True if the loaded library is the bounds-checked build."""
    return bool(lib().shmm_bounds_checked())


def shmm_kernel_launches() -> int:
    return lib().shmm_kernel_launches()
