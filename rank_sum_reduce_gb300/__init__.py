"""Python binding of libcar (include/car.h): argument marshalling only.

Every ``car_*`` function here has the name and arguments of the C entry point
and returns its status code; all work runs in libcar's CUDA kernels.  Device
buffers are passed as integer addresses (``tensor.data_ptr()``), streams as
integer handles (``torch.cuda.current_stream().cuda_stream``).

``Car`` is a small convenience wrapper over the same calls for torch tensors.
There is no CPU fallback: importing the binding without a built libcar.so
raises ImportError.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libcar.so")

CAR_BF16, CAR_FP16, CAR_FP32 = 0, 1, 2
CAR_OK, CAR_ERR_ARG, CAR_ERR_ALIGN, CAR_ERR_SIZE, CAR_ERR_CUDA, CAR_ERR_STALE_FLAG, CAR_ERR_HANDLE, CAR_ERR_TIMEOUT = \
    range(8)
CAR_FUSED_AUTO, CAR_FUSED_ROWS, CAR_FUSED_PIPELINE = 0, 1, 2
CAR_SCALE_ROW, CAR_SCALE_GROUP128, CAR_SCALE_MX32, CAR_SCALE_STATIC = 0, 1, 2, 3
SCALE_CODE = {"row": CAR_SCALE_ROW, "group128": CAR_SCALE_GROUP128, "mx32": CAR_SCALE_MX32, "static": CAR_SCALE_STATIC}
CAR_STALE_LIST_MAX = 65536
CAR_MAX_ROW_BYTES = 64 * 1024
DTYPE_CODE = {"bf16": CAR_BF16, "fp16": CAR_FP16, "fp32": CAR_FP32}
ELEM_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
STATUS_NAME = {CAR_OK: "CAR_OK", CAR_ERR_ARG: "CAR_ERR_ARG", CAR_ERR_ALIGN: "CAR_ERR_ALIGN",
               CAR_ERR_SIZE: "CAR_ERR_SIZE", CAR_ERR_CUDA: "CAR_ERR_CUDA",
               CAR_ERR_STALE_FLAG: "CAR_ERR_STALE_FLAG", CAR_ERR_HANDLE: "CAR_ERR_HANDLE",
               CAR_ERR_TIMEOUT: "CAR_ERR_TIMEOUT"}


class car_stale_report(ctypes.Structure):
    _fields_ = [("n_stale", ctypes.c_uint64), ("n_listed", ctypes.c_uint32), ("cap", ctypes.c_uint32),
                ("entries", ctypes.POINTER(ctypes.c_uint32 * 2))]


class car_dropout(ctypes.Structure):
    _fields_ = [("p", ctypes.c_float), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64), ("offset_dev", ctypes.c_void_p)]


class car_branch(ctypes.Structure):
    _fields_ = [("norm_weight", ctypes.c_void_p), ("norm_eps", ctypes.c_float), ("gate", ctypes.c_void_p),
                ("gate_rows", ctypes.c_int64), ("residual_scale", ctypes.c_float), ("dropout", ctypes.POINTER(car_dropout))]


class car_branch_grads(ctypes.Structure):
    _fields_ = [("dx", ctypes.c_void_p), ("dresidual", ctypes.c_void_p), ("dweight", ctypes.c_void_p),
                ("dnorm_weight", ctypes.c_void_p), ("dgate", ctypes.c_void_p)]


if not os.path.exists(LIB_PATH):
    raise ImportError(f"libcar.so is not built ({LIB_PATH}); run `python -c 'import __graft_entry__ as g; "
                      "g.build()'` or `python rank_sum_reduce_gb300/build.py`")

_lib = ctypes.CDLL(LIB_PATH)

_vp = ctypes.c_void_p
_pvp = ctypes.c_void_p  # a pointer table: the bytes that _table packs
_ctx_pp = ctypes.POINTER(ctypes.c_void_p)
_SIGS = {
    "car_create": (ctypes.c_int, [ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, _ctx_pp]),
    "car_destroy": (ctypes.c_int, [_vp]),
    "car_reduce": (ctypes.c_int, [_vp, _pvp, _vp, _vp]),
    "car_reduce_two_shot": (ctypes.c_int, [_vp, _pvp, _vp, _vp]),
    "car_reduce_residual_rmsnorm": (ctypes.c_int, [_vp, _pvp, _vp, _vp, ctypes.c_float, _vp, _vp, _vp, _vp]),
    "car_reduce_residual_rmsnorm_quant": (ctypes.c_int, [_vp, _pvp, _vp, _vp, ctypes.c_float, ctypes.c_int, _vp, _vp,
                                                         _vp, _vp, _vp, _vp]),
    "car_quant_scale_bytes": (ctypes.c_size_t, [_vp, ctypes.c_int]),
    "car_reduce_residual_rmsnorm_backward": (ctypes.c_int, [_vp, _pvp, _vp, _vp, ctypes.c_float, _vp, _vp, _vp, _vp,
                                                            _vp]),
    "car_backward_workspace_bytes": (ctypes.c_size_t, [_vp]),
    "car_reduce_dropout": (ctypes.c_int, [_vp, _pvp, _vp, _vp, _vp]),
    "car_reduce_branch_residual_rmsnorm": (ctypes.c_int, [_vp, _pvp, _vp, _vp, _vp, ctypes.c_float, _vp, _vp, _vp, _vp]),
    "car_reduce_branch_residual_rmsnorm_backward": (ctypes.c_int, [_vp, _pvp, _vp, _vp, _vp, _vp, ctypes.c_float, _vp, _vp,
                                                                   _vp, _vp]),
    "car_branch_workspace_bytes": (ctypes.c_size_t, [_vp, ctypes.POINTER(car_branch)]),
    "car_grads_create": (ctypes.c_int, [ctypes.c_int, ctypes.c_int64, ctypes.POINTER(ctypes.c_int64),
                                        ctypes.POINTER(ctypes.c_int), _pvp, _pvp, _ctx_pp]),
    "car_grads_destroy": (ctypes.c_int, [_vp]),
    "car_grads_reduce": (ctypes.c_int, [_vp, ctypes.c_float, _vp, _vp]),
    "car_grads_clip": (ctypes.c_int, [_vp, _vp, ctypes.c_float, _vp, _vp]),
    "car_grads_reduce_clip": (ctypes.c_int, [_vp, ctypes.c_float, ctypes.c_float, _vp, _vp]),
    "car_grads_reduce_clip_once": (ctypes.c_int, [_vp, ctypes.c_float, ctypes.c_float, _vp, _vp]),
    "car_ll128_wire_bytes": (ctypes.c_size_t, [_vp]),
    "car_ll128_encode": (ctypes.c_int, [_vp, _vp, ctypes.c_uint64, _vp, _vp]),
    "car_ll128_decode_reduce": (ctypes.c_int, [_vp, _pvp, ctypes.c_uint64, ctypes.c_int, _vp, _vp]),
    "car_ll128_report": (ctypes.c_int, [_vp, ctypes.POINTER(car_stale_report)]),
    "car_ll_wire_bytes": (ctypes.c_size_t, [_vp]),
    "car_ll_encode": (ctypes.c_int, [_vp, _vp, ctypes.c_uint32, _vp, _vp]),
    "car_ll_decode_reduce": (ctypes.c_int, [_vp, _pvp, ctypes.c_uint32, ctypes.c_int, _vp, _vp]),
    "car_ll_report": (ctypes.c_int, [_vp, ctypes.POINTER(car_stale_report)]),
    "car_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "car_last_error": (ctypes.c_char_p, []),
    "car_tune_fused": (ctypes.c_int, [_vp, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    "car_sync": (ctypes.c_int, [_vp, _vp]),
    "car_test_delay_partial": (ctypes.c_int, [_vp, ctypes.c_uint64, ctypes.c_int, ctypes.c_int64, ctypes.c_uint64]),
    "car_lamport_buffer_bytes": (ctypes.c_size_t, [_vp]),
    "car_lamport_init": (ctypes.c_int, [_vp, _vp, _vp]),
    "car_lamport_push": (ctypes.c_int, [_vp, _vp, ctypes.c_int, ctypes.c_uint64, _vp, _vp]),
    "car_lamport_reduce_residual_rmsnorm": (ctypes.c_int, [_vp, _vp, ctypes.c_uint64, ctypes.c_int, _vp, _vp,
                                                           ctypes.c_float, _vp, _vp, _vp, _vp]),
    "car_lamport_report": (ctypes.c_int, [_vp, ctypes.POINTER(car_stale_report)]),
    "car_ll128_decode_reduce_noalloc": (ctypes.c_int, [ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                                                       _pvp, ctypes.c_uint64, ctypes.c_int, _vp, _vp,
                                                       ctypes.c_uint32, _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = tuple(_SIGS)


def lib():
    return _lib


@functools.lru_cache(maxsize=64)
def _packer(n: int):
    return struct.Struct(f"{n}P").pack


def _table(ptrs):
    """Host array of device pointers, as bytes (a call reads it before it returns)."""
    try:
        return _packer(len(ptrs))(*ptrs)
    except struct.error:  # not plain ints in range: as ctypes takes them
        return bytes((ctypes.c_void_p * len(ptrs))(*[int(p) for p in ptrs]))


# ---------------------------------------------------------------------------
# 1:1 wrappers of the C entry points
# ---------------------------------------------------------------------------
def car_create(W: int, M: int, N: int, dtype: int):
    """Returns (status, handle); handle is an int address or None."""
    out = ctypes.c_void_p()
    st = _lib.car_create(W, M, N, dtype, ctypes.byref(out))
    return st, out.value


def car_destroy(h) -> int:
    return _lib.car_destroy(h)


def car_reduce(h, inputs, ar_out: int, stream: int = 0) -> int:
    return _lib.car_reduce(h, _table(inputs) if inputs is not None else None, ar_out, stream)


def car_reduce_two_shot(h, inputs, ar_out: int, stream: int = 0) -> int:
    return _lib.car_reduce_two_shot(h, _table(inputs) if inputs is not None else None, ar_out, stream)


def car_reduce_residual_rmsnorm(h, inputs, residual: int, weight: int, eps: float, residual_out: int,
                                norm_out: int, ar_out: int | None, stream: int = 0) -> int:
    return _lib.car_reduce_residual_rmsnorm(h, _table(inputs) if inputs is not None else None, residual, weight,
                                            eps, residual_out, norm_out, ar_out, stream)


def car_reduce_residual_rmsnorm_quant(h, inputs, residual: int, weight: int, eps: float, kind: int, residual_out: int,
                                      q_out: int, scales: int, norm_out: int | None, ar_out: int | None,
                                      stream: int = 0) -> int:
    return _lib.car_reduce_residual_rmsnorm_quant(h, _table(inputs) if inputs is not None else None, residual, weight,
                                                  eps, kind, residual_out, q_out, scales, norm_out, ar_out, stream)


def car_quant_scale_bytes(h, kind: int) -> int:
    return int(_lib.car_quant_scale_bytes(h, kind))


def car_reduce_residual_rmsnorm_backward(h, dnorm, residual_out: int, weight: int, eps: float,
                                         dresidual_out: int | None, dx: int, dweight: int | None,
                                         workspace: int | None, stream: int = 0) -> int:
    return _lib.car_reduce_residual_rmsnorm_backward(h, _table(dnorm) if dnorm is not None else None, residual_out,
                                                     weight, eps, dresidual_out, dx, dweight, workspace, stream)


def car_backward_workspace_bytes(h) -> int:
    return int(_lib.car_backward_workspace_bytes(h))


def _ref(struct):
    return ctypes.byref(struct) if struct is not None else None


def car_reduce_dropout(h, inputs, drop, ar_out: int, stream: int = 0) -> int:
    """drop: a car_dropout."""
    return _lib.car_reduce_dropout(h, _table(inputs) if inputs is not None else None, _ref(drop), ar_out, stream)


def car_reduce_branch_residual_rmsnorm(h, inputs, branch, residual: int, weight: int, eps: float, residual_out: int,
                                       norm_out: int, ar_out: int | None, stream: int = 0) -> int:
    """branch: a car_branch."""
    return _lib.car_reduce_branch_residual_rmsnorm(h, _table(inputs) if inputs is not None else None, _ref(branch), residual,
                                                   weight, eps, residual_out, norm_out, ar_out, stream)


def car_reduce_branch_residual_rmsnorm_backward(h, dnorm, branch, ar: int | None, residual_out: int, weight: int,
                                                eps: float, dresidual_out: int | None, out, workspace: int | None,
                                                stream: int = 0) -> int:
    """branch: a car_branch; out: a car_branch_grads, or its bytes."""
    return _lib.car_reduce_branch_residual_rmsnorm_backward(h, _table(dnorm) if dnorm is not None else None, _ref(branch), ar,
                                                            residual_out, weight, eps, dresidual_out,
                                                            out if isinstance(out, bytes) else _ref(out), workspace,
                                                            stream)


def car_branch_workspace_bytes(h, branch) -> int:
    return int(_lib.car_branch_workspace_bytes(h, _ref(branch)))


def car_grads_create(W: int, numel, dtypes, inputs, outs):
    """inputs: W * n device addresses, rank-major; outs: n.  Returns (status, handle)."""
    n = len(numel)
    out = ctypes.c_void_p()
    st = _lib.car_grads_create(W, n, (ctypes.c_int64 * n)(*numel), (ctypes.c_int * n)(*dtypes),
                               _table(inputs) if inputs is not None else None,
                               _table(outs) if outs is not None else None, ctypes.byref(out))
    return st, out.value


def car_grads_destroy(g) -> int:
    return _lib.car_grads_destroy(g)


def car_grads_reduce(g, scale: float, sumsq: int, stream: int = 0) -> int:
    return _lib.car_grads_reduce(g, scale, sumsq, stream)


def car_grads_clip(g, sumsq: int, max_norm: float, norm_out: int | None, stream: int = 0) -> int:
    return _lib.car_grads_clip(g, sumsq, max_norm, norm_out, stream)


def car_grads_reduce_clip(g, scale: float, max_norm: float, norm_out: int | None, stream: int = 0) -> int:
    return _lib.car_grads_reduce_clip(g, scale, max_norm, norm_out, stream)


def car_grads_reduce_clip_once(g, scale: float, max_norm: float, norm_out: int | None, stream: int = 0) -> int:
    return _lib.car_grads_reduce_clip_once(g, scale, max_norm, norm_out, stream)


def car_ll128_wire_bytes(h) -> int:
    return int(_lib.car_ll128_wire_bytes(h))


def car_ll128_encode(h, data: int, flag: int, wire: int, stream: int = 0) -> int:
    return _lib.car_ll128_encode(h, data, flag, wire, stream)


def car_ll128_decode_reduce(h, wires, expected_flag: int, max_polls: int, ar_out: int, stream: int = 0) -> int:
    return _lib.car_ll128_decode_reduce(h, _table(wires) if wires is not None else None, expected_flag, max_polls,
                                        ar_out, stream)


def _report(fn, h, cap: int):
    entries = (ctypes.c_uint32 * 2 * max(cap, 1))()
    rep = car_stale_report(0, 0, cap, ctypes.cast(entries, ctypes.POINTER(ctypes.c_uint32 * 2)))
    st = fn(h, ctypes.byref(rep))
    pairs = [(entries[i][0], entries[i][1]) for i in range(rep.n_listed)]
    return st, int(rep.n_stale), pairs


def car_ll128_report(h, cap: int = CAR_STALE_LIST_MAX):
    """Returns (status, n_stale, [(rank, line), ...])."""
    return _report(_lib.car_ll128_report, h, cap)


def car_ll128_decode_reduce_noalloc(W: int, M: int, N: int, dtype: int, wires, expected_flag: int, max_polls: int,
                                    ar_out: int, stale_out: int, cap: int, stream: int = 0) -> int:
    """Handle-free LL128 decode-reduce that allocates nothing (see car.h):
    stale_out is a device buffer of 16 + 8*cap bytes."""
    return _lib.car_ll128_decode_reduce_noalloc(W, M, N, dtype, _table(wires) if wires is not None else None,
                                                expected_flag, max_polls, ar_out, stale_out, cap, stream)


def car_ll_wire_bytes(h) -> int:
    return int(_lib.car_ll_wire_bytes(h))


def car_ll_encode(h, data: int, flag: int, wire: int, stream: int = 0) -> int:
    return _lib.car_ll_encode(h, data, flag, wire, stream)


def car_ll_decode_reduce(h, wires, expected_flag: int, max_polls: int, ar_out: int, stream: int = 0) -> int:
    return _lib.car_ll_decode_reduce(h, _table(wires) if wires is not None else None, expected_flag, max_polls,
                                     ar_out, stream)


def car_ll_report(h, cap: int = CAR_STALE_LIST_MAX):
    return _report(_lib.car_ll_report, h, cap)


def car_lamport_buffer_bytes(h) -> int:
    return int(_lib.car_lamport_buffer_bytes(h))


def car_lamport_init(h, comm: int, stream: int = 0) -> int:
    return _lib.car_lamport_init(h, comm, stream)


def car_lamport_push(h, data: int, rank: int, round_: int, comm: int, stream: int = 0) -> int:
    return _lib.car_lamport_push(h, data, rank, round_, comm, stream)


def car_lamport_reduce_residual_rmsnorm(h, comm: int, round_: int, max_polls: int, residual: int, weight: int,
                                        eps: float, residual_out: int, norm_out: int, ar_out: int | None,
                                        stream: int = 0) -> int:
    return _lib.car_lamport_reduce_residual_rmsnorm(h, comm, round_, max_polls, residual, weight, eps,
                                                    residual_out, norm_out, ar_out, stream)


def car_lamport_report(h, cap: int = CAR_STALE_LIST_MAX):
    return _report(_lib.car_lamport_report, h, cap)


def car_status_string(st: int) -> str:
    return _lib.car_status_string(st).decode()


def car_last_error() -> str:
    return _lib.car_last_error().decode()


def car_tune_fused(h, kernel: int, cluster: int, threads: int, vpt: int) -> int:
    return _lib.car_tune_fused(h, kernel, cluster, threads, vpt)


def car_sync(h, stream: int = 0) -> int:
    return _lib.car_sync(h, stream)


def car_test_delay_partial(h, wait_limit_ns: int, cta: int, row: int, delay_ns: int) -> int:
    return _lib.car_test_delay_partial(h, wait_limit_ns, cta, row, delay_ns)


# ---------------------------------------------------------------------------
# torch convenience layer (still only marshalling)
# ---------------------------------------------------------------------------
class CarError(RuntimeError):
    def __init__(self, status: int, what: str):
        detail = car_last_error() if status == CAR_ERR_CUDA else ""
        super().__init__(f"{what}: {STATUS_NAME.get(status, status)} {detail}".strip())
        self.status = status


def check(status: int, what: str = "car") -> None:
    if status:  # not CAR_OK
        raise CarError(status, what)


@functools.lru_cache(maxsize=1)
def _cuda():
    import torch

    return torch.cuda


@functools.lru_cache(maxsize=1)
def _raw_stream():
    """device index -> handle of torch's current stream.  torch.cuda.current_stream builds a Stream object first
    (1.1 to 2.9 us a call, measured on GB300's host, against 0.1): the raw form is used where torch has it."""
    import torch

    return getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: torch.cuda.current_stream(d).cuda_stream)


def _stream(stream, device=None):
    """Handle of `stream`, or of torch's current stream on `device` (by default the current one)."""
    if stream is None:
        return _raw_stream()(_cuda().current_device() if device is None else device)
    return stream if isinstance(stream, int) else stream.cuda_stream


@functools.lru_cache(maxsize=1)
def _types():
    """Types of the outputs that are not of the handle's own: q_out, scales by kind, dweight."""
    import torch

    f32 = (torch.float32,)
    return ((torch.float8_e4m3fn, torch.uint8),
            {k: (torch.uint8, torch.float8_e8m0fnu) if k == "mx32" else f32 for k in SCALE_CODE}, f32)


def _check_type(t, allowed, what: str) -> None:
    if t.dtype not in allowed:
        raise ValueError(f"{what}: {t.dtype}, the call needs {' or '.join(str(d) for d in allowed)}")


@functools.lru_cache(maxsize=1)
def _own_types():
    """The handles' types, by name."""
    import torch

    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _check_own_type(t, own, what: str) -> None:
    """A tensor of a handle's type: that, or raw bytes in one of whole numbers."""
    if t.dtype is not own and (t.is_floating_point() or t.is_complex()):
        raise ValueError(f"{what}: {t.dtype}, the handle's type is {own}")


def _ptr(t, nbytes: int, what: str, device=None) -> int:
    """Device pointer of a tensor the library will read or write `nbytes` of:
    it must be a contiguous CUDA tensor at least that large, on `device` when
    given (any dtype: the library sees bytes)."""
    if (t.get_device() == device if device is not None else t.is_cuda) and t.is_contiguous() and t.nbytes >= nbytes:
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"{what}: expected a CUDA tensor")
    if device is not None and t.device.index != device:
        raise ValueError(f"{what}: on cuda:{t.device.index}, the handle is on cuda:{device}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor")
    raise ValueError(f"{what}: {t.numel() * t.element_size()} bytes, the call needs {nbytes}")


class Dropout:
    """Dropout with probability p (rounded to a multiple of 2^-16) whose mask is a function of seed, offset and the
    element's place alone (see car_dropout): a backward with the same values sees the forward's mask.  offset_dev, if
    given, is a CUDA tensor of one 64-bit integer that is added to offset when a kernel runs, so that a captured call can
    be given another mask at every replay.  seed and offset are any integers, taken mod 2^64.  Every field may be set
    anew between calls, which take what it holds then; the object keeps offset_dev, whose address each call takes."""

    def __init__(self, p, seed, offset=0, offset_dev=None):
        self.struct = car_dropout()
        self.address = ctypes.addressof(self.struct)   # quicker to pass than a reference
        self.p, self.seed, self.offset, self.offset_dev = p, seed, offset, offset_dev

    def __copy__(self):   # with a struct of its own
        return Dropout(self.p, self.seed, self.offset, self.offset_dev)

    @property
    def p(self) -> float:
        return self._p

    @p.setter
    def p(self, value: float):
        if not 0.0 <= value <= 1.0:
            raise ValueError(f"p: {value} is not in [0, 1]")
        self._p = self.struct.p = value

    @property
    def seed(self) -> int:
        return self.struct.seed

    @seed.setter
    def seed(self, value: int):
        self.struct.seed = value % 2**64

    @property
    def offset(self) -> int:
        return self.struct.offset

    @offset.setter
    def offset(self, value: int):
        self.struct.offset = value % 2**64

    @property
    def offset_dev(self):
        return self._offset_dev

    @offset_dev.setter
    def offset_dev(self, t):
        if t is not None:
            import torch

            _check_type(t, (torch.int64, torch.uint64), "offset_dev")
            _ptr(t, 8, "offset_dev")
        self._offset_dev = t
        self.struct.offset_dev = t.data_ptr() if t is not None else None


class Branch:
    """What a block adds to the residual stream (see car_branch): the rank sum, normalised if there is a norm_weight
    [N], times the gate, dropped out; residual_scale multiplies the residual.  gate_rows: 1 for a gate [N] (or [1, N]) of
    all rows, G for one row [G, N] for each of G samples of M / G consecutive rows, 0 for [M, N], a row of its own for
    every row.  norm_weight and gate are contiguous CUDA tensors of the handle's type (or its bytes in a type of whole
    numbers) with just so many values: a gate of more rows than gate_rows is refused.  Every field may be set anew
    between calls, which take what it holds then; the object keeps its tensors, whose addresses each call takes (a
    parameter's data may be another tensor's by then)."""

    def __init__(self, norm_weight=None, norm_eps=1e-6, gate=None, gate_rows=1, residual_scale=1.0, dropout=None):
        self.struct = car_branch()
        self.ref, self.address = ctypes.byref(self.struct), ctypes.addressof(self.struct)
        self.norm_weight, self.gate = norm_weight, gate   # their addresses: written into the struct here and by every call
        self.norm_eps, self.gate_rows, self.residual_scale, self.dropout = norm_eps, gate_rows, residual_scale, dropout

    def __copy__(self):   # with a struct of its own; its tensors and dropout are the same objects
        return Branch(self.norm_weight, self.norm_eps, self.gate, self.gate_rows, self.residual_scale, self.dropout)

    @property
    def norm_weight(self):
        return self._norm_weight

    @norm_weight.setter
    def norm_weight(self, t):
        self.struct.norm_weight = t.data_ptr() if t is not None else None
        self._norm_weight = t

    @property
    def gate(self):
        return self._gate

    @gate.setter
    def gate(self, t):
        self.struct.gate = t.data_ptr() if t is not None else None
        self._gate = t

    @property
    def norm_eps(self) -> float:
        return self._norm_eps

    @norm_eps.setter
    def norm_eps(self, value: float):
        self._norm_eps = self.struct.norm_eps = value

    @property
    def gate_rows(self) -> int:
        return self._gate_rows

    @gate_rows.setter
    def gate_rows(self, value: int):
        if value < 0:
            raise ValueError(f"gate_rows: {value} is negative")
        self._gate_rows = self.struct.gate_rows = value

    @property
    def residual_scale(self) -> float:
        return self._residual_scale

    @residual_scale.setter
    def residual_scale(self, value: float):
        self._residual_scale = self.struct.residual_scale = value

    @property
    def dropout(self):
        return self._dropout

    @dropout.setter
    def dropout(self, value):
        self.struct.dropout = ctypes.pointer(value.struct) if value is not None else None
        self._dropout = value


class Car:
    """A libcar handle for W rank buffers of [M, N] elements of one dtype.

    The methods take torch tensors and pass their device pointers to the C
    ABI; each tensor must be a contiguous CUDA tensor of at least the bytes
    the call reads or writes (ValueError otherwise).  Tensors of the handle's
    type are taken as bytes; those of another type are checked for it."""

    def __init__(self, W: int, M: int, N: int, dtype: str):
        st, h = car_create(W, M, N, DTYPE_CODE[dtype])
        check(st, "car_create")
        self.h, self.W, self.M, self.N, self.dtype = h, W, M, N, dtype
        self.D = M * N * ELEM_SIZE[dtype]      # bytes per rank
        D, Nw = self.D, N * ELEM_SIZE[dtype]
        self._row = Nw                         # bytes of one row
        # bytes that the tensors of a call need, in the order of its arguments
        self._quant_sizes = [(D, Nw, D, M * N, car_quant_scale_bytes(h, k), D, D) for k in range(len(SCALE_CODE))]
        self._backward_sizes = None   # found when first asked for
        self._branch_sizes = {}       # the same, by gate_rows
        self._type = _own_types()[dtype]
        import torch

        self.device = torch.cuda.current_device()

    def _p(self, t, nbytes: int, what: str) -> int:
        return _ptr(t, nbytes, what, self.device)

    def _ranks(self, ts, nbytes: int, what: str):
        if len(ts) != self.W:
            raise ValueError(f"{what}: {len(ts)} tensors for W = {self.W}")
        dev = self.device  # one test for all is quicker than _ptr for each, which then names the one that failed
        got = [t.data_ptr() for t in ts if t.get_device() == dev and t.is_contiguous() and t.nbytes >= nbytes]
        if len(got) == self.W:
            return got
        return [self._p(t, nbytes, f"{what}[{r}]") for r, t in enumerate(ts)]

    def close(self):
        if self.h is not None:
            check(car_destroy(self.h), "car_destroy")
            self.h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def ll128_wire_bytes(self) -> int:
        return car_ll128_wire_bytes(self.h)

    @property
    def ll_wire_bytes(self) -> int:
        return car_ll_wire_bytes(self.h)

    def reduce(self, xs, ar_out, stream=None):
        check(car_reduce(self.h, self._ranks(xs, self.D, "inputs"), self._p(ar_out, self.D, "ar_out"), _stream(stream)),
              "car_reduce")

    def reduce_two_shot(self, xs, ar_out, stream=None):
        check(car_reduce_two_shot(self.h, self._ranks(xs, self.D, "inputs"), self._p(ar_out, self.D, "ar_out"),
                                  _stream(stream)), "car_reduce_two_shot")

    def reduce_residual_rmsnorm(self, xs, residual, weight, eps, residual_out, norm_out, ar_out=None, stream=None):
        D = self.D
        check(car_reduce_residual_rmsnorm(self.h, self._ranks(xs, D, "inputs"), self._p(residual, D, "residual"),
                                          self._p(weight, D // self.M, "weight"), eps,
                                          self._p(residual_out, D, "residual_out"), self._p(norm_out, D, "norm_out"),
                                          self._p(ar_out, D, "ar_out") if ar_out is not None else None,
                                          _stream(stream)), "car_reduce_residual_rmsnorm")

    def quant_scales_shape(self, kind: str) -> tuple:
        """Shape of the scales of the 8-bit output: fp32, or one byte each for "mx32"."""
        groups = {"row": 1, "group128": -(-self.N // 128), "mx32": -(-self.N // 32)}
        return (1,) if kind == "static" else (self.M, groups[kind])

    def _ptrs(self, ts, sizes, names):
        """Device pointers of several tensors, each checked as by _ptr (None stays None)."""
        dev = self.device  # one test for all is quicker than _ptr for each, which then names the one that failed
        got = [None if t is None else t.data_ptr() if t.get_device() == dev and t.is_contiguous() and t.nbytes >= n else 0
               for t, n in zip(ts, sizes)]
        if 0 in got:
            got = [None if t is None else _ptr(t, n, what, dev) for t, n, what in zip(ts, sizes, names)]
        return got

    def reduce_residual_rmsnorm_quant(self, xs, residual, weight, eps, kind, residual_out, q_out, scales,
                                      norm_out=None, ar_out=None, stream=None):
        """kind: "row", "group128", "mx32" or "static" (see car_scale_kind).  q_out: M * N bytes (float8_e4m3fn or
        uint8); scales: quant_scales_shape(kind), float32 (for "mx32" uint8 or float8_e8m0fnu), written, or read for
        "static"."""
        code = SCALE_CODE.get(kind)
        if code is None:
            raise ValueError(f"kind: {kind!r} is none of {', '.join(SCALE_CODE)}")
        q_types, scale_types, _ = _types()
        _check_type(q_out, q_types, "q_out")
        _check_type(scales, scale_types[kind], "scales")
        res, w, ro, q, sc, no, ar = self._ptrs(
            (residual, weight, residual_out, q_out, scales, norm_out, ar_out), self._quant_sizes[code],
            ("residual", "weight", "residual_out", "q_out", "scales", "norm_out", "ar_out"))
        check(_lib.car_reduce_residual_rmsnorm_quant(self.h, _table(self._ranks(xs, self.D, "inputs")), res, w, eps, code,
                                                     ro, q, sc, no, ar, _stream(stream, self.device)),
              "car_reduce_residual_rmsnorm_quant")

    @property
    def backward_workspace_bytes(self) -> int:
        if self._backward_sizes is None:
            D, N = self.D, self.N
            self._backward_sizes = (D, D // self.M, D, D, 4 * N, car_backward_workspace_bytes(self.h))
        return self._backward_sizes[-1]

    def reduce_residual_rmsnorm_backward(self, dnorm, residual_out, weight, eps, dresidual_out, dx, dweight=None,
                                         workspace=None, stream=None):
        """dresidual_out and dweight may be None; dweight is fp32.  With a dweight, workspace (backward_workspace_bytes
        bytes) is taken from torch's allocator on the current stream when none is given."""
        if dweight is not None:
            _check_type(dweight, _types()[2], "dweight")
        need = self.backward_workspace_bytes
        if dweight is None:
            need = 0
        if need and workspace is None:
            import torch

            if stream is not None and _stream(stream) != torch.cuda.current_stream().cuda_stream:
                raise ValueError("workspace: give one for a call on another stream than the current one")
            workspace = torch.empty(need, dtype=torch.uint8, device=dx.device)
        h, w, dro, out, dw, ws = self._ptrs(
            (residual_out, weight, dresidual_out, dx, dweight, workspace if need else None), self._backward_sizes,
            ("residual_out", "weight", "dresidual_out", "dx", "dweight", "workspace"))
        check(_lib.car_reduce_residual_rmsnorm_backward(self.h, _table(self._ranks(dnorm, self.D, "dnorm")), h, w, eps, dro,
                                                        out, dw, ws, _stream(stream, self.device)),
              "car_reduce_residual_rmsnorm_backward")

    def _dropout(self, dropout):
        """Address of its struct, with what its tensor is now."""
        t = dropout._offset_dev
        if t is not None:
            dropout.struct.offset_dev = self._p(t, 8, "offset_dev")
        return dropout.address

    def _branch(self, branch):
        """Address of its struct, with what its tensors are now."""
        w, g, d, s, own, dev = branch._norm_weight, branch._gate, branch._dropout, branch.struct, self._type, self.device
        if w is None:
            s.norm_weight = None
        elif w.dtype is own and w.nbytes == self._row and w.get_device() == dev and w.is_contiguous():
            s.norm_weight = w.data_ptr()
        else:
            s.norm_weight = self._values(w, self._row, "norm_weight")
        if g is None:
            s.gate = None
        else:
            n = (branch._gate_rows or self.M) * self._row
            if g.dtype is own and g.nbytes == n and g.get_device() == dev and g.is_contiguous():
                s.gate = g.data_ptr()
            else:
                s.gate = self._values(g, n, "gate")
        if d is not None and d._offset_dev is not None:
            self._dropout(d)
        return branch.address

    def _values(self, t, nbytes: int, what: str) -> int:
        """Address of a tensor of the handle's type that holds just that much."""
        _check_own_type(t, self._type, what)
        at = self._p(t, nbytes, what)
        if t.nbytes != nbytes:
            raise ValueError(f"{what}: shape {tuple(t.shape)}, the call takes {nbytes // t.element_size()} values")
        return at

    def reduce_dropout(self, xs, dropout, ar_out, stream=None):
        """ar_out = dropout of the rank sum; its gradient is the same call on the gradient's rank contributions."""
        check(_lib.car_reduce_dropout(self.h, _table(self._ranks(xs, self.D, "inputs")), self._dropout(dropout),
                                      self._p(ar_out, self.D, "ar_out"), _stream(stream, self.device)), "car_reduce_dropout")

    def reduce_branch_residual_rmsnorm(self, xs, branch, residual, weight, eps, residual_out, norm_out, ar_out=None,
                                       stream=None):
        """reduce_residual_rmsnorm with a Branch between the rank sum and the residual add.  ar_out: the rank sum, which
        the backward needs behind a norm and for the gate's gradient."""
        D = self.D
        if weight.dtype is not self._type:
            _check_own_type(weight, self._type, "weight")
        res, w, ro, no, ar = self._ptrs((residual, weight, residual_out, norm_out, ar_out), (D, self._row, D, D, D),
                                        ("residual", "weight", "residual_out", "norm_out", "ar_out"))
        check(_lib.car_reduce_branch_residual_rmsnorm(self.h, _table(self._ranks(xs, D, "inputs")),
                                                      self._branch(branch), res, w, eps, ro, no, ar,
                                                      _stream(stream, self.device)), "car_reduce_branch_residual_rmsnorm")

    def branch_workspace_bytes(self, branch=None) -> int:
        """Of the backward's workspace; depends on whether rows share a row of the branch's gate."""
        key = branch._gate_rows if branch is not None and branch._gate is not None else 0
        need = self._branch_sizes.get(key)
        if need is None:
            gate = 16 if key else None   # any: a shared gate, or none
            need = self._branch_sizes[key] = car_branch_workspace_bytes(self.h, car_branch(gate=gate, gate_rows=key))
        return need

    def reduce_branch_residual_rmsnorm_backward(self, dnorm, branch, ar, residual_out, weight, eps, dresidual_out, dx,
                                                dresidual=None, dweight=None, dnorm_weight=None, dgate=None,
                                                workspace=None, stream=None):
        """Gradients of reduce_branch_residual_rmsnorm.  ar may be None without a norm and a dgate; dresidual_out and
        every gradient but dx may be None.  dweight and dnorm_weight are fp32 [N]; dgate is fp32 like the gate, or with
        gate_rows 0 [M, N] of the handle's type.  workspace (branch_workspace_bytes(branch) bytes) is taken from torch's
        allocator on the current stream when one is needed and none is given."""
        f32, D, N, rows = _types()[2], self.D, self.N, branch._gate_rows
        shared = rows > 0
        for t, what in ((dweight, "dweight"), (dnorm_weight, "dnorm_weight"), (dgate if shared else None, "dgate")):
            if t is not None and t.dtype not in f32:
                _check_type(t, f32, what)
        own = self._type
        if weight.dtype is not own:
            _check_own_type(weight, own, "weight")
        if not shared and dgate is not None and dgate.dtype is not own:
            _check_own_type(dgate, own, "dgate")
        need = 0
        if dweight is not None or dnorm_weight is not None or (dgate is not None and shared):
            need = self.branch_workspace_bytes(branch)
        if need and workspace is None:
            import torch

            if stream is not None and _stream(stream) != torch.cuda.current_stream().cuda_stream:
                raise ValueError("workspace: give one for a call on another stream than the current one")
            workspace = torch.empty(need, dtype=torch.uint8, device=dx.device)
        a, h, w, dro, out, dr, dw, dw1, dg, ws = self._ptrs(
            (ar, residual_out, weight, dresidual_out, dx, dresidual, dweight, dnorm_weight, dgate, workspace if need else None),
            (D, D, self._row, D, D, D, 4 * N, 4 * N, 4 * N * rows if shared else D, need),
            ("ar", "residual_out", "weight", "dresidual_out", "dx", "dresidual", "dweight", "dnorm_weight", "dgate", "workspace"))
        check(_lib.car_reduce_branch_residual_rmsnorm_backward(
            self.h, _table(self._ranks(dnorm, D, "dnorm")), self._branch(branch), a, h, w, eps, dro,
            _packer(5)(out, dr or 0, dw or 0, dw1 or 0, dg or 0), ws, _stream(stream, self.device)),
            "car_reduce_branch_residual_rmsnorm_backward")

    def ll128_encode(self, data, flag, wire, stream=None):
        check(car_ll128_encode(self.h, self._p(data, self.D, "data"), flag, self._p(wire, self.ll128_wire_bytes, "wire"),
                               _stream(stream)), "car_ll128_encode")

    def ll128_decode_reduce(self, wires, expected_flag, ar_out, max_polls=1, stream=None):
        check(car_ll128_decode_reduce(self.h, self._ranks(wires, self.ll128_wire_bytes, "wires"), expected_flag,
                                      max_polls, self._p(ar_out, self.D, "ar_out"), _stream(stream)),
              "car_ll128_decode_reduce")

    def ll128_report(self, cap=CAR_STALE_LIST_MAX):
        st, n, pairs = car_ll128_report(self.h, cap)
        if st not in (CAR_OK, CAR_ERR_STALE_FLAG):
            check(st, "car_ll128_report")
        return n, pairs

    def ll_encode(self, data, flag, wire, stream=None):
        check(car_ll_encode(self.h, self._p(data, self.D, "data"), flag, self._p(wire, self.ll_wire_bytes, "wire"),
                            _stream(stream)), "car_ll_encode")

    def ll_decode_reduce(self, wires, expected_flag, ar_out, max_polls=1, stream=None):
        check(car_ll_decode_reduce(self.h, self._ranks(wires, self.ll_wire_bytes, "wires"), expected_flag,
                                   max_polls, self._p(ar_out, self.D, "ar_out"), _stream(stream)),
              "car_ll_decode_reduce")

    def ll_report(self, cap=CAR_STALE_LIST_MAX):
        st, n, pairs = car_ll_report(self.h, cap)
        if st not in (CAR_OK, CAR_ERR_STALE_FLAG):
            check(st, "car_ll_report")
        return n, pairs

    @property
    def lamport_buffer_bytes(self) -> int:
        return car_lamport_buffer_bytes(self.h)

    def lamport_init(self, comm, stream=None):
        check(car_lamport_init(self.h, self._p(comm, self.lamport_buffer_bytes, "comm"), _stream(stream)),
              "car_lamport_init")

    def lamport_push(self, data, rank, round_, comm, stream=None):
        check(car_lamport_push(self.h, self._p(data, self.D, "data"), rank, round_,
                               self._p(comm, self.lamport_buffer_bytes, "comm"), _stream(stream)), "car_lamport_push")

    def lamport_reduce_residual_rmsnorm(self, comm, round_, residual, weight, eps, residual_out, norm_out,
                                        ar_out=None, max_polls=1, stream=None):
        D = self.D
        check(car_lamport_reduce_residual_rmsnorm(self.h, self._p(comm, self.lamport_buffer_bytes, "comm"), round_,
                                                  max_polls, self._p(residual, D, "residual"),
                                                  self._p(weight, D // self.M, "weight"), eps,
                                                  self._p(residual_out, D, "residual_out"), self._p(norm_out, D, "norm_out"),
                                                  self._p(ar_out, D, "ar_out") if ar_out is not None else None,
                                                  _stream(stream)), "car_lamport_reduce_residual_rmsnorm")

    def lamport_report(self, cap=CAR_STALE_LIST_MAX):
        st, n, pairs = car_lamport_report(self.h, cap)
        if st not in (CAR_OK, CAR_ERR_STALE_FLAG):
            check(st, "car_lamport_report")
        return n, pairs

    def tune_fused(self, kernel=CAR_FUSED_AUTO, cluster=0, threads=0, vpt=0):
        check(car_tune_fused(self.h, kernel, cluster, threads, vpt), "car_tune_fused")

    def sync(self, stream=None):
        check(car_sync(self.h, _stream(stream)), "car_sync")


class Grads:
    """The gradients of one data-parallel step: rank sum, global norm, clipping.

    inputs: W sequences of n tensors (one per rank); outs: n tensors.  Tensor
    t of every rank and of outs has the same number of elements and the same
    type (bf16, fp16 or fp32); all are contiguous on one CUDA device.  outs[t]
    may be inputs[r][t] itself.  The object keeps the tensors."""

    def __init__(self, inputs, outs):
        import torch

        code = {torch.bfloat16: CAR_BF16, torch.float16: CAR_FP16, torch.float32: CAR_FP32}
        self.inputs, self.outs, self.h = [list(ts) for ts in inputs], list(outs), None
        if not self.inputs or not self.outs:
            raise ValueError("inputs, outs: need at least one rank and one tensor")
        self.device, self._f32, self._f64 = self.outs[0].device.index, torch.float32, torch.float64
        for t, o in enumerate(self.outs):
            if o.dtype not in code:
                raise ValueError(f"outs[{t}]: {o.dtype} is not bf16, fp16 or fp32")
        n, flat = len(self.outs), []
        for r, ts in enumerate(self.inputs):
            if len(ts) != n:
                raise ValueError(f"inputs[{r}]: {len(ts)} tensors for {n} outputs")
            for t, (x, o) in enumerate(zip(ts, self.outs)):
                if x.dtype != o.dtype or x.numel() != o.numel():
                    raise ValueError(f"inputs[{r}][{t}]: {x.numel()} x {x.dtype}, outs[{t}] is {o.numel()} x {o.dtype}")
                flat.append(_ptr(x, 0, f"inputs[{r}][{t}]", self.device))
        to = [_ptr(o, 0, f"outs[{t}]", self.device) for t, o in enumerate(self.outs)]
        with torch.cuda.device(self.device):
            st, h = car_grads_create(len(self.inputs), [o.numel() for o in self.outs], [code[o.dtype] for o in self.outs],
                                     flat, to)
        if st == CAR_ERR_ARG and car_last_error():
            raise ValueError(car_last_error())
        check(st, "car_grads_create")
        self.h = h

    def close(self):
        if self.h is not None:
            check(car_grads_destroy(self.h), "car_grads_destroy")
            self.h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _scalar(self, t, nbytes: int, what: str, dtype) -> int:
        if t.dtype != dtype:
            raise ValueError(f"{what}: {t.dtype}, the call needs {dtype}")
        return _ptr(t, nbytes, what, self.device)

    def reduce(self, scale, sumsq, stream=None):
        """outs = scale * rank sums; sumsq (float64, one element) = the sum of their squares."""
        check(car_grads_reduce(self.h, scale, self._scalar(sumsq, 8, "sumsq", self._f64), _stream(stream, self.device)),
              "car_grads_reduce")

    def clip(self, sumsq, max_norm, norm_out=None, stream=None):
        """outs *= min(1, max_norm / (sqrt(sumsq) + 1e-6)); norm_out (float32, one element) = sqrt(sumsq)."""
        check(car_grads_clip(self.h, self._scalar(sumsq, 8, "sumsq", self._f64), max_norm,
                             self._scalar(norm_out, 4, "norm_out", self._f32) if norm_out is not None else None,
                             _stream(stream, self.device)), "car_grads_clip")

    def reduce_clip(self, scale, max_norm, norm_out=None, stream=None, once=False):
        """Both, for gradients that are all in this object.  once: no sum is rounded to its type before it is clipped,
        at the cost of reading the ranks' 16-bit tensors again when it is."""
        call = car_grads_reduce_clip_once if once else car_grads_reduce_clip
        check(call(self.h, scale, max_norm, self._scalar(norm_out, 4, "norm_out", self._f32) if norm_out is not None else None,
                   _stream(stream, self.device)), "car_grads_reduce_clip")
