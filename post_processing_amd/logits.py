"""Python binding of the operators over rows of logits (include/ws_logits.h).

Argument marshalling only, as in ``ws``: every step runs in the HIP library.

A call object binds its configuration and buffers once and enqueues the
operator each time ``run`` is called, on the buffers' contents of that moment:

    rows = make_rows(rows=T, vocab=V, dtype=ws.DTYPE_BF16)
    call = LogProbs(rows, logits, targets=targets, logprob=logprob)
    call.run(stream)

Buffers are torch tensors (anything with ``data_ptr()``) or integer device
addresses.  A tensor's element type, device and size are checked when the call
object is built; an address is taken as it is.  ``stream`` is a hipStream_t
handle (int) or None for the null stream, as in ``ws.run_noalloc``.  The call
object keeps the tensors alive: keep it until the stream has passed its last
run, and for as long as a graph that captured it may be replayed.

When an operator needs a workspace and none is given, the call object holds
one of its own, taken from torch; so two runs of one call object must not
overlap in time, while two call objects may.  torch hands out memory whose last
user may still be queued on its current stream, so building such a call object
waits for that stream: the runs may then go to any stream.  Built while torch
captures that stream there is nothing to wait for, and the call object belongs
to that graph: run it on the capturing stream, or one that waits for it, and
nowhere else.  Buffers and workspaces that are given are the caller's to order.
"""
from __future__ import annotations

import ctypes
from ctypes import POINTER, Structure, byref, c_float, c_int, c_int32, c_int64, c_size_t, c_void_p

from . import ws

DISTILL_RENORM = 0
DISTILL_TAIL = 1
DISTILL_MAX_K = 128
MAX_ROWS = 1 << 22


class Rows(Structure):
    _fields_ = [("device", c_int32), ("dtype", c_int32), ("rows", c_int32), ("vocab", c_int32),
                ("row_stride", c_int64), ("temperature", c_float), ("reserved", c_int32)]


class RowStats(Structure):
    _fields_ = [("max", c_float), ("logsum", c_float)]


class LogProbsArgs(Structure):
    _fields_ = [("logits", c_void_p), ("targets", c_void_p), ("logprob", c_void_p),
                ("entropy", c_void_p), ("top", c_void_p), ("stats", c_void_p),
                ("workspace", c_void_p), ("workspace_bytes", c_size_t), ("top_k", c_int32),
                ("reserved", c_int32)]


class LogProbsGradArgs(Structure):
    _fields_ = [("logits", c_void_p), ("stats", c_void_p), ("targets", c_void_p),
                ("grad_logprob", c_void_p), ("entropy", c_void_p), ("grad_entropy", c_void_p),
                ("top", c_void_p), ("grad_top", c_void_p), ("grad_logits", c_void_p),
                ("grad_stride", c_int64), ("top_k", c_int32), ("reserved", c_int32)]


class DistillArgs(Structure):
    _fields_ = [("logits", c_void_p), ("teacher", c_void_p), ("loss", c_void_p),
                ("stats", c_void_p), ("tail", c_void_p), ("grad_loss", c_void_p),
                ("grad_logits", c_void_p), ("grad_stride", c_int64), ("workspace", c_void_p),
                ("workspace_bytes", c_size_t), ("teacher_k", c_int32), ("mode", c_int32),
                ("reserved", c_int32 * 2)]


class DistillGradArgs(Structure):
    _fields_ = [("logits", c_void_p), ("teacher", c_void_p), ("stats", c_void_p),
                ("tail", c_void_p), ("grad_loss", c_void_p), ("grad_logits", c_void_p),
                ("grad_stride", c_int64), ("teacher_k", c_int32), ("mode", c_int32)]


_lib = None


def load():
    """The lane library with this header's prototypes set."""
    global _lib
    if _lib is not None:
        return _lib
    lib = ws.load()
    lib.ws_logprobs_workspace.argtypes = [POINTER(Rows), c_int32, POINTER(c_size_t)]
    lib.ws_distill_workspace.argtypes = [POINTER(Rows), c_int32, c_int32, POINTER(c_size_t)]
    lib.ws_logprobs.argtypes = [POINTER(Rows), POINTER(LogProbsArgs), c_void_p]
    lib.ws_logprobs_grad.argtypes = [POINTER(Rows), POINTER(LogProbsGradArgs), c_void_p]
    lib.ws_distill.argtypes = [POINTER(Rows), POINTER(DistillArgs), c_void_p]
    lib.ws_distill_grad.argtypes = [POINTER(Rows), POINTER(DistillGradArgs), c_void_p]
    for name in ("ws_logprobs_workspace", "ws_distill_workspace", "ws_logprobs",
                 "ws_logprobs_grad", "ws_distill", "ws_distill_grad"):
        getattr(lib, name).restype = c_int
    _lib = lib
    return lib


def _field(name, v, bits) -> int:
    """`v` as the ABI's field of `bits` takes it; ctypes would wrap it silently."""
    if not -(1 << bits - 1) <= v < 1 << bits - 1:
        raise ValueError(f"{name} = {v} does not fit {bits} bits")
    return v


def _int32(name, v) -> int:
    return _field(name, v, 32)


def _int64(name, v) -> int:
    return _field(name, v, 64)


def make_rows(*, rows, vocab, dtype=ws.DTYPE_F32, row_stride=None, temperature=1.0,
              device=0) -> Rows:
    r = Rows()
    r.device = _int32("device", device)
    r.dtype = _int32("dtype", dtype)
    r.rows = _int32("rows", rows)
    r.vocab = _int32("vocab", vocab)
    r.row_stride = _int64("row_stride", vocab if row_stride is None else row_stride)
    r.temperature = temperature
    return r


def logprobs_workspace(rows: Rows, top_k: int = 0) -> int:
    """Bytes of workspace ws_logprobs needs for this shape."""
    n = c_size_t(0)
    _check(load().ws_logprobs_workspace(byref(rows), _int32("top_k", top_k), byref(n)),
           "ws_logprobs_workspace")
    return n.value


def distill_workspace(rows: Rows, mode: int, gradient: bool) -> int:
    """Bytes of workspace ws_distill needs for this shape and mode."""
    n = c_size_t(0)
    _check(load().ws_distill_workspace(byref(rows), _int32("mode", mode), 1 if gradient else 0, byref(n)),
           "ws_distill_workspace")
    return n.value


def _check(rc: int, what: str) -> None:
    if rc != ws.WS_OK:
        raise ws.WsError(rc, what)


_LOGIT_TYPES = {ws.DTYPE_F32: "torch.float32", ws.DTYPE_F16: "torch.float16",
                ws.DTYPE_BF16: "torch.bfloat16"}


def _buffer(name, x, rows: Rows, types, count) -> int | None:
    """Address of a packed buffer of at least `count` elements.  A tensor is
    checked; an element may also be spelled as several smaller ones (a
    score/index pair as two int32)."""
    if x is not None and hasattr(x, "data_ptr") and hasattr(x, "dtype"):
        if str(x.dtype) not in types:
            raise ValueError(f"{name}: {x.dtype}, expected {' or '.join(types)}")
        if not x.is_cuda or x.device.index != rows.device:
            raise ValueError(f"{name} is on {x.device}, expected cuda:{rows.device}")
        if not x.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if x.numel() < count:
            raise ValueError(f"{name} holds {x.numel()} elements, needs {count}")
    return ws._addr(x)


def _matrix(name, x, rows: Rows, stride: int) -> int | None:
    """Address of a [rows][vocab] matrix whose rows lie `stride` apart."""
    if x is not None and hasattr(x, "data_ptr") and hasattr(x, "dtype"):
        if str(x.dtype) != _LOGIT_TYPES.get(rows.dtype):
            raise ValueError(f"{name}: {x.dtype}, expected {_LOGIT_TYPES.get(rows.dtype)}")
        if not x.is_cuda or x.device.index != rows.device:
            raise ValueError(f"{name} is on {x.device}, expected cuda:{rows.device}")
        if x.dim() != 2 or tuple(x.shape) != (rows.rows, rows.vocab):
            raise ValueError(f"{name}: shape {tuple(x.shape)}, expected "
                             f"{(rows.rows, rows.vocab)}")
        if (rows.vocab > 1 and x.stride(1) != 1) or (rows.rows > 1 and x.stride(0) != stride):
            raise ValueError(f"{name}: strides {x.stride()}, expected ({stride}, 1)")
    return ws._addr(x)


_F32 = ("torch.float32",)
_I32 = ("torch.int32",)
_PAIR = ("torch.float32", "torch.int32")


class _Call:
    """A bound call: ``run`` enqueues it on `stream`."""

    _name = ""

    def _bind(self, rows: Rows, args, *keep):
        self._rows = Rows.from_buffer_copy(rows)
        self._args = args
        self._keep = keep
        self._fn = getattr(load(), self._name)
        self._refs = (byref(self._rows), byref(self._args))

    def _own_workspace(self, rows: Rows, args, given, need: int):
        if given is None and need:
            import torch
            given = torch.empty(need, dtype=torch.uint8, device=f"cuda:{rows.device}")
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream(rows.device).synchronize()
        elif hasattr(given, "is_cuda") and (not given.is_cuda or not given.is_contiguous()
                                            or given.device.index != rows.device):
            raise ValueError(f"workspace must be contiguous and on cuda:{rows.device}")
        args.workspace = ws._addr(given)
        if given is not None:
            args.workspace_bytes = given.numel() * given.element_size() \
                if hasattr(given, "numel") else need
        return given

    def submit(self, stream=None) -> int:
        """Enqueue on `stream`; returns the status."""
        return self._fn(*self._refs, stream)

    def run(self, stream=None) -> None:
        """Enqueue on `stream`; raises WsError on a refusal."""
        rc = self._fn(*self._refs, stream)
        if rc != ws.WS_OK:
            raise ws.WsError(rc, self._name)


class LogProbs(_Call):
    """ws_logprobs: log probabilities of `targets`, entropy and the `top_k`
    best alternatives (`top`: [rows][top_k] score/index pairs, an int32 or
    float32 tensor of two elements a pair)."""

    _name = "ws_logprobs"

    def __init__(self, rows: Rows, logits, *, targets=None, logprob=None, entropy=None, top_k=0,
                 top=None, stats=None, workspace=None):
        n = rows.rows
        a = LogProbsArgs()
        a.logits = _matrix("logits", logits, rows, rows.row_stride)
        a.targets = _buffer("targets", targets, rows, _I32, n)
        a.logprob = _buffer("logprob", logprob, rows, _F32, n)
        a.entropy = _buffer("entropy", entropy, rows, _F32, n)
        a.top = _buffer("top", top, rows, _PAIR, 2 * n * top_k)
        a.stats = _buffer("stats", stats, rows, _F32, 2 * n)
        a.top_k = _int32("top_k", top_k)
        workspace = self._own_workspace(rows, a, workspace, logprobs_workspace(rows, top_k))
        self._bind(rows, a, logits, targets, logprob, entropy, top, stats, workspace)


class LogProbsGrad(_Call):
    """ws_logprobs_grad: the gradient of LogProbs' outputs."""

    _name = "ws_logprobs_grad"

    def __init__(self, rows: Rows, logits, stats, grad_logits, *, targets=None,
                 grad_logprob=None, entropy=None, grad_entropy=None, top_k=0, top=None,
                 grad_top=None, grad_stride=None):
        n = rows.rows
        a = LogProbsGradArgs()
        a.grad_stride = _stride(grad_logits, rows, grad_stride)
        a.logits = _matrix("logits", logits, rows, rows.row_stride)
        a.grad_logits = _matrix("grad_logits", grad_logits, rows, a.grad_stride)
        a.stats = _buffer("stats", stats, rows, _F32, 2 * n)
        a.targets = _buffer("targets", targets, rows, _I32, n)
        a.grad_logprob = _buffer("grad_logprob", grad_logprob, rows, _F32, n)
        a.entropy = _buffer("entropy", entropy, rows, _F32, n)
        a.grad_entropy = _buffer("grad_entropy", grad_entropy, rows, _F32, n)
        a.top = _buffer("top", top, rows, _PAIR, 2 * n * top_k)
        a.grad_top = _buffer("grad_top", grad_top, rows, _F32, n * top_k)
        a.top_k = _int32("top_k", top_k)
        self._bind(rows, a, logits, stats, grad_logits, targets, grad_logprob, entropy,
                   grad_entropy, top, grad_top)


class Distill(_Call):
    """ws_distill: the loss of every row, and with `grad_logits` and
    `grad_loss` its gradient."""

    _name = "ws_distill"

    def __init__(self, rows: Rows, logits, teacher, teacher_k, mode, loss, *, stats=None,
                 tail=None, grad_loss=None, grad_logits=None, grad_stride=None, workspace=None):
        n = rows.rows
        a = DistillArgs()
        a.logits = _matrix("logits", logits, rows, rows.row_stride)
        a.teacher = _buffer("teacher", teacher, rows, _PAIR, 2 * n * teacher_k)
        a.loss = _buffer("loss", loss, rows, _F32, n)
        a.stats = _buffer("stats", stats, rows, _F32, 2 * n)
        a.tail = _buffer("tail", tail, rows, _F32, n)
        a.grad_loss = _buffer("grad_loss", grad_loss, rows, _F32, n)
        if grad_logits is not None:
            a.grad_stride = _stride(grad_logits, rows, grad_stride)
            a.grad_logits = _matrix("grad_logits", grad_logits, rows, a.grad_stride)
        a.teacher_k = _int32("teacher_k", teacher_k)
        a.mode = _int32("mode", mode)
        need = distill_workspace(rows, mode, grad_logits is not None)
        workspace = self._own_workspace(rows, a, workspace, need)
        self._bind(rows, a, logits, teacher, loss, stats, tail, grad_loss, grad_logits, workspace)


class DistillGrad(_Call):
    """ws_distill_grad: the gradient from an earlier Distill's stats and, with
    DISTILL_TAIL, tail."""

    _name = "ws_distill_grad"

    def __init__(self, rows: Rows, logits, teacher, teacher_k, mode, stats, grad_loss,
                 grad_logits, *, tail=None, grad_stride=None):
        n = rows.rows
        a = DistillGradArgs()
        a.grad_stride = _stride(grad_logits, rows, grad_stride)
        a.logits = _matrix("logits", logits, rows, rows.row_stride)
        a.teacher = _buffer("teacher", teacher, rows, _PAIR, 2 * n * teacher_k)
        a.stats = _buffer("stats", stats, rows, _F32, 2 * n)
        a.tail = _buffer("tail", tail, rows, _F32, n)
        a.grad_loss = _buffer("grad_loss", grad_loss, rows, _F32, n)
        a.grad_logits = _matrix("grad_logits", grad_logits, rows, a.grad_stride)
        a.teacher_k = _int32("teacher_k", teacher_k)
        a.mode = _int32("mode", mode)
        self._bind(rows, a, logits, teacher, stats, tail, grad_loss, grad_logits)


def _stride(grad_logits, rows: Rows, given) -> int:
    """The gradient's row stride: as given, a tensor's own, or packed rows."""
    if given is not None:
        return _int64("grad_stride", given)
    if rows.rows > 1 and hasattr(grad_logits, "stride"):
        return grad_logits.stride(0)
    return rows.vocab
