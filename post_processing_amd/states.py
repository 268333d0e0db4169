"""Python binding of the operators over rows of hidden states
(include/ws_states.h): embedding lookup and its gradient, layer norm and its
gradients.

Argument marshalling only, as in ``ws``.  Call objects are those of ``logits``:
each binds its configuration and buffers once and enqueues the operator each
time ``run`` is called, on the buffers' contents of that moment, and the same
holds of buffers, streams, graphs and workspaces:

    shape = make_states(rows=T, width=D, dtype=ws.DTYPE_BF16)
    call = LayerNorm(shape, x, y, weight=weight, bias=bias)
    call.run(stream)
"""
from __future__ import annotations

from ctypes import POINTER, Structure, byref, c_float, c_int, c_int32, c_int64, c_size_t, c_void_p

from . import logits, ws
from .logits import _F32, _I32, _LOGIT_TYPES, _buffer, _Call, _check, _int32, _int64

MAX_WIDTH = 1 << 20
MAX_TOKENS = 1 << 24


class States(Structure):
    _fields_ = [("device", c_int32), ("dtype", c_int32), ("rows", c_int32), ("width", c_int32),
                ("row_stride", c_int64)]


class NormStats(Structure):
    _fields_ = [("mean", c_float), ("inverse", c_float)]


class EmbedArgs(Structure):
    _fields_ = [("table", c_void_p), ("table_stride", c_int64), ("ids", c_void_p),
                ("out", c_void_p), ("vocab", c_int32), ("scale", c_float)]


class EmbedGradArgs(Structure):
    _fields_ = [("grad_out", c_void_p), ("ids", c_void_p), ("grad_table", c_void_p),
                ("grad_stride", c_int64), ("workspace", c_void_p), ("workspace_bytes", c_size_t),
                ("vocab", c_int32), ("grad_dtype", c_int32), ("accumulate", c_int32),
                ("scale", c_float)]


class LayerNormArgs(Structure):
    _fields_ = [("x", c_void_p), ("weight", c_void_p), ("bias", c_void_p), ("y", c_void_p),
                ("y_stride", c_int64), ("stats", c_void_p), ("weight_dtype", c_int32),
                ("eps", c_float)]


class LayerNormGradArgs(Structure):
    _fields_ = [("x", c_void_p), ("stats", c_void_p), ("weight", c_void_p), ("grad_y", c_void_p),
                ("grad_y_stride", c_int64), ("grad_x", c_void_p), ("grad_x_stride", c_int64),
                ("grad_weight", c_void_p), ("grad_bias", c_void_p), ("workspace", c_void_p),
                ("workspace_bytes", c_size_t), ("weight_dtype", c_int32), ("reserved", c_int32)]


_lib = None


def load():
    """The lane library with this header's prototypes set."""
    global _lib
    if _lib is not None:
        return _lib
    lib = logits.load()
    lib.ws_embed.argtypes = [POINTER(States), POINTER(EmbedArgs), c_void_p]
    lib.ws_embed_grad_workspace.argtypes = [POINTER(States), c_int32, POINTER(c_size_t)]
    lib.ws_embed_grad.argtypes = [POINTER(States), POINTER(EmbedGradArgs), c_void_p]
    lib.ws_layernorm.argtypes = [POINTER(States), POINTER(LayerNormArgs), c_void_p]
    lib.ws_layernorm_grad_workspace.argtypes = [POINTER(States), POINTER(c_size_t)]
    lib.ws_layernorm_grad.argtypes = [POINTER(States), POINTER(LayerNormGradArgs), c_void_p]
    for name in ("ws_embed", "ws_embed_grad_workspace", "ws_embed_grad", "ws_layernorm",
                 "ws_layernorm_grad_workspace", "ws_layernorm_grad"):
        getattr(lib, name).restype = c_int
    _lib = lib
    return lib


def make_states(*, rows, width, dtype=ws.DTYPE_F32, row_stride=None, device=0) -> States:
    t = States()
    t.device = _int32("device", device)
    t.dtype = _int32("dtype", dtype)
    t.rows = _int32("rows", rows)
    t.width = _int32("width", width)
    t.row_stride = _int64("row_stride", width if row_stride is None else row_stride)
    return t


def embed_grad_workspace(states: States, vocab: int) -> int:
    """Bytes of workspace ws_embed_grad needs for these rows and this vocabulary."""
    n = c_size_t(0)
    _check(load().ws_embed_grad_workspace(byref(states), _int32("vocab", vocab), byref(n)),
           "ws_embed_grad_workspace")
    return n.value


def layernorm_grad_workspace(states: States) -> int:
    """Bytes of workspace ws_layernorm_grad needs for gradients of weight or bias."""
    n = c_size_t(0)
    _check(load().ws_layernorm_grad_workspace(byref(states), byref(n)),
           "ws_layernorm_grad_workspace")
    return n.value


def _rows(name, x, device, dtype, rows, width, stride) -> int | None:
    """Address of a [rows][width] matrix whose rows lie `stride` apart."""
    if x is not None and hasattr(x, "data_ptr") and hasattr(x, "dtype"):
        if str(x.dtype) != _LOGIT_TYPES.get(dtype):
            raise ValueError(f"{name}: {x.dtype}, expected {_LOGIT_TYPES.get(dtype)}")
        if not x.is_cuda or x.device.index != device:
            raise ValueError(f"{name} is on {x.device}, expected cuda:{device}")
        if x.dim() != 2 or tuple(x.shape) != (rows, width):
            raise ValueError(f"{name}: shape {tuple(x.shape)}, expected {(rows, width)}")
        if (width > 1 and x.stride(1) != 1) or (rows > 1 and x.stride(0) != stride):
            raise ValueError(f"{name}: strides {x.stride()}, expected ({stride}, 1)")
    return ws._addr(x)


def _stride(name, x, rows, width, given) -> int:
    """A matrix's row stride: as given, a tensor's own, or packed rows."""
    if given is not None:
        return _int64(name, given)
    if rows > 1 and hasattr(x, "stride"):
        return x.stride(0)
    return width


def _column(name, x, states: States, dtype) -> int | None:
    """Address of a [width] vector of `dtype`."""
    return _buffer(name, x, states, (_LOGIT_TYPES.get(dtype),), states.width)


class Embed(_Call):
    """ws_embed: out[r] = scale * table[ids[r]]; `states` describes `out`."""

    _name = "ws_embed"

    def __init__(self, states: States, table, ids, out, *, vocab, table_stride=None, scale=1.0):
        load()
        a = EmbedArgs()
        a.vocab = _int32("vocab", vocab)
        a.table_stride = _stride("table_stride", table, vocab, states.width, table_stride)
        a.table = _rows("table", table, states.device, states.dtype, vocab, states.width,
                        a.table_stride)
        a.ids = _buffer("ids", ids, states, _I32, states.rows)
        a.out = _rows("out", out, states.device, states.dtype, states.rows, states.width,
                      states.row_stride)
        a.scale = scale
        self._bind(states, a, table, ids, out)


class EmbedGrad(_Call):
    """ws_embed_grad: the gradient of Embed's table, written whole or, with
    `accumulate`, added to what it holds; `states` describes `grad_out`."""

    _name = "ws_embed_grad"

    def __init__(self, states: States, grad_out, ids, grad_table, *, vocab, grad_stride=None,
                 grad_dtype=None, accumulate=False, scale=1.0, workspace=None):
        load()
        a = EmbedGradArgs()
        a.vocab = _int32("vocab", vocab)
        a.grad_dtype = states.dtype if grad_dtype is None else _int32("grad_dtype", grad_dtype)
        a.grad_stride = _stride("grad_stride", grad_table, vocab, states.width, grad_stride)
        a.grad_out = _rows("grad_out", grad_out, states.device, states.dtype, states.rows,
                           states.width, states.row_stride)
        a.ids = _buffer("ids", ids, states, _I32, states.rows)
        a.grad_table = _rows("grad_table", grad_table, states.device, a.grad_dtype, vocab,
                             states.width, a.grad_stride)
        a.accumulate = 1 if accumulate else 0
        a.scale = scale
        workspace = self._own_workspace(states, a, workspace, embed_grad_workspace(states, vocab))
        self._bind(states, a, grad_out, ids, grad_table, workspace)


class LayerNorm(_Call):
    """ws_layernorm: y of every row and, with `stats` ([rows][2] float32), what
    LayerNormGrad needs of it; `states` describes `x`."""

    _name = "ws_layernorm"

    def __init__(self, states: States, x, y, *, weight=None, bias=None, weight_dtype=None,
                 eps=1e-5, stats=None, y_stride=None):
        load()
        n, width = states.rows, states.width
        a = LayerNormArgs()
        a.weight_dtype = states.dtype if weight_dtype is None else _int32("weight_dtype",
                                                                          weight_dtype)
        a.y_stride = _stride("y_stride", y, n, width, y_stride)
        a.x = _rows("x", x, states.device, states.dtype, n, width, states.row_stride)
        a.y = _rows("y", y, states.device, states.dtype, n, width, a.y_stride)
        a.weight = _column("weight", weight, states, a.weight_dtype)
        a.bias = _column("bias", bias, states, a.weight_dtype)
        a.stats = _buffer("stats", stats, states, _F32, 2 * n)
        a.eps = eps
        self._bind(states, a, x, y, weight, bias, stats)


class LayerNormGrad(_Call):
    """ws_layernorm_grad: the gradients of LayerNorm's rows, weight and bias,
    those of the three that are given; `states` describes `x`."""

    _name = "ws_layernorm_grad"

    def __init__(self, states: States, x, stats, grad_y, *, weight=None, weight_dtype=None,
                 grad_x=None, grad_weight=None, grad_bias=None, grad_y_stride=None,
                 grad_x_stride=None, workspace=None):
        load()
        n, width = states.rows, states.width
        a = LayerNormGradArgs()
        a.weight_dtype = states.dtype if weight_dtype is None else _int32("weight_dtype",
                                                                          weight_dtype)
        a.grad_y_stride = _stride("grad_y_stride", grad_y, n, width, grad_y_stride)
        a.x = _rows("x", x, states.device, states.dtype, n, width, states.row_stride)
        a.stats = _buffer("stats", stats, states, _F32, 2 * n)
        a.grad_y = _rows("grad_y", grad_y, states.device, states.dtype, n, width, a.grad_y_stride)
        a.weight = _column("weight", weight, states, a.weight_dtype)
        if grad_x is not None:
            a.grad_x_stride = _stride("grad_x_stride", grad_x, n, width, grad_x_stride)
            a.grad_x = _rows("grad_x", grad_x, states.device, states.dtype, n, width,
                             a.grad_x_stride)
        a.grad_weight = _column("grad_weight", grad_weight, states, a.weight_dtype)
        a.grad_bias = _column("grad_bias", grad_bias, states, a.weight_dtype)
        need = 0
        if grad_weight is not None or grad_bias is not None:
            need = layernorm_grad_workspace(states)
        workspace = self._own_workspace(states, a, workspace, need)
        self._bind(states, a, x, stats, grad_y, weight, grad_x, grad_weight, grad_bias, workspace)
