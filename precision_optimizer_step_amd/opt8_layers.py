"""ctypes binding of the operators in include/opt8_layers.h: token embeddings and
their gradient, the RMS norm (with the residual's addition and 8-bit codes) and its
backward pass, the norm and clipping of a list of gradients.

Argument marshalling only, as in `opt8_products`: a make_* function checks torch
tensors and returns the C struct, an opt8_* function queues it on a stream.  Raises
ValueError on a mismatch and Opt8Error on the library's own refusals; no CPU fallback.
"""

import ctypes
import struct

import torch

from . import opt8 as _opt8
from .opt8 import Opt8Error, _check  # noqa: F401
from .opt8_products import (  # noqa: F401
    OPT8_FP8_BLOCK, OPT8_TYPE_BF16, OPT8_TYPE_FP16, OPT8_TYPE_FP32, OPT8_TYPE_E4M3, OPT8_TYPE_E5M2,
    _CODES, _TYPE, _WIDE, _Descriptor, _ceil, _matrix, _on, _placed, _ptr, _queue_on, _scales)

OPT8_ID_INT32 = 0
OPT8_ID_INT64 = 1

OPT8_GRAD_PIECE = 8192
OPT8_GRAD_PIECE_BYTES = 24
OPT8_GRAD_WORKSPACE = 16384

_IDS = {torch.int32: OPT8_ID_INT32, torch.int64: OPT8_ID_INT64}

_P, _L, _I, _F, _D = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_double


class opt8_embedding(_Descriptor):
    _fields_ = [("ids", _P), ("table", _P), ("place_ids", _P), ("place_table", _P), ("y", _P),
                ("tokens", _L), ("vocab", _L), ("places", _L), ("d", _L), ("ldtable", _L), ("ldplace", _L), ("ldy", _L),
                ("scale", _F), ("type", _I), ("id_type", _I)]


class opt8_embedding_grad(_Descriptor):
    _fields_ = [("ids", _P), ("dy", _P), ("dtable", _P), ("workspace", _P), ("workspace_bytes", _L),
                ("tokens", _L), ("vocab", _L), ("d", _L), ("lddy", _L), ("lddtable", _L),
                ("scale", _F), ("type", _I), ("dtable_type", _I), ("id_type", _I), ("accumulate", _I)]


class opt8_rms_norm(_Descriptor):
    _fields_ = [("x", _P), ("residual", _P), ("weight", _P), ("sum", _P), ("y", _P), ("q", _P), ("scale", _P), ("rstd", _P),
                ("rows", _L), ("d", _L), ("ldx", _L), ("ldresidual", _L), ("ldsum", _L), ("ldy", _L), ("ldq", _L),
                ("eps", _F), ("type", _I), ("weight_type", _I), ("q_type", _I)]


class opt8_rms_norm_grad(_Descriptor):
    _fields_ = [("dy", _P), ("x", _P), ("weight", _P), ("rstd", _P), ("dsum", _P), ("dx", _P), ("dweight", _P),
                ("workspace", _P), ("workspace_bytes", _L), ("rows", _L), ("d", _L),
                ("lddy", _L), ("ldx", _L), ("lddsum", _L), ("lddx", _L),
                ("type", _I), ("weight_type", _I), ("dweight_type", _I)]


class opt8_grad(ctypes.Structure):
    _fields_ = [("grad", _P), ("out", _P), ("numel", _L), ("type", _I), ("out_type", _I)]


class opt8_grads(_Descriptor):
    _fields_ = [("table", _P), ("table_bytes", _L), ("squares", _P), ("norm", _P), ("workspace", _P), ("workspace_bytes", _L),
                ("max_norm", _D)]


_CALLS = {"opt8_embedding_forward": opt8_embedding, "opt8_embedding_backward": opt8_embedding_grad,
          "opt8_rms_norm_forward": opt8_rms_norm, "opt8_rms_norm_backward": opt8_rms_norm_grad,
          "opt8_grad_norm": opt8_grads, "opt8_grad_clip": opt8_grads}
_fns = None


def _functions():
    global _fns
    if _fns is None:
        lib = _opt8.lib()
        fns = {}
        for name, kind in _CALLS.items():
            fn = getattr(lib, name)
            fn.argtypes = [ctypes.POINTER(kind), ctypes.c_void_p]
            fn.restype = ctypes.c_int
            fns[name] = fn
        for name, count in (("opt8_embedding_workspace", 3), ("opt8_rms_norm_workspace", 2)):
            fn = getattr(lib, name)
            fn.argtypes = [_L] * count
            fn.restype = _L
            fns[name] = fn
        fn = lib.opt8_grad_table_bytes
        fn.argtypes = [ctypes.c_void_p, _I]
        fn.restype = _L
        fns["opt8_grad_table_bytes"] = fn
        fn = lib.opt8_grad_table
        fn.argtypes = [ctypes.c_void_p, _I, ctypes.c_void_p, _L]
        fn.restype = ctypes.c_int
        fns["opt8_grad_table"] = fn
        _fns = fns
    return _fns


# ----------------------------------------------------------------------------- checks
def _vector(what, t, dtypes, n):
    if t.shape == (n,) and t.dtype in dtypes and t.is_contiguous():
        return
    if t.dtype not in dtypes:
        raise ValueError(f"{what}: dtype {t.dtype} not allowed here (expected one of "
                         f"{', '.join(str(d) for d in dtypes)})")
    if t.shape != (n,):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected ({n},)")
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")


def _work(workspace):
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace: must be contiguous torch.uint8")


def _dim2(what, t):
    if t.dim() != 2:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected a matrix")


# ----------------------------------------------------------------------------- embeddings
def make_embedding(ids, table, y, scale=1.0, place_ids=None, place_table=None) -> opt8_embedding:
    """y [tokens, d] = scale * table[ids] (+ place_table[place_ids]) for ids int32 or int64
    [tokens] and tables [rows, d], all matrices bf16, fp16 or fp32.  An id outside its table
    (a padding of -1) stands for a row of zeros."""
    _dim2("table", table)
    vocab, d = table.shape
    tokens = ids.numel()
    if table.dtype not in _WIDE:
        raise ValueError(f"table: dtype {table.dtype} not allowed here (expected one of {', '.join(str(t) for t in _WIDE)})")
    kind = (table.dtype,)
    _vector("ids", ids, tuple(_IDS), tokens)
    ldtable = _matrix("table", table, kind, vocab, d)
    ldy = _matrix("y", y, kind, tokens, d)
    places, ldplace = 0, d
    if (place_ids is None) != (place_table is None):
        raise ValueError("place_ids and place_table go together")
    if place_table is not None:
        _dim2("place_table", place_table)
        places = place_table.shape[0]
        _vector("place_ids", place_ids, (ids.dtype,), tokens)
        ldplace = _matrix("place_table", place_table, kind, places, d)
    device = _placed(("ids", "table", "y", "place_ids", "place_table"), (ids, table, y, place_ids, place_table))
    return _on(device, opt8_embedding(ids.data_ptr(), table.data_ptr(), _ptr(place_ids), _ptr(place_table), y.data_ptr(),
                                      tokens, vocab, places, d, ldtable, ldplace, ldy, scale, _TYPE[table.dtype],
                                      _IDS[ids.dtype]))


def make_embedding_grad(ids, dy, dtable, workspace, scale=1.0, accumulate=False) -> opt8_embedding_grad:
    """dtable [vocab, d] = scale * (sums of dy [tokens, d] over the tokens of each id), with zeros
    in rows without a token; or, with accumulate, added to the rows that have one.  dtable: dy's
    type or fp32.  workspace: a contiguous uint8 tensor of at least
    opt8_embedding_workspace(tokens, vocab, d) bytes, one for each call that may run at the same time."""
    _dim2("dtable", dtable)
    vocab, d = dtable.shape
    tokens = ids.numel()
    _vector("ids", ids, tuple(_IDS), tokens)
    lddy = _matrix("dy", dy, _WIDE, tokens, d)
    lddtable = _matrix("dtable", dtable, (dy.dtype, torch.float32), vocab, d)
    _work(workspace)
    device = _placed(("ids", "dy", "dtable", "workspace"), (ids, dy, dtable, workspace))
    return _on(device, opt8_embedding_grad(ids.data_ptr(), dy.data_ptr(), dtable.data_ptr(), workspace.data_ptr(),
                                           workspace.numel(), tokens, vocab, d, lddy, lddtable, scale, _TYPE[dy.dtype],
                                           _TYPE[dtable.dtype], _IDS[ids.dtype], bool(accumulate)))


def opt8_embedding_workspace(tokens: int, vocab: int, d: int) -> int:
    """Bytes of workspace that the embedding's gradient needs."""
    return int(_functions()["opt8_embedding_workspace"](int(tokens), int(vocab), int(d)))


# ----------------------------------------------------------------------------- RMS norm
def make_rms_norm(x, weight, y=None, q=None, scale=None, rstd=None, residual=None, sum=None, eps=1e-6) -> opt8_rms_norm:
    """The norm of t = x + residual (or x) [rows, d], times weight [d] (x's type or fp32): y of x's
    type; q (float8_e4m3fn or float8_e5m2, rows a multiple of 16 bytes apart) with scale float32
    [ceil(d/128), rows], as operand a of the 8-bit product; rstd float32 [rows] for the backward
    pass; sum receives t.  Outputs may be None, not all; sum may be x or residual itself."""
    _dim2("x", x)
    rows, d = x.shape
    ldx = _matrix("x", x, _WIDE, rows, d)
    kind = (x.dtype,)
    _vector("weight", weight, (x.dtype, torch.float32), d)
    ldresidual = ldsum = ldy = d
    ldq = q_type = 0
    if residual is not None:
        ldresidual = _matrix("residual", residual, kind, rows, d)
    if sum is not None:
        if residual is None:
            raise ValueError("sum goes with a residual")
        ldsum = _matrix("sum", sum, kind, rows, d)
    if y is not None:
        ldy = _matrix("y", y, kind, rows, d)
    if (q is None) != (scale is None):
        raise ValueError("q and scale go together")
    if q is not None:
        ldq = _matrix("q", q, _CODES, rows, d, owned=True)
        q_type = _TYPE[q.dtype]
        _scales("scale", scale, _ceil(d), rows)
    if rstd is not None:
        _vector("rstd", rstd, (torch.float32,), rows)
    device = _placed(("x", "weight", "y", "q", "scale", "rstd", "residual", "sum"),
                     (x, weight, y, q, scale, rstd, residual, sum))
    return _on(device, opt8_rms_norm(x.data_ptr(), _ptr(residual), weight.data_ptr(), _ptr(sum), _ptr(y), _ptr(q), _ptr(scale),
                                     _ptr(rstd), rows, d, ldx, ldresidual, ldsum, ldy, ldq, eps, _TYPE[x.dtype],
                                     _TYPE[weight.dtype], q_type))


def make_rms_norm_grad(dy, x, weight, rstd, dx, dweight, workspace=None, dsum=None) -> opt8_rms_norm_grad:
    """dx [rows, d] and dweight [d] of the norm from dy, the rows x that it normalised (the forward
    pass's sum where it had a residual) and its rstd; dsum, if given, is added to dx.  dx or dweight
    may be None; dx may be dy or dsum itself.  dweight: x's type or fp32.  workspace (for dweight):
    a contiguous uint8 tensor of at least opt8_rms_norm_workspace(rows, d) bytes, one for each call
    that may run at the same time."""
    _dim2("x", x)
    rows, d = x.shape
    ldx = _matrix("x", x, _WIDE, rows, d)
    kind = (x.dtype,)
    lddy = _matrix("dy", dy, kind, rows, d)
    _vector("weight", weight, (x.dtype, torch.float32), d)
    _vector("rstd", rstd, (torch.float32,), rows)
    if dx is None and dweight is None:
        raise ValueError("dx and dweight are both None")
    lddx = lddsum = d
    if dx is not None:
        lddx = _matrix("dx", dx, kind, rows, d)
    if dsum is not None:
        lddsum = _matrix("dsum", dsum, kind, rows, d)
    dweight_type = x.dtype
    if dweight is not None:
        _vector("dweight", dweight, (x.dtype, torch.float32), d)
        dweight_type = dweight.dtype
        if workspace is None:
            raise ValueError("workspace: needed for dweight")
    if workspace is not None:
        _work(workspace)
    device = _placed(("x", "dy", "weight", "rstd", "dx", "dweight", "workspace", "dsum"),
                     (x, dy, weight, rstd, dx, dweight, workspace, dsum))
    return _on(device, opt8_rms_norm_grad(dy.data_ptr(), x.data_ptr(), weight.data_ptr(), rstd.data_ptr(), _ptr(dsum), _ptr(dx),
                                          _ptr(dweight), _ptr(workspace), 0 if workspace is None else workspace.numel(),
                                          rows, d, lddy, ldx, lddsum, lddx, _TYPE[x.dtype], _TYPE[weight.dtype],
                                          _TYPE[dweight_type]))


def opt8_rms_norm_workspace(rows: int, d: int) -> int:
    """Bytes of workspace that the norm's backward pass needs for dweight."""
    return int(_functions()["opt8_rms_norm_workspace"](int(rows), int(d)))


# ----------------------------------------------------------------------------- gradients of a list
def _flat(what, t, device):
    if t.dtype not in _TYPE or t.dtype not in _WIDE:
        raise ValueError(f"{what}: dtype {t.dtype} not allowed here (expected one of {', '.join(str(d) for d in _WIDE)})")
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    if t.get_device() != device:
        raise ValueError(f"{what}: on {t.device}, but the first gradient is on "
                         f"{'cpu' if device < 0 else f'cuda:{device}'}")


def opt8_grad_table(grads, outs=None) -> torch.Tensor:
    """The table of a list of gradients (contiguous bf16, fp16 or fp32 tensors of any shapes on the
    current device), as a uint8 tensor beside them: made once, and passed to make_grads while the
    gradients stay at their addresses.  outs: where the clipped values go, one tensor (of any of the
    types) or None, for in place, to a gradient.  Raises Opt8Error where buffers overlap."""
    grads = list(grads)
    outs = [None] * len(grads) if outs is None else list(outs)
    if len(outs) != len(grads):
        raise ValueError(f"outs: {len(outs)} of them for {len(grads)} gradients")
    device = grads[0].get_device() if grads else torch.cuda.current_device()
    fields = []
    for i, (g, o) in enumerate(zip(grads, outs)):
        _flat(f"gradient {i}", g, device)
        kind = _TYPE[g.dtype]
        if o is None:
            fields += (g.data_ptr(), 0, g.numel(), kind, kind)
        else:
            _flat(f"out {i}", o, device)
            if o.numel() != g.numel():
                raise ValueError(f"out {i}: holds {o.numel()} elements, its gradient {g.numel()}")
            fields += (g.data_ptr(), o.data_ptr(), g.numel(), kind, _TYPE[o.dtype])
    if device < 0:
        raise ValueError(f"gradient 0: on {grads[0].device}; the operators run on a GPU")
    if device != torch.cuda.current_device():
        raise ValueError(f"gradient 0: on cuda:{device}, but the current device is cuda:{torch.cuda.current_device()}")
    fns = _functions()
    listed = struct.pack("=" + "QQqii" * len(grads), *fields)
    size = fns["opt8_grad_table_bytes"](listed, len(grads))
    if size < 0:
        _check(int(size))
    table = bytearray(size)
    _check(fns["opt8_grad_table"](listed, len(grads), (ctypes.c_char * size).from_buffer(table), size))
    return torch.frombuffer(table, dtype=torch.uint8).to(f"cuda:{device}")


def make_grads(table, squares, norm=None, workspace=None, max_norm=1.0) -> opt8_grads:
    """The list of a table for opt8_grad_norm and opt8_grad_clip: squares float64 [1], norm float32
    [1] or None, workspace (for opt8_grad_norm) a contiguous uint8 tensor of at least
    OPT8_GRAD_WORKSPACE bytes, one for each call that may run at the same time.  The descriptor keeps
    the table (the kernels go where it says)."""
    if table.dtype != torch.uint8 or table.dim() != 1 or not table.is_contiguous():
        raise ValueError("table: expected what opt8_grad_table returned")
    _vector("squares", squares, (torch.float64,), 1)
    if norm is not None:
        _vector("norm", norm, (torch.float32,), 1)
    if workspace is not None:
        _work(workspace)
    device = _placed(("squares", "table", "norm", "workspace"), (squares, table, norm, workspace))
    desc = _on(device, opt8_grads(table.data_ptr(), table.numel(), squares.data_ptr(), _ptr(norm),
                                  _ptr(workspace), 0 if workspace is None else workspace.numel(), max_norm))
    desc.kept = table
    return desc


# ----------------------------------------------------------------------------- calls
def _call(name, desc, stream, check):
    handle = _queue_on(desc, stream)
    rc = (_fns or _functions())[name](desc, handle or None)
    return _check(rc) if check and rc else rc


def opt8_embedding_forward(embedding: opt8_embedding, stream=None, check: bool = True) -> int:
    """Queue the lookup on a stream of the tensors' device, which has to be the current one (a
    torch.cuda.Stream, a raw handle, or None for torch's current stream); the tensors must live
    until it has run."""
    return _call("opt8_embedding_forward", embedding, stream, check)


def opt8_embedding_backward(grad: opt8_embedding_grad, stream=None, check: bool = True) -> int:
    """Queue the embedding's gradient; arguments as for opt8_embedding_forward."""
    return _call("opt8_embedding_backward", grad, stream, check)


def opt8_rms_norm_forward(norm: opt8_rms_norm, stream=None, check: bool = True) -> int:
    """Queue the norm; arguments as for opt8_embedding_forward."""
    return _call("opt8_rms_norm_forward", norm, stream, check)


def opt8_rms_norm_backward(grad: opt8_rms_norm_grad, stream=None, check: bool = True) -> int:
    """Queue the norm's backward pass; arguments as for opt8_embedding_forward."""
    return _call("opt8_rms_norm_backward", grad, stream, check)


def opt8_grad_norm(grads: opt8_grads, stream=None, check: bool = True) -> int:
    """Queue squares = the sum of the list's squares and norm = its root; arguments as for
    opt8_embedding_forward (the gradients themselves must live too)."""
    return _call("opt8_grad_norm", grads, stream, check)


def opt8_grad_clip(grads: opt8_grads, stream=None, check: bool = True) -> int:
    """Queue the clipping of the list to max_norm, by the norm that `squares` says; arguments as for
    opt8_grad_norm."""
    return _call("opt8_grad_clip", grads, stream, check)
