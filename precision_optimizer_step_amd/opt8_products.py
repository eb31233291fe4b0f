"""ctypes binding of the operators in include/opt8_products.h: 8-bit block-scaled
quantiser and matrix product, gated feed-forward block and its backward pass.

Argument marshalling only, as in `opt8`: a make_* function checks torch tensors
(the library can check alignment, sizes and overlap only) and returns the C
struct, an opt8_* function queues it on a stream.  Raises ValueError on a
mismatch and Opt8Error on the library's own refusals; no CPU fallback.
"""

import ctypes

import torch

from . import opt8 as _opt8
from .opt8 import Opt8Error, _check, _stream_handle  # noqa: F401

OPT8_FP8_BLOCK = 128

OPT8_TYPE_BF16 = 0
OPT8_TYPE_FP16 = 1
OPT8_TYPE_FP32 = 2
OPT8_TYPE_E4M3 = 3
OPT8_TYPE_E5M2 = 4

OPT8_FP8_BLOCK_ROW = 0
OPT8_FP8_BLOCK_TILE = 1

OPT8_ACT_SILU = 0
OPT8_ACT_GELU = 1
OPT8_ACT_GELU_TANH = 2

_TYPE = {torch.bfloat16: OPT8_TYPE_BF16, torch.float16: OPT8_TYPE_FP16, torch.float32: OPT8_TYPE_FP32,
         torch.float8_e4m3fn: OPT8_TYPE_E4M3, torch.float8_e5m2: OPT8_TYPE_E5M2}
_WIDE = (torch.bfloat16, torch.float16, torch.float32)
_HALF = (torch.bfloat16, torch.float16)
_CODES = (torch.float8_e4m3fn, torch.float8_e5m2)

_P, _L, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


class _Descriptor(ctypes.Structure):
    device = None     # index of the GPU that the tensors are on; None in a struct filled by hand


class opt8_fp8_quant(_Descriptor):
    _fields_ = [("x", _P), ("q", _P), ("scale", _P), ("qt", _P), ("scale_t", _P),
                ("rows", _L), ("cols", _L), ("ldx", _L), ("ldq", _L), ("ldt", _L),
                ("x_type", _I), ("q_type", _I), ("block", _I)]


class opt8_fp8_product(_Descriptor):
    _fields_ = [("a", _P), ("scale_a", _P), ("b", _P), ("scale_b", _P), ("c", _P),
                ("m", _L), ("n", _L), ("k", _L), ("lda", _L), ("ldb", _L), ("ldc", _L),
                ("a_type", _I), ("b_type", _I), ("c_type", _I), ("block_b", _I)]


class opt8_gated_ffn(_Descriptor):
    _fields_ = [("x", _P), ("w_gate", _P), ("w_up", _P), ("h", _P), ("gate", _P), ("up", _P),
                ("rows", _L), ("d", _L), ("f", _L), ("ldx", _L), ("ldw", _L), ("ldh", _L), ("ldg", _L),
                ("type", _I), ("act", _I)]


class opt8_gated_ffn_grad(_Descriptor):
    _fields_ = [("dh", _P), ("x", _P), ("w_gate", _P), ("w_up", _P), ("gate", _P), ("up", _P),
                ("dx", _P), ("dw_gate", _P), ("dw_up", _P), ("workspace", _P), ("workspace_bytes", _L),
                ("rows", _L), ("d", _L), ("f", _L), ("ldx", _L), ("ldw", _L), ("lddh", _L), ("ldg", _L),
                ("lddx", _L), ("lddw", _L), ("type", _I), ("act", _I)]


_CALLS = {"opt8_fp8_quantize": opt8_fp8_quant, "opt8_fp8_matmul": opt8_fp8_product,
          "opt8_gated_ffn_forward": opt8_gated_ffn, "opt8_gated_ffn_backward": opt8_gated_ffn_grad}
_fns = None


def _functions():
    global _fns
    if _fns is None:
        lib = _opt8.lib()
        fns = {}
        for name, struct in _CALLS.items():
            fn = getattr(lib, name)
            fn.argtypes = [ctypes.POINTER(struct), ctypes.c_void_p]
            fn.restype = ctypes.c_int
            fns[name] = fn
        fn = lib.opt8_gated_ffn_workspace
        fn.argtypes = [_L, _L, _L]
        fn.restype = _L
        fns["workspace"] = fn
        _fns = fns
    return _fns


# ----------------------------------------------------------------------------- checks
def _matrix(what, t, dtypes, rows, cols, owned=False):
    """The row distance of a [rows, cols] torch matrix with dense rows.  owned: the
    last row's last 16 bytes must belong to the tensor's storage whole (the library
    reads rows in pieces of 16)."""
    if t.dtype not in dtypes:
        raise ValueError(f"{what}: dtype {t.dtype} not allowed here (expected one of "
                         f"{', '.join(str(d) for d in dtypes)})")
    if t.shape != (rows, cols):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected ({rows}, {cols})")
    step, unit = t.stride()
    if cols > 1 and unit != 1:
        raise ValueError(f"{what}: the values of a row must be adjacent (strides {t.stride()})")
    if rows > 1 and step < cols:
        raise ValueError(f"{what}: rows overlap (strides {t.stride()})")
    if rows <= 1:
        # a single row's distance is arbitrary: the smallest that keeps 16-byte rows
        each = max(1, 16 // t.element_size())
        step = -(-cols // each) * each if owned else cols
    if owned and rows and cols:
        each = 16 // t.element_size()
        end = t.storage_offset() + (rows - 1) * step + -(-cols // each) * each
        if end > t.untyped_storage().nbytes() // t.element_size():
            raise ValueError(f"{what}: its storage ends inside the last 16 bytes of the last row")
    return step


def _scales(what, t, blocks, across):
    if t.dtype != torch.float32:
        raise ValueError(f"{what}: dtype {t.dtype} not allowed here (expected torch.float32)")
    if t.shape != (blocks, across):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected ({blocks}, {across})")
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")


def _placed(names, tensors):
    """The one GPU that all are on, and that one current (a call queues on the current device)."""
    first = tensors[0].get_device()
    for i, t in enumerate(tensors):
        if t is not None and t.get_device() != first:
            raise ValueError(f"{names[i]}: on {t.device}, but {names[0]} is on {tensors[0].device}")
    if first < 0:
        raise ValueError(f"{names[0]}: on {tensors[0].device}; the operators run on a GPU")
    if first != torch.cuda.current_device():
        raise ValueError(f"{names[0]}: on cuda:{first}, but the current device is cuda:{torch.cuda.current_device()}")
    return first


def _on(device, desc):
    desc.device = device
    return desc


def _ceil(n):
    return -(-n // OPT8_FP8_BLOCK)


def _ptr(t):
    return None if t is None else t.data_ptr()


# ----------------------------------------------------------------------------- 8-bit operands
def make_fp8_quant(x, q=None, scale=None, qt=None, scale_t=None, block=OPT8_FP8_BLOCK_ROW) -> opt8_fp8_quant:
    """Codes and scales of x [rows, cols], of its transpose (qt, scale_t), or of both.

    x: bf16, fp16 or fp32.  q [rows, cols], qt [cols, rows]: torch.float8_e4m3fn or
    float8_e5m2, rows a multiple of 16 bytes apart.  scale float32 [ceil(cols/128),
    rows] (block ROW) or [ceil(cols/128), ceil(rows/128)] (TILE); scale_t the same
    for the transpose.
    """
    if x.dim() != 2:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected a matrix")
    rows, cols = x.shape
    ldx = _matrix("x", x, _WIDE, rows, cols)
    if block not in (OPT8_FP8_BLOCK_ROW, OPT8_FP8_BLOCK_TILE):
        raise ValueError(f"unknown block {block}")
    if q is None and qt is None:
        raise ValueError("q and qt are both None")
    tile = block == OPT8_FP8_BLOCK_TILE
    ldq = ldt = 0
    kind = None
    for what, t, s, r, c in (("q", q, scale, rows, cols), ("qt", qt, scale_t, cols, rows)):
        if (t is None) != (s is None):
            raise ValueError(f"{what} and its scales go together")
        if t is None:
            continue
        ld = _matrix(what, t, _CODES, r, c, owned=True)
        _scales("scale" if what == "q" else "scale_t", s, _ceil(c), _ceil(r) if tile else r)
        if kind is not None and t.dtype != kind:
            raise ValueError("q and qt have different types")
        kind = t.dtype
        if what == "q":
            ldq = ld
        else:
            ldt = ld
    device = _placed(("x", "q", "scale", "qt", "scale_t"), (x, q, scale, qt, scale_t))
    return _on(device, opt8_fp8_quant(x.data_ptr(), _ptr(q), _ptr(scale), _ptr(qt), _ptr(scale_t), rows, cols, ldx, ldq,
                                      ldt, _TYPE[x.dtype], _TYPE[kind], block))


def make_fp8_product(a, scale_a, b, scale_b, c, block_b=OPT8_FP8_BLOCK_TILE) -> opt8_fp8_product:
    """c [m, n] = a b^T for codes a [m, k] (e4m3 or e5m2, ROW scales) and b [n, k] (e4m3,
    scales by block_b), scales as opt8_fp8_quantize lays them out; c bf16 or fp16."""
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError(f"a, b: shapes {tuple(a.shape)}, {tuple(b.shape)}, expected matrices")
    (m, k), n = a.shape, b.shape[0]
    if block_b not in (OPT8_FP8_BLOCK_ROW, OPT8_FP8_BLOCK_TILE):
        raise ValueError(f"unknown block {block_b}")
    lda = _matrix("a", a, _CODES, m, k, owned=True)
    ldb = _matrix("b", b, _CODES[:1], n, k, owned=True)
    ldc = _matrix("c", c, _HALF, m, n)
    _scales("scale_a", scale_a, _ceil(k), m)
    _scales("scale_b", scale_b, _ceil(k), _ceil(n) if block_b == OPT8_FP8_BLOCK_TILE else n)
    device = _placed(("a", "scale_a", "b", "scale_b", "c"), (a, scale_a, b, scale_b, c))
    return _on(device, opt8_fp8_product(a.data_ptr(), scale_a.data_ptr(), b.data_ptr(), scale_b.data_ptr(), c.data_ptr(), m,
                                        n, k, lda, ldb, ldc, _TYPE[a.dtype], _TYPE[b.dtype], _TYPE[c.dtype], block_b))


# ----------------------------------------------------------------------------- gated feed-forward block
def _weights(w_gate, w_up, x):
    if w_gate.dim() != 2 or x.dim() != 2:
        raise ValueError(f"x, w_gate: shapes {tuple(x.shape)}, {tuple(w_gate.shape)}, expected matrices")
    rows, d = x.shape
    f = w_gate.shape[0]
    if x.dtype not in _HALF:
        raise ValueError(f"x: dtype {x.dtype} not allowed here (expected one of {', '.join(str(t) for t in _HALF)})")
    kind = (x.dtype,)
    ldx = _matrix("x", x, kind, rows, d, owned=True)
    ldw = _matrix("w_gate", w_gate, kind, f, d, owned=True)
    if _matrix("w_up", w_up, kind, f, d, owned=True) != ldw:
        raise ValueError("w_gate and w_up have different row distances")
    return rows, d, f, kind, ldx, ldw


def make_gated_ffn(x, w_gate, w_up, h, gate=None, up=None, act=OPT8_ACT_SILU) -> opt8_gated_ffn:
    """h = act(x w_gate^T) * (x w_up^T) for x [rows, d], weights [f, d], all bf16 or all
    fp16; gate and up [rows, f] receive the two projections for the backward pass."""
    rows, d, f, kind, ldx, ldw = _weights(w_gate, w_up, x)
    ldh = _matrix("h", h, kind, rows, f)
    if (gate is None) != (up is None):
        raise ValueError("gate and up go together")
    ldg = f
    if gate is not None:
        ldg = _matrix("gate", gate, kind, rows, f)
        if _matrix("up", up, kind, rows, f) != ldg:
            raise ValueError("gate and up have different row distances")
    device = _placed(("x", "w_gate", "w_up", "h", "gate", "up"), (x, w_gate, w_up, h, gate, up))
    return _on(device, opt8_gated_ffn(x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), h.data_ptr(), _ptr(gate), _ptr(up),
                                      rows, d, f, ldx, ldw, ldh, ldg, _TYPE[x.dtype], act))


def make_gated_ffn_grad(dh, x, w_gate, w_up, gate, up, dx, dw_gate, dw_up, workspace,
                        act=OPT8_ACT_SILU) -> opt8_gated_ffn_grad:
    """Gradients of the block from dh [rows, f] and the stored gate and up: dx [rows, d]
    and dw_gate, dw_up [f, d] (dx, or both dw, may be None).  workspace: a contiguous
    uint8 tensor of at least opt8_gated_ffn_workspace(rows, d, f) bytes, one for each call
    that may run at the same time."""
    rows, d, f, kind, ldx, ldw = _weights(w_gate, w_up, x)
    lddh = _matrix("dh", dh, kind, rows, f, owned=True)
    ldg = _matrix("gate", gate, kind, rows, f, owned=True)
    if _matrix("up", up, kind, rows, f, owned=True) != ldg:
        raise ValueError("gate and up have different row distances")
    if (dw_gate is None) != (dw_up is None):
        raise ValueError("dw_gate and dw_up go together")
    if dx is None and dw_gate is None:
        raise ValueError("dx and both dw are None")
    lddx, lddw = d, d
    if dx is not None:
        lddx = _matrix("dx", dx, kind, rows, d)
    if dw_gate is not None:
        lddw = _matrix("dw_gate", dw_gate, kind, f, d)
        if _matrix("dw_up", dw_up, kind, f, d) != lddw:
            raise ValueError("dw_gate and dw_up have different row distances")
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace: must be contiguous torch.uint8")
    device = _placed(("x", "dh", "w_gate", "w_up", "gate", "up", "dx", "dw_gate", "dw_up", "workspace"),
                     (x, dh, w_gate, w_up, gate, up, dx, dw_gate, dw_up, workspace))
    return _on(device, opt8_gated_ffn_grad(dh.data_ptr(), x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), gate.data_ptr(),
                                           up.data_ptr(), _ptr(dx), _ptr(dw_gate), _ptr(dw_up), workspace.data_ptr(),
                                           workspace.numel(), rows, d, f, ldx, ldw, lddh, ldg, lddx, lddw, _TYPE[x.dtype],
                                           act))


def opt8_gated_ffn_workspace(rows: int, d: int, f: int) -> int:
    """Bytes of workspace that the backward pass needs."""
    return int(_functions()["workspace"](int(rows), int(d), int(f)))


# ----------------------------------------------------------------------------- calls
def _call(name, desc, stream, check):
    device = desc.device
    if device is None:
        handle = _stream_handle(stream)
    else:
        here = torch.cuda.current_device()
        if here != device:
            raise ValueError(f"the tensors are on cuda:{device}, but the current device is cuda:{here}")
        if stream is None:
            # torch.cuda.current_stream() builds an object for it (3 us, as long as a whole small call)
            handle = torch._C._cuda_getCurrentRawStream(device)
        else:
            where = getattr(stream, "device", None)      # a raw handle does not say
            if where is not None and where.index != device:
                raise ValueError(f"the tensors are on cuda:{device}, but the stream is on {where}")
            handle = _stream_handle(stream)
    rc = (_fns or _functions())[name](desc, handle or None)
    return _check(rc) if check and rc else rc


def opt8_fp8_quantize(quant: opt8_fp8_quant, stream=None, check: bool = True) -> int:
    """Queue the quantisation on a stream of the tensors' device, which has to be the current
    one (a torch.cuda.Stream, a raw handle, or None for torch's current stream); the tensors
    must live until it has run."""
    return _call("opt8_fp8_quantize", quant, stream, check)


def opt8_fp8_matmul(product: opt8_fp8_product, stream=None, check: bool = True) -> int:
    """Queue the 8-bit product; arguments as for opt8_fp8_quantize."""
    return _call("opt8_fp8_matmul", product, stream, check)


def opt8_gated_ffn_forward(ffn: opt8_gated_ffn, stream=None, check: bool = True) -> int:
    """Queue the gated block; arguments as for opt8_fp8_quantize."""
    return _call("opt8_gated_ffn_forward", ffn, stream, check)


def opt8_gated_ffn_backward(grad: opt8_gated_ffn_grad, stream=None, check: bool = True) -> int:
    """Queue the gated block's backward pass; arguments as for opt8_fp8_quantize."""
    return _call("opt8_gated_ffn_backward", grad, stream, check)
