"""Operators of a transformer block over packed tokens: argument marshalling.

    linear         out = act(x W^T + bias) + residual
    norm_residual  h' = residual_scale h + gate * post(y);  u = pre(h') (1 + scale) + shift
    attention      softmax(scale q k^T) v of packed sequences, grouped heads, causal or not
    op_status      what the kernels found wrong on the device (bad groups, bad offsets)

The kernels are in ``libgdit.so`` (``csrc/ops.cu``); the formulas, limits and
error rules are those of ``include/gdit.h``.  Every call is one kernel on
``stream`` (default: torch's current stream of the tensors' device), allocates
nothing but the outputs it returns and may be captured in a CUDA graph.
"""

from __future__ import annotations

import ctypes
import struct

import torch

from . import _lib
from ._lib import (GDIT_ACT_GELU, GDIT_ACT_GELU_TANH, GDIT_ACT_NONE, GDIT_ACT_RELU, GDIT_ACT_SILU,  # noqa: F401
                   GDIT_BF16, GDIT_F32, GDIT_NORM_LAYER, GDIT_NORM_NONE, GDIT_NORM_RMS, check)

__all__ = ["linear", "norm_residual", "attention", "op_status"]

ACTIVATIONS = {None: GDIT_ACT_NONE, "none": GDIT_ACT_NONE, "relu": GDIT_ACT_RELU, "gelu": GDIT_ACT_GELU,
               "gelu_tanh": GDIT_ACT_GELU_TANH, "silu": GDIT_ACT_SILU}
NORMS = {None: GDIT_NORM_NONE, "none": GDIT_NORM_NONE, "layer": GDIT_NORM_LAYER, "rms": GDIT_NORM_RMS}
_DTYPE = {torch.float32: GDIT_F32, torch.bfloat16: GDIT_BF16}
_bf16, _f32, _i32 = torch.bfloat16, torch.float32, torch.int32


class _Op:
    """An entry point that takes one struct of arguments.

    The struct is packed by a format of its members' types and passed as bytes: a call of a few microseconds has no
    time for a ctypes structure, which takes two."""

    def __init__(self, name, args):
        letter = {ctypes.c_void_p: "P", ctypes.c_int64: "q", ctypes.c_int: "i", ctypes.c_float: "f"}
        self.name, self.fn = name, None
        self.pack = struct.Struct("@" + "".join(letter[t] for _, t in args._fields_)).pack

    def __call__(self, device, stream, *args):
        """The call, on the tensors' device and its current stream."""
        if self.fn is None:
            self.fn = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_char_p, ctypes.c_void_p)((self.name, _lib.lib()))
        try:
            a = self.pack(*args)
        except (struct.error, OverflowError) as e:
            raise ValueError(f"{self.name}: an argument is no number of its type: {e}") from None
        if torch._C._cuda_getDevice() == device:
            rc = self.fn(a, torch._C._cuda_getCurrentRawStream(device) if stream is None else stream)
        else:
            with torch.cuda.device(device):
                rc = self.fn(a, torch._C._cuda_getCurrentRawStream(device) if stream is None else stream)
        if rc < 0:
            check(rc)


_linear = _Op("gdit_linear", _lib.gdit_linear_args)
_norm_residual = _Op("gdit_norm_residual", _lib.gdit_norm_args)
_attention = _Op("gdit_attention", _lib.gdit_attention_args)


def _code(table, key, what):
    try:
        return table[key]
    except (KeyError, TypeError):
        raise ValueError(f"{what} is {key!r}, expected one of {[k for k in table if k is not None]}") from None


def _dtype(t, what):
    try:
        return _DTYPE[t]
    except KeyError:
        raise TypeError(f"{what} must be float32 or bfloat16, got {t}") from None


def _rows(t, name, device, rows, cols):
    """Row stride of a [rows, cols] matrix with dense rows."""
    if t.shape != (rows, cols):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(rows, cols)}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError(f"the rows of {name} must be dense")
    if s0 < cols:
        if rows > 1:
            raise ValueError(f"the rows of {name} overlap")
        return (cols + 7) // 8 * 8   # one row: its stride addresses nothing
    return s0


def _vector(t, name, device, shape, dtype=_f32):
    """Address of an optional contiguous vector or table."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} tensor on cuda:{device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def _device(t, name):
    d = t.get_device()
    if d < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    return d


def _matrix(like, rows, cols, dtype):
    """A new [rows, cols] matrix on the device of `like`."""
    if like.dtype is dtype and like.shape == (rows, cols) and like.is_contiguous():
        return torch.empty_like(like)   # the quickest way to one
    return like.new_empty((rows, cols), dtype=dtype)


def linear(x, w, bias=None, *, activation="none", residual=None, out=None, out_dtype=None, stream=None):
    """act(x w^T + bias) + residual for bf16 x [m, k] and w [n, k] (k a multiple of 8).

    bias: float32 [n].  activation: "none", "relu", "gelu" (erf), "gelu_tanh" or "silu".  residual and the result are
    [m, n] of out_dtype (float32 or bfloat16; default: out's, else residual's, else bfloat16).  out may be the
    residual: the sum is then added in place.  The rows of x, w, residual and out may be strided."""
    d = _device(x, "x")
    if x.dtype != _bf16 or w.dtype != _bf16:
        raise TypeError("x and w must be bfloat16")
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x must be [m, k] and w [n, k]")
    m, k = x.shape
    n = w.shape[0]
    ldx, ldw = _rows(x, "x", d, m, k), _rows(w, "w", d, n, k)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else residual.dtype if residual is not None else _bf16
    code = _dtype(out_dtype, "out_dtype")
    ldr, res = n, 0
    if residual is not None:
        if residual.dtype != out_dtype:
            raise TypeError(f"residual is {residual.dtype}, the output {out_dtype}: they must be the same")
        ldr, res = _rows(residual, "residual", d, m, n), residual.data_ptr()
    if out is None:
        out = _matrix(x if residual is None else residual, m, n, out_dtype)
        ldo = n
    else:
        if out.dtype != out_dtype:
            raise TypeError(f"out is {out.dtype}, expected {out_dtype}")
        ldo = _rows(out, "out", d, m, n)
    _linear(d, stream, x.data_ptr(), w.data_ptr(), _vector(bias, "bias", d, (n,)), res, out.data_ptr(), m, ldx, ldw, ldr,
            ldo, n, k, code, _code(ACTIVATIONS, activation, "activation"))
    return out


def _groups(t, name, device, dim):
    """(pointer, groups) of a [dim] or [groups, dim] table."""
    if t is None:
        return 0, 1
    groups = 1 if t.dim() == 1 else t.shape[0]
    if groups < 1:
        raise ValueError(f"{name} has no group")
    return _vector(t, name, device, (dim,) if t.dim() == 1 else (groups, dim)), groups


def norm_residual(h, y=None, *, post=None, post_gain=None, post_bias=None, gate=None, residual_scale=1.0, pre=None,
                  pre_gain=None, pre_bias=None, scale=None, shift=None, row_group=None, eps=1e-5, out_h=None,
                  out_u=None, u_dtype=None, stream=None):
    """The end of one block and the start of the next on the residual stream h [rows, dim]:

        h' = residual_scale * h + gate * post(y)
        u  = pre(h') * (1 + scale) + shift

    and returns (h', u).  post and pre are None, "layer" or "rms", with optional float32 gains and biases [dim].
    gate, scale and shift are float32 [dim], or [groups, dim] with row_group (int32 [rows]) naming each row's group.
    h and y are float32 or bfloat16; h' has h's type, u has u_dtype (default: out_u's, else y's, else bfloat16).
    Without y the branch is left out, and h' is h itself when residual_scale is 1.  u is None when there is nothing
    to compute for it (no pre, scale or shift, and neither out_u nor u_dtype).  out_h may be h, for an update in
    place."""
    d = _device(h, "h")
    if h.dim() != 2:
        raise ValueError("h must be [rows, dim]")
    rows, dim = h.shape
    hd = _dtype(h.dtype, "h")
    pre_code, post_code = _code(NORMS, pre, "pre"), _code(NORMS, post, "post")
    ldh = _rows(h, "h", d, rows, dim)
    ldy, yp, yd = dim, 0, GDIT_BF16
    if y is not None:
        ldy, yp, yd = _rows(y, "y", d, rows, dim), y.data_ptr(), _dtype(y.dtype, "y")
    elif post_code or post_gain is not None or post_bias is not None or gate is not None:
        raise ValueError("post and gate act on y, which is not given")
    gp, gate_groups = _groups(gate, "gate", d, dim)
    scp, g1 = _groups(scale, "scale", d, dim)
    shp, g2 = _groups(shift, "shift", d, dim)
    if scale is not None and shift is not None and g1 != g2:
        raise ValueError(f"scale has {g1} groups, shift {g2}")
    mod_groups = g1 if scale is not None else g2
    rg = 0
    if row_group is not None:
        rg = _vector(row_group, "row_group", d, (rows,), _i32)
    elif gate_groups > 1 or mod_groups > 1:
        raise ValueError("row_group is needed: gate, scale or shift have several groups")
    if not post_code and (post_gain is not None or post_bias is not None):
        raise ValueError("post_gain and post_bias need post")
    if not pre_code and (pre_gain is not None or pre_bias is not None):
        raise ValueError("pre_gain and pre_bias need pre")
    want_h = y is not None or residual_scale != 1.0 or out_h is not None
    want_u = bool(pre_code) or scale is not None or shift is not None or out_u is not None or u_dtype is not None
    ldoh = ldou = dim
    ohp = oup = 0
    if want_h:
        if out_h is None:
            out_h = _matrix(h, rows, dim, h.dtype)
        else:
            if out_h.dtype != h.dtype:
                raise TypeError(f"out_h is {out_h.dtype}, h is {h.dtype}: they must be the same")
            ldoh = _rows(out_h, "out_h", d, rows, dim)
        ohp = out_h.data_ptr()
    ud = GDIT_BF16
    if want_u:
        if u_dtype is None:
            u_dtype = out_u.dtype if out_u is not None else y.dtype if y is not None else _bf16
        ud = _dtype(u_dtype, "u_dtype")
        if out_u is None:
            out_u = _matrix(h if y is None else y, rows, dim, u_dtype)
        else:
            if out_u.dtype != u_dtype:
                raise TypeError(f"out_u is {out_u.dtype}, expected {u_dtype}")
            ldou = _rows(out_u, "out_u", d, rows, dim)
        oup = out_u.data_ptr()
    if not want_h and not want_u:
        raise ValueError("nothing to compute: give y, a residual_scale, pre, scale or shift")
    vec = (dim,)
    _norm_residual(d, stream, h.data_ptr(), yp, ohp, oup, _vector(post_gain, "post_gain", d, vec),
                   _vector(post_bias, "post_bias", d, vec), gp, _vector(pre_gain, "pre_gain", d, vec),
                   _vector(pre_bias, "pre_bias", d, vec), scp, shp, rg, rows, ldh, ldy, ldoh, ldou, dim, hd, yd, ud,
                   post_code, pre_code, gate_groups, mod_groups, residual_scale, eps)
    return (out_h if want_h else h), (out_u if want_u else None)


def _heads(t, name, device):
    if t.dtype is not _bf16 or t.get_device() != device:
        raise TypeError(f"{name} must be a bfloat16 tensor on cuda:{device}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim], got {tuple(t.shape)}")
    n, heads, dim = t.shape
    st, sh, sd = t.stride()
    if sd != 1 and dim > 1:
        raise ValueError(f"the last dimension of {name} must be dense")
    # the stride of a dimension of one element addresses nothing
    return n, heads, dim, st if n > 1 else heads * dim, sh if heads > 1 else dim


def attention(q, k, v, cu_q, cu_k, *, max_q, max_k, causal=True, scale=None, k_len=None, out=None, return_lse=False,
              stream=None):
    """Attention of packed sequences: bf16 q [total_q, heads, head_dim], k and v [total_k, kv_heads, head_dim].

    Sequence b has the queries cu_q[b]:cu_q[b+1] and the keys cu_k[b]:cu_k[b+1] (int32 [batch + 1] on the device), or,
    with k_len (int32 [batch]), the first k_len[b] keys of that range: a slot of a cache.  causal: the last query of a
    sequence sees all its keys, the one before it all but the last, and so on, which serves whole prompts, further
    pieces of prompts and single tokens over a cache.  max_q and max_k bound the sequences' lengths.  heads is a
    multiple of kv_heads; head_dim a multiple of 8 up to 128; q, k and v may be slices of one tensor.

    Returns the output [total_q, heads, head_dim], or (output, lse) with return_lse: lse float32 [total_q, heads].
    A query without keys gives 0 and -inf.  Rows behind the last sequence are not written."""
    d = _device(q, "q")
    tq, heads, dim, qt, qh = _heads(q, "q", d)
    tk, kv_heads, dk, kt, kh = _heads(k, "k", d)
    tv, hv, dv, vt, vh = _heads(v, "v", d)
    if dk != dim or v.shape != k.shape:
        raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)} and v {tuple(v.shape)} do not fit together")
    if cu_q.dim() != 1 or cu_q.shape[0] < 1:
        raise ValueError("cu_q must be [batch + 1]")
    batch = cu_q.shape[0] - 1
    if out is None:
        out = torch.empty_like(q) if q.is_contiguous() else q.new_empty((tq, heads, dim))
        ot, oh = heads * dim, dim
    else:
        to, ho, do, ot, oh = _heads(out, "out", d)
        if out.shape != q.shape:
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {tuple(q.shape)}")
    lse, lp = None, 0
    if return_lse:
        lse = q.new_empty((tq, heads), dtype=_f32)
        lp = lse.data_ptr()
    _attention(d, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lp,
               _vector(cu_q, "cu_q", d, (batch + 1,), _i32), _vector(cu_k, "cu_k", d, (batch + 1,), _i32),
               _vector(k_len, "k_len", d, (batch,), _i32), tq, tk, qt, qh, kt, kh, vt, vh, ot, oh, batch, heads, kv_heads,
               dim, max_q, max_k, bool(causal), dim ** -0.5 if scale is None else scale)
    return (out, lse) if return_lse else out


def op_status(device=None, stream=None) -> int:
    """0, or the (negative) status code of what the operators' kernels on `device` (default: the current one) have
    found wrong since the last call.  Synchronizes `stream` (default: the device's current stream)."""
    index = torch.cuda.current_device() if device is None else torch.device("cuda", device).index \
        if isinstance(device, int) else torch.device(device).index
    if index is None:
        index = torch.cuda.current_device()
    st = torch.cuda.current_stream(index).cuda_stream if stream is None else stream
    return _lib.gdit_op_status(index, st)
