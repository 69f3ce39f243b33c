"""Operators of a transformer block over packed tokens.

    linear         out = act(x W^T + bias) + residual
    norm_residual  h' = residual_scale h + gate * post(y);  u = pre(h') (1 + scale) + shift
    attention      softmax(scale q k^T) v of packed sequences, grouped heads, causal or not
    op_status      what the kernels found wrong on the device (bad groups, bad offsets)

The kernels are in ``libgdit.so`` (``csrc/ops.cu``); the formulas, limits and
error rules are those of ``include/gdit.h``.  Arguments are checked and outputs
made in ``_binding.so`` (``csrc/binding.cpp``): a call costs the CPU 4 to 6
microseconds, of which the launch takes 3.  Every call is one kernel on
``stream`` (a handle; default: torch's current stream of the tensors' device),
allocates nothing but the outputs it returns and may be captured in a CUDA
graph.  Outputs belong to the stream of the call, as under
``torch.cuda.stream``: another stream waits for it before it reads them.  The
operators have no backward pass: where gradients are on, a tensor that requires
one is refused (RuntimeError); ``torch.no_grad()`` or ``detach()`` says that none
is wanted.
"""

from __future__ import annotations

import ctypes

import torch

from . import _lib
from .build import BINDING

__all__ = ["linear", "norm_residual", "attention", "op_status"]


def _load():
    """The compiled binding, with the entry points of the loaded library."""
    import importlib.machinery
    import importlib.util
    import os
    if not os.path.exists(BINDING):
        raise RuntimeError(f"{BINDING} not found: run flow_matching_dit_b200.build.build() first")
    loader = importlib.machinery.ExtensionFileLoader(__package__ + "._binding", BINDING)
    m = importlib.util.module_from_spec(importlib.util.spec_from_loader(loader.name, loader))
    if m.torch_version != torch.__version__.split("+")[0]:
        raise RuntimeError(f"{BINDING} was built for torch {m.torch_version}, this is {torch.__version__}: run "
                           "flow_matching_dit_b200.build.build(force=True)")
    loader.exec_module(m)
    L = _lib.lib()
    m.init(*(ctypes.cast(f, ctypes.c_void_p).value for f in (L.gdit_linear, L.gdit_norm_residual, L.gdit_attention)),
           _lib.check)
    return m


_binding = _load()
_call_linear, _call_norm_residual, _call_attention = _binding.linear, _binding.norm_residual, _binding.attention


def linear(x, w, bias=None, *, activation="none", residual=None, out=None, out_dtype=None, stream=None):
    """act(x w^T + bias) + residual for bf16 x [m, k] and w [n, k] (k a multiple of 8).

    bias: float32 [n].  activation: "none", "relu", "gelu" (erf), "gelu_tanh" or "silu".  residual and the result are
    [m, n] of out_dtype (float32 or bfloat16; default: out's, else residual's, else bfloat16).  out may be the
    residual: the sum is then added in place.  It may not overlap x or w.  The rows of x, w, residual and out may be
    strided."""
    return _call_linear(x, w, bias, activation, residual, out, out_dtype, stream)


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
    place, and out_u may be y."""
    return _call_norm_residual(h, y, post, post_gain, post_bias, gate, residual_scale, pre, pre_gain, pre_bias, scale,
                               shift, row_group, eps, out_h, out_u, u_dtype, stream)


def attention(q, k, v, cu_q, cu_k, *, max_q, max_k, causal=True, scale=None, k_len=None, out=None, return_lse=False,
              stream=None):
    """Attention of packed sequences: bf16 q [total_q, heads, head_dim], k and v [total_k, kv_heads, head_dim].

    Sequence b has the queries cu_q[b]:cu_q[b+1] and the keys cu_k[b]:cu_k[b+1] (int32 [batch + 1] on the device), or,
    with k_len (int32 [batch]), the first k_len[b] keys of that range: a slot of a cache.  causal: the last query of a
    sequence sees all its keys, the one before it all but the last, and so on, which serves whole prompts, further
    pieces of prompts and single tokens over a cache.  max_q and max_k bound the sequences' lengths.  heads is a
    multiple of kv_heads; head_dim a multiple of 8 up to 128; q, k and v may be slices of one tensor, and out may be q,
    but not overlap k or v.

    Returns the output [total_q, heads, head_dim], or (output, lse) with return_lse: lse float32 [total_q, heads].
    A query without keys gives 0 and -inf.  Rows behind the last sequence are not written."""
    return _call_attention(q, k, v, cu_q, cu_k, max_q, max_k, causal, scale, k_len, out, return_lse, stream)


def op_status(device=None, stream=None) -> int:
    """0, or the (negative) status code of what the operators' kernels on `device` (default: the current one) have
    found wrong since the last call.  Synchronizes `stream` (default: the device's current stream)."""
    index = torch.cuda.current_device() if device is None else torch.device("cuda", device).index \
        if isinstance(device, int) else torch.device(device).index
    if index is None:
        index = torch.cuda.current_device()
    st = torch.cuda.current_stream(index).cuda_stream if stream is None else stream
    return _lib.gdit_op_status(index, st)
