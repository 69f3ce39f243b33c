"""Host-side rules of the operators (linear, norm_residual, attention): struct
layouts, refusals before any CUDA call, calls with nothing to do.  No GPU."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest

from flow_matching_dit_b200 import _lib
from flow_matching_dit_b200.build import HEADER, LIB, build

STRUCTS = ("gdit_linear_args", "gdit_norm_args", "gdit_attention_args")
FAKE = 1 << 20   # a pointer that is never followed: 16-byte aligned


@pytest.fixture(scope="module")
def L():
    build()
    return _lib.lib()


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not installed")
def test_struct_layouts_equal_the_headers(tmp_path):
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "gdit.h"', "int main(void) {"]
    for name in STRUCTS:
        lines.append(f'printf("{name} %d\\n", (int)sizeof({name}));')
        for f, _ in getattr(_lib, name)._fields_:
            lines.append(f'printf("{name}.{f} %d\\n", (int)offsetof({name}, {f}));')
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0; }"]))
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.dirname(HEADER),
                    str(src), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    want = dict(zip(out[::2], map(int, out[1::2])))
    for name in STRUCTS:
        T = getattr(_lib, name)
        assert ctypes.sizeof(T) == want[name]
        for f, _ in T._fields_:
            assert getattr(T, f).offset == want[f"{name}.{f}"], (name, f)


def test_codes_equal_the_headers():
    src = open(HEADER).read()
    defs = dict((n, int(v)) for n, v in re.findall(r"#define\s+(GDIT_(?:ACT|NORM)_[A-Z_]+)\s+(\d+)", src))
    assert len(defs) == 8
    for n, v in defs.items():
        assert getattr(_lib, n) == v, n


def linear_args(**over):
    a = dict(x=FAKE, w=FAKE, bias=FAKE, residual=None, out=FAKE, m=4, ldx=64, ldw=64, ldr=32, ldo=32, n=32, k=64,
             out_dtype=_lib.GDIT_BF16, activation=_lib.GDIT_ACT_NONE)
    a.update(over)
    return _lib.gdit_linear_args(**a)


@pytest.mark.parametrize("over, word", [
    (dict(x=None), "NULL"), (dict(w=None), "NULL"), (dict(out=None), "NULL"), (dict(m=-1), "m -1"),
    (dict(m=1 << 31), "out of range"), (dict(m=2 ** 31 - 1024), "out of range"),
    (dict(n=2 ** 31 - 1, ldo=1 << 32), "out of range"), (dict(k=2 ** 31 - 8, ldx=1 << 32, ldw=1 << 32), "out of range"),
    (dict(n=0), "n >= 1"), (dict(k=0), "k >= 8"), (dict(k=60), "multiple of 8"),
    (dict(ldx=56), "ldx"), (dict(ldx=68), "ldx"), (dict(ldw=63), "ldw"), (dict(ldo=31), "ldo"),
    (dict(residual=FAKE, ldr=31), "ldr"), (dict(x=FAKE + 8), "16-byte"), (dict(w=FAKE + 2), "16-byte"),
    (dict(out=FAKE + 1), "aligned"), (dict(bias=FAKE + 2), "aligned"),
    (dict(out_dtype=_lib.GDIT_F32, out=FAKE + 2), "aligned"), (dict(out_dtype=7), "out_dtype"),
    (dict(activation=5), "activation"), (dict(activation=-1), "activation"),
])
def test_linear_refuses(L, over, word):
    assert L.gdit_linear(ctypes.byref(linear_args(**over)), None) == _lib.GDIT_EINVAL
    assert word in L.gdit_last_error(None).decode()


def norm_args(**over):
    a = dict(h=FAKE, y=FAKE, out_h=FAKE, out_u=FAKE, rows=4, ldh=32, ldy=32, ldoh=32, ldou=32, dim=32,
             h_dtype=_lib.GDIT_F32, y_dtype=_lib.GDIT_BF16, u_dtype=_lib.GDIT_BF16, post=0, pre=1, gate_groups=1,
             mod_groups=1, residual_scale=1.0, eps=1e-5)
    a.update(over)
    return _lib.gdit_norm_args(**a)


@pytest.mark.parametrize("over, word", [
    (dict(h=None), "NULL h"), (dict(out_h=None, out_u=None), "both NULL"), (dict(rows=-1), "rows"),
    (dict(dim=0), "dim"), (dict(dim=16385, ldh=20000, ldy=20000, ldoh=20000, ldou=20000), "dim"),
    (dict(ldh=31), "ldh"), (dict(ldy=31), "ldy"), (dict(ldoh=31), "ldoh"), (dict(ldou=31), "ldou"),
    (dict(h_dtype=2), "dtype"), (dict(y_dtype=-1), "dtype"), (dict(u_dtype=9), "dtype"), (dict(post=3), "norm kind"),
    (dict(pre=-1), "norm kind"), (dict(gate_groups=0), "group counts"), (dict(mod_groups=2), "row_group"),
    (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(residual_scale=float("inf")), "residual_scale"),
    (dict(y=None, post=1), "need y"), (dict(y=None, gate=FAKE), "need y"), (dict(h=FAKE + 2), "aligned"),
    (dict(out_u=FAKE + 1), "aligned"), (dict(pre_gain=FAKE + 1), "aligned"),
])
def test_norm_refuses(L, over, word):
    assert L.gdit_norm_residual(ctypes.byref(norm_args(**over)), None) == _lib.GDIT_EINVAL
    assert word in L.gdit_last_error(None).decode()


def attention_args(**over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, out=FAKE, cu_q=FAKE, cu_k=FAKE, total_q=8, total_k=8, q_token_stride=256,
             q_head_stride=64, k_token_stride=128, k_head_stride=64, v_token_stride=128, v_head_stride=64,
             out_token_stride=256, out_head_stride=64, batch=1, heads=4, kv_heads=2, head_dim=64, max_q=8, max_k=8,
             causal=1, scale=0.125)
    a.update(over)
    return _lib.gdit_attention_args(**a)


@pytest.mark.parametrize("over, word", [
    (dict(q=None), "NULL"), (dict(cu_q=None), "NULL"), (dict(cu_k=None), "NULL"), (dict(out=None), "NULL"),
    (dict(k=None), "NULL k or v"), (dict(v=None), "NULL k or v"), (dict(batch=-1), "batch"), (dict(batch=65536), "batch"),
    (dict(heads=3), "multiple of kv_heads"), (dict(kv_heads=0), "kv_heads"), (dict(heads=258, kv_heads=2), "above 128"),
    (dict(head_dim=4), "head_dim"), (dict(head_dim=60), "head_dim"), (dict(head_dim=136), "head_dim"),
    (dict(total_q=-1), "total_q"), (dict(total_k=1 << 31), "total_k"), (dict(total_k=2 ** 31 - 1024), "total_k"),
    (dict(total_q=2 ** 31 - 1024), "total_q"), (dict(max_q=-1), "max_q"),
    (dict(scale=float("inf")), "scale"), (dict(scale=float("nan")), "scale"), (dict(q=FAKE + 8), "16-byte"),
    (dict(k=FAKE + 2), "16-byte"), (dict(q_token_stride=257), "stride"), (dict(v_head_stride=-8), "stride"),
    (dict(k_token_stride=-128), "stride"), (dict(out_head_stride=-1), "out stride"), (dict(lse=FAKE + 2), "aligned"),
    (dict(out=FAKE + 1), "aligned"),
])
def test_attention_refuses(L, over, word):
    assert L.gdit_attention(ctypes.byref(attention_args(**over)), None) == _lib.GDIT_EINVAL
    assert word in L.gdit_last_error(None).decode()


def test_null_arguments_are_refused(L):
    for f in (L.gdit_linear, L.gdit_norm_residual, L.gdit_attention):
        assert f(None, None) == _lib.GDIT_EINVAL


def test_nothing_to_do_is_not_an_error(L):
    """No row, no sequence: valid, and no CUDA call is made."""
    assert L.gdit_linear(ctypes.byref(linear_args(m=0, x=None, out=None)), None) == _lib.GDIT_OK
    assert L.gdit_norm_residual(ctypes.byref(norm_args(rows=0, h=None)), None) == _lib.GDIT_OK
    assert L.gdit_attention(ctypes.byref(attention_args(batch=0)), None) == _lib.GDIT_OK
    assert L.gdit_attention(ctypes.byref(attention_args(total_q=0, q=None)), None) == _lib.GDIT_OK


def test_valid_calls_without_a_gpu_say_so(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is here")
    for f, a in ((L.gdit_linear, linear_args()), (L.gdit_norm_residual, norm_args()),
                 (L.gdit_attention, attention_args())):
        assert f(ctypes.byref(a), None) == _lib.GDIT_ENODEV
    assert L.gdit_op_status(0, None) == _lib.GDIT_ENODEV


def test_binding_refuses_before_the_library():
    import torch

    import flow_matching_dit_b200 as gdit
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        gdit.linear(x, x)
    with pytest.raises(TypeError):
        gdit.norm_residual(x)
    with pytest.raises(TypeError):
        gdit.attention(x, x, x, x, x, max_q=1, max_k=1)
    with pytest.raises(AttributeError):
        gdit.no_such_operator
