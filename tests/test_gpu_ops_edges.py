"""The operators where their layouts, values or callers are unusual, against
the 64-bit forms and with the tolerances of test_gpu_ops."""

import math

import pytest

from tests.gpu_util import require_gpu
from tests.test_gpu_ops import U16, act64, attention64, check_linear, clean, gen, linear64, norm64, rnd, within

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


# ---------------------------------------------------------------------------------------------- linear

@pytest.mark.parametrize("m", [33, 2500])
def test_linear_gelu_is_good_relative_to_its_small_values(m):
    """out = v Phi(v) by f32 and one bf16 value v a row.  Phi(-a) = 2^L(a): L is off by at most 2^-21 up to a = 1, 2^-17 at
    5, 2^-15.8 up to 7, 2^-12 up to 10 and 2^-10.7 to the end, its own rounding is 2^-24 of at most 128 (2^-17) and the
    exponential's 2^-22; those sum to less than the bounds here.  Where v is positive Phi(-v) is at most half of the
    factor.  Results below 13 2^-126 are 0."""
    import torch
    from flow_matching_dit_b200 import linear
    n, k = 1040, 64
    a = torch.cat([torch.logspace(-30, 0, 200), torch.linspace(1, 14, 900)]).cuda()
    z = torch.cat([a, -a, torch.zeros(2, device="cuda")]).bfloat16()
    z = z.repeat(m // len(z) + 1)[:m] if m > len(z) else z[torch.linspace(0, len(z) - 1, m).long().cuda()]
    x, w = (torch.zeros(r, k, device="cuda", dtype=torch.bfloat16) for r in (m, n))
    x[:, 0], w[:, 0] = z, 1
    got = linear(x, w, activation="gelu", out_dtype=torch.float32)
    v = z.double()[:, None].expand(m, n)
    ref = 0.5 * v * torch.erfc(-v * 0.5 ** 0.5)
    a = v.abs()
    rel = torch.where((v > 0) | (a <= 1), 2.0 ** -19, torch.where(a <= 5, 2.0 ** -16, torch.where(a <= 7, 2.0 ** -14.5, 2.0 ** -10)))
    within(got, ref, rel * ref.abs() + 13 * 2.0 ** -126, "gelu")
    clean()


def test_linear_one_row_of_any_stride():
    """One row of x, or of w, whose stride addresses nothing."""
    import torch
    from flow_matching_dit_b200 import linear
    g = gen(9)
    k = 72
    for m, n in ((1, 40), (6, 1), (1, 1)):
        x, w = (rnd(g, rows + 1, k + 9, dtype=torch.bfloat16)[:rows, :k] if rows == 1 else rnd(g, rows, k, dtype=torch.bfloat16)
                for rows in (m, n))
        assert m > 1 or x.stride(0) == k + 9
        got = linear(x, w, activation="silu", out_dtype=torch.float32)
        within(got, *linear64(x, w, None, "silu", None, torch.float32), f"{m} x {n}")
    two = rnd(g, 2, k + 9, dtype=torch.bfloat16)[:, :k]
    with pytest.raises(RuntimeError):
        linear(two, rnd(g, 8, k, dtype=torch.bfloat16))
    clean()


PAIR_SIZES = [(4100, 4104, 2048, 256), (4100, 4103, 2048, 256), (4100, 1032, 520, 128), (4100, 1030, 520, 128)]


def on_pairs(m, n, k, bn, dt, residual=True, aligned=None):
    """Sizes that run on pairs of CTAs with tiles of bn columns, by the planner."""
    import torch
    from flow_matching_dit_b200 import GDIT_BF16, GDIT_F32, debug_linear_plan
    if aligned is None:
        aligned = n * (4 if dt == torch.float32 else 2) % 16 == 0
    plan = debug_linear_plan(m, n, k, GDIT_F32 if dt == torch.float32 else GDIT_BF16, residual, aligned, num_sms=0)
    assert plan == {"pair": True, "bn": bn, "splits": 1}


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("bias, residual", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("m, n, k, bn", PAIR_SIZES)
def test_linear_pair_epilogues(m, n, k, bn, act, out, bias, residual):
    """Each epilogue of the pair kernel: outputs by TMA boxes and, where rows begin anywhere, by words; last tiles of 4 rows
    and of 8, 7 or 6 columns."""
    import torch
    on_pairs(m, n, k, bn, {"bf16": torch.bfloat16, "f32": torch.float32}[out], residual)
    check_linear(m, n, k, act, out, bias, residual, seed=5, std=2.0)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("offset, pad", [(8, 16), (0, 8), (1, 5), (3, 0)])
@pytest.mark.parametrize("m, n, k, bn", [(4100, 4104, 2048, 256), (4100, 1032, 520, 128)])
def test_linear_pair_strided_and_in_place(m, n, k, bn, out, offset, pad):
    """Outputs inside wider rows, aligned for TMA and not, the residual another tensor or the output itself; what lies around
    them stays as it was."""
    import torch
    from flow_matching_dit_b200 import linear
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[out]
    g = gen(n + offset)
    x, w = rnd(g, m, k, dtype=torch.bfloat16), rnd(g, n, k, std=k ** -0.5, dtype=torch.bfloat16)
    b = rnd(g, n)
    wide = rnd(g, m, offset + n + pad, dtype=dt)
    size = wide.element_size()
    aligned = offset * size % 16 == 0 and wide.shape[1] * size % 16 == 0
    on_pairs(m, n, k, bn, dt, True, aligned)
    view, before = wide[:, offset:offset + n], wide.clone()
    other = rnd(g, m, offset + n + pad, dtype=dt)[:, offset:offset + n]
    for residual in (other, None, view):
        ref, tol = linear64(x, w, b, "silu", None if residual is None else residual.clone(), dt)
        assert linear(x, w, b, activation="silu", residual=residual, out=view) is view
        within(view, ref, tol)
        assert torch.equal(wide[:, :offset], before[:, :offset]) and torch.equal(wide[:, offset + n:], before[:, offset + n:])
    clean()


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_linear_pair_activations_far_out(act, out):
    """Arguments from tiny to far outside and NaN, one a row, beside rows of another size: no row reaches another."""
    import torch
    from flow_matching_dit_b200 import linear
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[out]
    m, n, k = 4100, 4104, 2048
    on_pairs(m, n, k, 256, dt, False)
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e-4, -1e-4, 0.5, -0.5, 3.0, -3.0, 6.0, -6.0, 20.0, -20.0, 42.0, -42.0, 60.0, -60.0,
                      100.0, -100.0, 1e4, -1e4, 1e12, -1e12, 1e20, -1e20, 3e38, -3e38, float("nan"), -2.0, 90.0], device="cuda").bfloat16()
    z = z.repeat(m // len(z) + 1)[:m]
    x, w = torch.zeros(m, k, device="cuda", dtype=torch.bfloat16), torch.zeros(n, k, device="cuda", dtype=torch.bfloat16)
    x[:, 1000], w[:, 1000] = z, 1
    got = linear(x, w, activation=act, out_dtype=dt)
    v = z.double()[:, None].expand(m, n)
    ref = act64(v, act) if act != "gelu_tanh" else v * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (v + 0.044715 * v ** 3))
    # exponentials and reciprocals to a few 2^-22, arguments of 2 (2/pi)^0.5 log2(e) (v + 0.044715 v^3) < 62 to 2^-23 of them, nothing
    # below 2^-62 of the argument; then the output's half step
    tol = 2.0 ** -16 * ref.abs() + 2.0 ** -61 * v.abs().clamp_max(64) + 1e-30
    within(got, ref, tol + (U16 if out == "bf16" else 0) * (ref.abs() + tol), act)
    clean()


# ---------------------------------------------------------------------------------------------- norm_residual

def padded(g, rows, dim, pad, dtype, std=1.0):
    """[rows, dim] at the front of rows of dim + pad values, and the whole buffer."""
    whole = rnd(g, rows, dim + pad, std=std, dtype=dtype)
    return whole[:, :dim], whole


@pytest.mark.parametrize("pad", [1, 2, 3])
@pytest.mark.parametrize("dim", [4, 128, 256, 260, 512, 1024, 2048, 4096, 8192, 16380, 16384])
def test_norm_rows_that_shift_at_widths_of_whole_units(dim, pad):
    """A width that is a multiple of 4 in rows whose stride is not: every row begins at another offset from an aligned
    address, and the row's last values lie behind those of a row that begins at one.  What is behind the rows stays."""
    import torch
    from flow_matching_dit_b200 import norm_residual
    f32, bf = torch.float32, torch.bfloat16
    for rows, h_type, u_type in ((9, f32, bf), (1300 if dim < 5000 else 300, bf, f32)):
        g = gen(dim * 4 + pad + rows)
        h, _ = padded(g, rows, dim, pad, h_type, 3.0)
        y, _ = padded(g, rows, dim, pad, bf)
        out_h, all_h = padded(g, rows, dim, pad, h_type)
        out_u, all_u = padded(g, rows, dim, pad, u_type)
        behind = all_h[:, dim:].clone(), all_u[:, dim:].clone()
        pg, gain, bias, scale, shift = (rnd(g, dim, std=0.2) + 1 for _ in range(5))
        norm_residual(h, y, post="rms", post_gain=pg, pre="layer", pre_gain=gain, pre_bias=bias, scale=scale, shift=shift,
                      out_h=out_h, out_u=out_u)
        rh, th, ru, tu = norm64(h, y, "rms", pg, None, None, 1.0, "layer", gain, bias, scale, shift, None, 1e-5, h_type, u_type)
        within(out_h, rh, th, "h'")
        within(out_u, ru, tu, "u")
        assert torch.equal(all_h[:, dim:], behind[0]) and torch.equal(all_u[:, dim:], behind[1])
    clean()


@pytest.mark.parametrize("dim", [1024, 16384])
def test_norm_in_place_in_wider_rows(dim):
    import torch
    from flow_matching_dit_b200 import norm_residual
    h, whole = padded(gen(dim), 300, dim, 1, torch.float32)
    before = whole.clone()
    norm_residual(h, residual_scale=0.5, out_h=h)
    assert torch.equal(h, before[:, :dim] * 0.5) and torch.equal(whole[:, dim:], before[:, dim:])
    clean()


# ---------------------------------------------------------------------------------------------- attention

@pytest.mark.parametrize("heads, kv_heads, dim", [(2, 1, 64), (8, 2, 128), (40, 2, 64), (128, 1, 64)])
@pytest.mark.parametrize("nq", [1, 3, 150])
@pytest.mark.parametrize("std", [1.0, 40.0])
def test_attention_nan_inside_a_sequence(heads, kv_heads, dim, nq, std):
    """A NaN in a query, in a visible key or value: the same outputs are NaN whichever kernel and however many parts the
    keys are taken in, a part of which a NaN is the only score and one whose scores are far below the others' (std 40)
    among them.  A key that causality hides does not matter."""
    import torch
    from flow_matching_dit_b200 import attention
    nan = float("nan")
    for nk, bad in ((nq, nq - 1), (129 + nq, 128 + nq), (1000 + nq, 0), (1000 + nq, 700), (3000 + nq, 2999)):
        for what in ("q", "k", "v"):
            g = gen(nk + nq + heads)
            q = rnd(g, 2 * nq, heads, dim, std=std, dtype=torch.bfloat16)
            k, v = (rnd(g, nk + 200, kv_heads, dim, std=s, dtype=torch.bfloat16) for s in (std, 1.0))
            # the values of the other places, and NaN where the formula has it: in the rows of the query, or of those that see the key
            ref, tol, rl, tl = attention64(q, k, v, [nq, nq], [nk, 200], [0, nk], True, dim ** -0.5)
            sees = torch.arange(2 * nq, device="cuda") < nq
            sees &= torch.arange(2 * nq, device="cuda") >= bad - (nk - nq)
            group = heads // kv_heads
            if what == "q":
                q[nq - 1, heads - 1, 3] = nan
                ref[nq - 1, heads - 1] = rl[nq - 1, heads - 1] = nan
            elif what == "k":
                k[bad, 0, dim - 1] = nan
                ref[sees, :group] = nan
                rl[sees, :group] = nan
            else:
                v[bad, kv_heads - 1, 5] = nan
                ref[sees, heads - group:, 5] = nan
            cu = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
            got, lse = attention(q, k, v, cu(0, nq, 2 * nq), cu(0, nk, nk + 200), max_q=nq, max_k=max(nk, 200), return_lse=True)
            assert torch.isnan(ref).any()
            if what == "v":   # a value may reach the queries of its sequence of which it is hidden, too
                got[:nq, :, 5] = torch.where(sees[:nq, None] | torch.isfinite(got[:nq, :, 5]), got[:nq, :, 5], ref[:nq, :, 5].to(got.dtype))
            within(got, ref, tol, f"{what} {nk}")
            within(lse, rl, tl, f"lse {what} {nk}")
    clean()


@pytest.mark.parametrize("nq", [1, 200])
@pytest.mark.parametrize("size, scale", [(2.0 ** 60, 2.0 ** -122), (2.0 ** 55, -2.0 ** -111), (2.0 ** -60, 2.0 ** 120), (1.0, 0.0)])
def test_attention_scales_far_from_one(nq, size, scale):
    """Queries and keys of magnitude `size`, whose scores the scale brings back to ordinary ones."""
    import torch
    from flow_matching_dit_b200 import attention
    g = gen(nq)
    q, k, v = (rnd(g, n, 2, 64, dtype=torch.bfloat16) for n in (nq, 300, 300))
    cu = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    got, lse = attention(q * size, k * size, v, cu(0, nq), cu(0, 300), max_q=nq, max_k=300, scale=scale, return_lse=True)
    ref, tol, rl, tl = attention64(q, k, v, [nq], [300], [0], True, scale * size ** 2)
    within(got, ref, tol, "out")
    within(lse, rl, tl, "lse")
    clean()


# ---------------------------------------------------------------------------------------------- streams

def test_outputs_belong_to_the_stream_given():
    """With stream= and no outputs given, these come from what the allocator keeps for that stream: not a block that the
    current stream may still read, and not one that it may be given while the call is under way."""
    import torch
    from flow_matching_dit_b200 import attention, linear, norm_residual, op_status
    g = gen(21)
    bf = torch.bfloat16
    x, w, h = rnd(g, 512, 512, dtype=bf), rnd(g, 512, 512, dtype=bf), rnd(g, 512, 512)
    q, cu = x.view(512, 4, 128), torch.tensor([0, 512], dtype=torch.int32, device="cuda")
    calls = [lambda st: (linear(x, w, stream=st),), lambda st: norm_residual(h, x, pre="rms", stream=st),
             lambda st: attention(q, q, q, cu, cu, max_q=512, max_k=512, return_lse=True, stream=st)]
    for handle in (0, 1):   # the default stream by its two handles
        assert torch.equal(calls[0](handle)[0], calls[0](None)[0])
    for call in calls:
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        st = torch.cuda.Stream()
        spare = [torch.empty_like(t) for t in want for _ in range(8)]
        free = {t.data_ptr() for t in spare}
        del spare   # free blocks of just these sizes on the current stream
        got = call(st.cuda_stream)
        assert torch.cuda.current_stream() != st
        st.synchronize()
        assert op_status(stream=st.cuda_stream) == 0
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        theirs = {t.data_ptr() for t in got}
        assert not theirs & free
        del got
        assert not theirs & {t.data_ptr() for t in [torch.empty_like(t) for t in want for _ in range(8)]}
        with torch.cuda.stream(st):
            assert theirs & {t.data_ptr() for t in [torch.empty_like(t) for t in want]}


# ---------------------------------------------------------------------------------------------- autograd

def test_tensors_that_require_a_gradient_are_refused():
    """No gradient is dropped silently: every tensor of each operator, outputs among them."""
    import torch
    from flow_matching_dit_b200 import attention, linear, norm_residual
    bf = torch.bfloat16
    mat = lambda dt=bf: torch.ones(8, 64, device="cuda", dtype=dt)  # noqa: E731
    vec = lambda: torch.ones(64, device="cuda")  # noqa: E731
    heads, cu = lambda: torch.ones(8, 1, 64, device="cuda", dtype=bf), torch.tensor([0, 8], dtype=torch.int32, device="cuda")  # noqa: E731
    calls = [(linear, dict(x=mat(), w=torch.ones(64, 64, device="cuda", dtype=bf), bias=vec(), residual=mat(), out=mat()), {}),
             (norm_residual, dict(h=mat(torch.float32), y=mat(), post_gain=vec(), post_bias=vec(), gate=vec(), pre_gain=vec(),
                                  pre_bias=vec(), scale=vec(), shift=vec(), out_h=mat(torch.float32), out_u=mat()),
              dict(post="layer", pre="layer")),
             (attention, dict(q=heads(), k=heads(), v=heads(), out=heads()), dict(cu_q=cu, cu_k=cu, max_q=8, max_k=8))]
    for f, tensors, rest in calls:
        f(**tensors, **rest)
        for name in tensors:
            with_grad = {**tensors, name: tensors[name].clone().requires_grad_()}
            with pytest.raises(RuntimeError, match=f"{name} requires a gradient"):
                f(**with_grad, **rest)
            with torch.no_grad():
                f(**with_grad, **rest)
            f(**{**tensors, name: with_grad[name].detach()}, **rest)
            if "out" not in name:
                with torch.inference_mode():
                    f(**with_grad, **rest)
    clean()


def test_writes_into_given_tensors_are_seen_by_autograd():
    """A tensor that autograd has kept and an operator has written since: its backward pass says so."""
    import torch
    from flow_matching_dit_b200 import attention, linear, norm_residual
    bf = torch.bfloat16
    x, h, cu = (torch.ones(8, 64, device="cuda", dtype=bf), torch.ones(8, 64, device="cuda"),
                torch.tensor([0, 8], dtype=torch.int32, device="cuda"))
    q, w = x.view(8, 1, 64), torch.ones(64, 64, device="cuda", dtype=bf)
    for call, shape, dtype in ((lambda t: linear(x, w, out=t), (8, 64), bf), (lambda t: norm_residual(h, x, out_h=t), (8, 64), h.dtype),
                               (lambda t: norm_residual(h, x, pre="rms", out_u=t), (8, 64), bf),
                               (lambda t: attention(q, q, q, cu, cu, max_q=8, max_k=8, out=t), (8, 1, 64), bf)):
        out = torch.ones(shape, device="cuda", dtype=dtype)
        leaf = torch.ones(shape, device="cuda", dtype=dtype, requires_grad=True)
        product = leaf * out
        before = out._version
        call(out)
        assert out._version > before
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            product.sum().backward()
        with torch.inference_mode():
            call(torch.ones(shape, device="cuda", dtype=dtype))   # such tensors have no version
    clean()
