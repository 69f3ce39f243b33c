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


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("less", [1, 2, 3, 4, 5, 7, 8])
@pytest.mark.parametrize("m, n, k, bn", [(4100, 4104, 2048, 256), (4100, 1032, 520, 128)])
def test_linear_pair_last_column_inside_16_bytes(m, n, k, bn, out, less):
    """Rows that TMA can address, of which the output takes a width that is no multiple of 16 bytes: nothing beside it is
    written, with a residual, without and in place."""
    import torch
    from flow_matching_dit_b200 import linear
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[out]
    g = gen(n + less)
    full, n = n, n - less
    on_pairs(m, n, k, bn, dt, True, True)
    x, w, b = rnd(g, m, k, dtype=torch.bfloat16), rnd(g, n, k, std=k ** -0.5, dtype=torch.bfloat16), rnd(g, n)
    wide = rnd(g, m, full + 8, dtype=dt)
    before, view = wide.clone(), wide[:, :n]
    for residual in (None, rnd(g, m, full + 8, dtype=dt)[:, :n], view):
        ref, tol = linear64(x, w, b, "relu", None if residual is None else residual.clone(), dt)
        linear(x, w, b, activation="relu", residual=residual, out=view)
        within(view, ref, tol)
        assert torch.equal(wide[:, n:], before[:, n:])
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


@pytest.mark.parametrize("m, n, k", [(140000, 16400, 8), (140001, 16401, 16), (2200, 1000003, 8)])
def test_linear_outputs_past_31_bits(m, n, k):
    """More than 2^31 outputs: the last ones lie where they should, bias and residual too."""
    import torch
    from flow_matching_dit_b200 import linear
    g = gen(m)
    x, w, b = rnd(g, m, k, dtype=torch.bfloat16), rnd(g, n, k, dtype=torch.bfloat16), rnd(g, n)
    out = torch.full((m, n), 3.0, device="cuda", dtype=torch.bfloat16)
    assert m * n > 2 ** 31 and linear(x, w, b, residual=out, out=out) is out
    for rows in (slice(0, 40), slice(m - 40, m)):
        within(out[rows], *linear64(x[rows], w, b, "none", torch.full((40, n), 3.0, device="cuda"), torch.bfloat16), f"rows {rows}")
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


def spread(t, how):
    """The values of t [tokens, heads, dim] in another layout."""
    import torch
    n, h, d = t.shape
    if how == "heads first":
        return t.transpose(0, 1).contiguous().transpose(0, 1)
    if how == "wide":        # room behind each head and each token
        big = torch.zeros(n, h + 1, d + 24, device="cuda", dtype=t.dtype)
    else:                    # "odd": rows that begin anywhere
        big = torch.zeros(n, h * (d + 3) + 1, device="cuda", dtype=t.dtype)[:, 1:].unflatten(1, (h, d + 3))
    big[:, :h, :d] = t
    return big[:, :h, :d]


@pytest.mark.parametrize("how", ["heads first", "wide", "odd"])
@pytest.mark.parametrize("heads, kv_heads, dim", [(4, 2, 64), (6, 2, 72), (2, 1, 40), (8, 2, 128), (64, 1, 64)])
@pytest.mark.parametrize("ql, kl", [([300, 7, 256], [300, 7, 256]), ([1, 1, 1], [300, 7, 2000]), ([9, 40], [3000, 40])])
def test_attention_layouts(ql, kl, heads, kv_heads, dim, how):
    """Queries, keys and values head by head or inside wider rows, outputs in those layouts and at odd elements: the same
    bits as dense, and nothing written beside them."""
    import torch
    from flow_matching_dit_b200 import attention
    g = gen(heads + dim)
    q, k, v = (rnd(g, n, h, dim, dtype=torch.bfloat16) for n, h in ((sum(ql), heads), (sum(kl), kv_heads), (sum(kl), kv_heads)))
    cu = lambda n: torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device="cuda")  # noqa: E731
    args, kw = (cu(ql), cu(kl)), dict(max_q=max(ql), max_k=max(kl), return_lse=True)
    want, lse = attention(q, k, v, *args, **kw)
    ref, tol, rl, tl = attention64(q, k, v, ql, kl, [sum(kl[:i]) for i in range(len(kl))], True, dim ** -0.5)
    within(want, ref, tol, "out")
    if how != "odd":
        got, l2 = attention(*(spread(t, how) for t in (q, k, v)), *args, **kw)
        assert torch.equal(got, want) and torch.equal(l2, lse)
    out = spread(torch.full_like(want, 9.0), how)
    base = out._base if out._base is not None else out
    count = int((base == 9.0).sum())
    got, l2 = attention(q, k, v, *args, out=out, **kw)
    assert got is out and torch.equal(out, want) and torch.equal(l2, lse)
    out.fill_(9.0)
    assert int((base == 9.0).sum()) == count and int((base != 0).sum()) == count   # zeros beside it, as before
    clean()


@pytest.mark.parametrize("batch", [4000, 65535])
def test_attention_as_many_sequences_as_there_may_be(batch):
    """One token over no, one or two keys in each of very many sequences, and prompts as short."""
    import torch
    from flow_matching_dit_b200 import attention
    g = gen(batch)
    heads, dim = 2, 64
    nk = torch.arange(batch, device="cuda") % 3
    ck = torch.cat([nk.new_zeros(1), nk.cumsum(0)])
    k, v = (rnd(g, int(ck[-1]), 1, dim, dtype=torch.bfloat16) for _ in range(2))
    for nq in (torch.ones_like(nk), nk):
        cq = torch.cat([nq.new_zeros(1), nq.cumsum(0)])
        q = rnd(g, int(cq[-1]), heads, dim, dtype=torch.bfloat16)
        got, lse = attention(q, k, v, cq.int(), ck.int(), max_q=int(nq.max()), max_k=2, causal=False, return_lse=True)
        seq = torch.repeat_interleave(torch.arange(batch, device="cuda"), nq)
        at = (ck[seq][:, None] + torch.arange(2, device="cuda")).clamp_max(k.shape[0] - 1)
        seen = torch.arange(2, device="cuda") < nk[seq][:, None]
        sc = torch.einsum("thd,tjd->thj", q.double(), k[at][:, :, 0].double()) * dim ** -0.5
        # roundings as in the other tests: scores, exponentials, probabilities in bf16 and the output's own
        e = (dim / 16 + 16) * 2.0 ** -23 * dim ** -0.5 * torch.einsum("thd,tjd->thj", q.double().abs(), k[at][:, :, 0].double().abs()).amax(-1)
        sc = sc.masked_fill(~seen[:, None], -math.inf)
        rl = torch.logsumexp(sc, -1)
        p = torch.exp(sc - rl.clamp_min(-1e300)[..., None])
        vv = v[at][:, :, 0].double()
        ref, mag = torch.einsum("thj,tjd->thd", p, vv), torch.einsum("thj,tjd->thd", p, vv.abs())
        t = mag * (U16 + 2.0 ** -16 + 2 * e[..., None])
        within(got, ref, t + U16 * (ref.abs() + t) + 1e-30, "out")
        within(lse, rl, e + 2.0 ** -16 + 2.0 ** -22 * rl.abs().nan_to_num(posinf=0) + 1e-30, "lse")
    clean()


def test_attention_queries_past_31_bits():
    """Queries and outputs of more than 2^31 elements: the last sequences."""
    import torch
    from flow_matching_dit_b200 import attention
    heads, kv_heads, dim, n, batch = 32, 8, 128, 700, 760
    g = gen(1)
    q = torch.empty(n * batch, heads, dim, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    k, v = (torch.empty(n * batch, kv_heads, dim, device="cuda", dtype=torch.bfloat16).normal_(generator=g) for _ in range(2))
    assert q.numel() > 2 ** 31
    cu = torch.arange(0, n * (batch + 1), n, dtype=torch.int32, device="cuda")
    out, lse = attention(q, k, v, cu, cu, max_q=n, max_k=n, return_lse=True)
    for b in (0, batch - 1):
        rows = slice(b * n, (b + 1) * n)
        ref, tol, rl, tl = attention64(q[rows], k[rows], v[rows], [n], [n], [0], True, dim ** -0.5)
        within(out[rows], ref, tol, f"sequence {b}")
        within(lse[rows], rl, tl, f"lse {b}")
    clean()


def test_attention_sequences_that_begin_late_or_are_all_empty():
    """Rows in front of the first sequence and behind the last one are left as they were; so are all where no sequence has a
    query."""
    import torch
    from flow_matching_dit_b200 import attention
    g = gen(2)
    cu = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for nq in (1, 60):
        q, k, v = (rnd(g, n, h, 64, dtype=torch.bfloat16) for n, h in ((2 * nq + 9, 4), (500, 2), (500, 2)))
        out = torch.full_like(q, 7.0)
        attention(q, k, v, cu(5, 5 + nq, 5 + 2 * nq), cu(100, 230, 499), max_q=nq, max_k=269, out=out)
        ref, tol, _, _ = attention64(q[5:5 + 2 * nq], k, v, [nq, nq], [130, 269], [100, 230], True, 0.125)
        within(out[5:5 + 2 * nq], ref, tol, "out")
        assert (out[:5] == 7).all() and (out[5 + 2 * nq:] == 7).all()
        out.fill_(7.0)
        attention(q, k, v, cu(0, 0, 0), cu(0, 20, 500), max_q=0, max_k=480, out=out)
        attention(q, k, v, cu(3, 3, 3), cu(0, 20, 500), max_q=nq, max_k=480, out=out)
        assert (out == 7).all()
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


def test_calls_from_several_host_threads():
    """Threads with a stream each run the three operators at the same time, errors among the calls."""
    import threading

    import torch
    from flow_matching_dit_b200 import GditError, attention, linear, norm_residual
    bf, made, errors = torch.bfloat16, [], []
    for i in range(4):
        g = gen(30 + i)
        n = 40 * i + 1
        made.append((rnd(g, n, 512), rnd(g, 512, 512, std=0.05, dtype=bf), rnd(g, 512),
                     torch.tensor([0, n], dtype=torch.int32, device="cuda"), n))

    def block(h, w, gain, cu, n):
        h, u = norm_residual(h, None, pre="rms", pre_gain=gain, u_dtype=bf)
        q = linear(u, w, activation="silu").view(n, 4, 128)
        return linear(attention(q, q, q, cu, cu, max_q=n, max_k=n).view(n, 512), w, residual=h, out_dtype=torch.float32)

    want = [block(*m) for m in made]
    torch.cuda.synchronize()

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(60):
                    got = block(*made[i])
                    with pytest.raises(GditError, match="multiple of 8"):
                        linear(made[i][1][:, :60], made[i][1][:, :60])
                torch.cuda.current_stream().synchronize()
                assert torch.equal(got, want[i])
        except BaseException as e:   # noqa: B902
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(made))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    clean()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_block_that_the_readme_shows(dtype):
    """Its lines as they stand, on a residual stream of either type."""
    import os
    import re

    import torch
    from flow_matching_dit_b200.build import ROOT
    text = open(os.path.join(ROOT, "README.md")).read()
    code = next(c for c in re.findall(r"```python\n(.*?)```", text, re.S) if "norm_residual" in c)
    g = gen(17)
    width, heads, kv_heads, dim, tokens, longest = 256, 4, 2, 64, 90, 60
    bf = torch.bfloat16
    mat = lambda n, k: rnd(g, n, k, std=k ** -0.5, dtype=bf)  # noqa: E731
    x = rnd(g, tokens, width, dtype={"f32": torch.float32, "bf16": bf}[dtype])
    names = dict(torch=torch, x=x, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, longest=longest,
                 cu=torch.tensor([0, 30, 90], dtype=torch.int32, device="cuda"), w_qkv=mat((heads + 2 * kv_heads) * dim, width),
                 b_qkv=rnd(g, (heads + 2 * kv_heads) * dim), w_o=mat(width, heads * dim), w_1=mat(4 * width, width),
                 w_2=mat(width, 4 * width), gate=rnd(g, width), **{f"g{i}": rnd(g, width, std=0.1) + 1 for i in (1, 2, 3)})
    exec(code, names)
    h = names["h"]
    assert h.dtype == x.dtype and h.shape == x.shape and torch.isfinite(h).all() and not torch.equal(h, x)


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


# ---------------------------------------------------------------------------------------------- waits

@pytest.mark.parametrize("limit_ns", [1000, 20_000_000])
def test_a_wait_that_runs_out_is_reported_and_calls_go_on(limit_ns):
    """The operators' waits on a barrier that nothing arrives at: the first ends after its limit, the others with it (their
    own would be 2 s), and the status says so once."""
    import time

    import torch
    from flow_matching_dit_b200 import _lib, debug_op_wait_expiry, linear, op_status
    x = rnd(gen(3), 64, 256, dtype=torch.bfloat16)
    want = linear(x, x)
    clean()
    t = time.perf_counter()
    assert debug_op_wait_expiry(0, limit_ns) == _lib.GDIT_ETIMEOUT
    assert limit_ns * 1e-9 <= time.perf_counter() - t < 1.0
    assert op_status() == 0
    assert torch.equal(linear(x, x), want)
    clean()
