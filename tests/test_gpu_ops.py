"""The operators against plain 64-bit forms of their formulas, through the
public entry points (flow_matching_dit_b200.linear, norm_residual, attention).

Tolerances count roundings (u16 = 2^-8: half a step of bf16; u32 = 2^-24):
  linear     the tensor cores add 16 products at a time to a running sum kept in 24 bits; each of the K/16 additions may
             lose 2^-23 of the largest partial sum, which is at most S = sum |x w|, and aligning the products another 16
             such steps at the outside: (K/16 + 16) 2^-23 S.  An activation's slope is at most 1.13, and its own f32
             evaluation is off by at most 2^-19 of its argument.  Then the output's own half step.
  norm       a sum over a row in a tree loses at most (log2 dim + 8) u32 of the sum of magnitudes; with the root, the
             quotient and the affine steps no value is off by more than 64 u32 of the magnitudes that make it up (twice
             that where post and pre follow one another).
  attention  probabilities are rounded to bf16 for the second product: u16 of sum p |v|; scores are off by at most
             (dim/16 + 16) 2^-23 sum |q k| scale and exp2 and the running rescales by 2^-16 together; then the output's half step.
"""

import math

import numpy as np
import pytest

from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

U16, U32 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rnd(g, *shape, std=1.0, dtype=None):
    import torch
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype or torch.float32)


def within(got, ref, tol, what=""):
    """|got - ref| <= tol elementwise, NaN and infinities in the same places."""
    import torch
    got = got.double()
    fin = torch.isfinite(ref)
    assert torch.equal(fin, torch.isfinite(got)), what
    assert torch.equal(ref[~fin].nan_to_num(123.0), got[~fin].nan_to_num(123.0)), what
    over = ((got - ref).abs() - tol)[fin]
    if over.numel():
        worst = float(over.max())
        assert worst <= 0, f"{what}: {worst:.3g} over the tolerance, {int((over > 0).sum())} of {over.numel()}"


def clean():
    from flow_matching_dit_b200 import op_status
    assert op_status() == 0


# ---------------------------------------------------------------------------------------------- linear

def act64(z, act):
    import torch
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def linear64(x, w, bias, act, residual, out_dtype):
    import torch
    z = x.double() @ w.double().t()
    s = x.double().abs() @ w.double().abs().t()
    if bias is not None:
        z, s = z + bias.double(), s + bias.double().abs()
    ref = act64(z, act)
    tol = 1.13 * (x.shape[1] / 16 + 16) * 2.0 ** -23 * s + 2.0 ** -19 * z.abs()
    if residual is not None:
        ref = ref + residual.double()
        tol = tol + 2 * U32 * residual.double().abs()
    return ref, tol + (U16 if out_dtype == torch.bfloat16 else U32) * (ref.abs() + tol) + 1e-30


def check_linear(m, n, k, act="none", out="bf16", bias=True, residual=False, seed=0, std=1.0):
    import torch
    from flow_matching_dit_b200 import linear
    g = gen(seed + m * 7 + n * 3 + k)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[out]
    x, w = rnd(g, m, k, std=std, dtype=torch.bfloat16), rnd(g, n, k, std=k ** -0.5, dtype=torch.bfloat16)
    b = rnd(g, n, std=0.5) if bias else None
    r = rnd(g, m, n, dtype=dt) if residual else None
    got = linear(x, w, b, activation=act, residual=r, out_dtype=dt)
    assert got.dtype == dt and got.shape == (m, n)
    within(got, *linear64(x, w, b, act, r, dt), f"{m}x{n}x{k} {act} {out}")
    clean()


@pytest.mark.parametrize("m, n, k", [
    (1, 1, 8), (1, 4096, 1024), (1, 17, 8200), (2, 31, 72), (7, 1000, 264), (16, 128, 64), (17, 1024, 1024),
    (33, 2056, 520), (64, 48, 4096), (65, 4096, 512), (127, 130, 128), (128, 128, 136), (129, 257, 64),
    (136, 1024, 4096), (255, 96, 40), (256, 256, 64), (257, 512, 1000), (300, 2048, 2048), (511, 513, 200),
    (600, 4096, 1024), (1237, 2056, 1096), (2049, 1025, 8), (4352, 1024, 1024), (70000, 40, 16),
])
@pytest.mark.parametrize("out, residual", [("bf16", False), ("f32", True)])
def test_linear_sizes(m, n, k, out, residual):
    check_linear(m, n, k, "none", out, True, residual)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("bias, residual", [(False, False), (True, True)])
@pytest.mark.parametrize("m, n, k", [(5, 72, 128), (200, 264, 192), (520, 512, 256)])
def test_linear_epilogues(m, n, k, act, out, bias, residual):
    check_linear(m, n, k, act, out, bias, residual, seed=3, std=2.0)


@pytest.mark.parametrize("m", [3, 140, 700])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_linear_strides_and_in_place_residual(m, out):
    """Rows of larger matrices, an output at an odd element with an odd row stride, the residual updated in place; the
    elements around the output stay as they were."""
    import torch
    from flow_matching_dit_b200 import linear
    g = gen(11 + m)
    n, k = 130, 96
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[out]
    x = rnd(g, m, 3 * k, dtype=torch.bfloat16)[:, k:2 * k]
    w = rnd(g, n, k + 40, std=0.1, dtype=torch.bfloat16)[:, 8:8 + k]
    b = rnd(g, n)
    for offset, width in ((1, 133), (8, 144)):
        big = rnd(g, m, width, dtype=dt)
        before = big.clone()
        view = big[:, offset:offset + n]
        ref, tol = linear64(x, w, b, "silu", view.clone(), dt)
        assert linear(x, w, b, activation="silu", residual=view, out=view) is view
        within(view, ref, tol)
        assert torch.equal(big[:, :offset], before[:, :offset]) and torch.equal(big[:, offset + n:], before[:, offset + n:])
    clean()


def test_linear_values_that_are_not_finite_stay_in_their_rows():
    import torch
    from flow_matching_dit_b200 import linear
    for m in (9, 300, 1030):
        g = gen(m)
        x, w = rnd(g, m, 256, dtype=torch.bfloat16), rnd(g, 520, 256, dtype=torch.bfloat16)
        ref = linear(x, w, activation="relu")
        x[m // 2, 3] = float("nan")
        got = linear(x, w, activation="relu")
        assert torch.isnan(got[m // 2]).all()
        keep = torch.arange(m, device="cuda") != m // 2
        assert torch.equal(got[keep], ref[keep])
    clean()


@pytest.mark.parametrize("m, n, k", [(1, 8192, 8192), (8, 11008, 4096), (3, 2671, 1792), (17, 1024, 1024), (33, 552, 5264),
                                     (200, 5000, 5000), (500, 500, 4000), (1015, 85, 5008), (300, 2048, 2048), (9, 16, 8)])
def test_linear_split_plans(m, n, k):
    """Sizes whose plans differ: tile widths, parts of K (clusters of any size up to 8), boxes of 8 to 128 rows."""
    check_linear(m, n, k, "silu", "bf16", True, True)
    check_linear(m, n, k, "none", "f32", False, True)


@pytest.mark.parametrize("m, n, k", [(2500, 2051, 136), (1821, 6388, 24), (4099, 1030, 520), (1111, 4097, 64)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_linear_many_rows_that_no_box_fits(m, n, k, out):
    """Outputs and residuals whose rows begin anywhere, over many tiles; and slices with room that stays as it was."""
    import torch
    from flow_matching_dit_b200 import linear
    check_linear(m, n, k, "gelu", out, True, True)
    check_linear(m, n, k, "none", out, False, False)
    g = gen(n)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[out]
    x, w = rnd(g, m, k, dtype=torch.bfloat16), rnd(g, n, k, std=k ** -0.5, dtype=torch.bfloat16)
    wide = torch.full((m, n + 6), 5.0, device="cuda", dtype=dt)
    r = rnd(g, m, n + 1, dtype=dt)[:, 1:]
    out_ = wide[:, 3:3 + n]
    linear(x, w, residual=r, out=out_)
    within(out_, *linear64(x, w, None, "none", r, dt))
    assert (wide[:, :3] == 5).all() and (wide[:, 3 + n:] == 5).all()
    out_.copy_(r)
    linear(x, w, residual=out_, out=out_)   # in place
    within(out_, *linear64(x, w, None, "none", r, dt))
    clean()


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("m", [4, 1100])
def test_linear_activations_far_out(act, m):
    """Arguments from tiny to far outside: out = act(z), z = the row's value, neighbours with another size in turn."""
    import torch
    from flow_matching_dit_b200 import linear
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e-4, -1e-4, 0.5, -0.5, 3.0, -3.0, 6.0, -6.0, 20.0, -20.0, 42.0, -42.0, 60.0,
                      -60.0, 100.0, -100.0, 1e4, -1e4, 1e12, -1e12, 1e20, -1e20, 3e38, -3e38, 2.0, -2.0, 90.0, -90.0],
                     device="cuda").bfloat16()
    n, k = 1024, 64
    x = torch.zeros(m, k, device="cuda", dtype=torch.bfloat16)
    x[:, 0] = z.repeat(m // 32 + 1)[:m]
    x[:, 1] = 1
    w = torch.zeros(n, k, device="cuda", dtype=torch.bfloat16)
    w[:, 0] = 1
    b = torch.zeros(n, device="cuda")
    got = linear(x, w, b, activation=act, out_dtype=torch.float32)
    w[:, 1] = z.repeat(n // 32 + 1)[:n]          # and along the columns
    x[:, 0] = 0
    across = linear(x, w, b, activation=act, out_dtype=torch.float32)
    for out, arg in ((got, z.repeat(m // 32 + 1)[:m, None].expand(m, n)), (across, z.repeat(n // 32 + 1)[None, :n].expand(m, n))):
        v = arg.double()
        ref = {"relu": v.clamp_min(0), "gelu": 0.5 * v * torch.erfc(-v / math.sqrt(2)),
               "gelu_tanh": v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)),
               "silu": v * torch.sigmoid(v)}[act]
        # an erf to 3e-7, exponentials and reciprocals to a few 2^-22, nothing below 2^-62 of the argument
        within(out, ref, 2.0 ** -19 * ref.abs() + 4e-7 * v.abs().clamp_max(8) + 2.0 ** -61 * v.abs().clamp_max(64) + 1e-30, act)
    clean()


def test_linear_refusals():
    import torch
    from flow_matching_dit_b200 import GditError, linear
    x, w = (torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    with pytest.raises(TypeError):
        linear(x.float(), w)
    with pytest.raises(TypeError):
        linear(x, w, out_dtype=torch.float16)
    with pytest.raises(TypeError):
        linear(x, w, residual=torch.zeros(8, 8, device="cuda"), out_dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        linear(x, w[:, :56])
    with pytest.raises(ValueError):
        linear(x, w, torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError):
        linear(x, w, activation="tanh")
    with pytest.raises(ValueError):
        linear(x.t(), w)
    with pytest.raises(ValueError):
        linear(x, w.cpu())
    with pytest.raises(GditError):
        linear(x[:, :60], w[:, :60])
    with pytest.raises(GditError):   # not 16-byte aligned
        linear(x[:, 4:60], w[:, 4:60])
    assert linear(x[:0], w).shape == (0, 8)


# ---------------------------------------------------------------------------------------------- norm_residual

def norm64(h, y, post, pg, pb, gate, rs, pre, g, b, scale, shift, group, eps, h_dtype, u_dtype):
    """(h', tolerance, u, tolerance) in 64 bits."""
    import torch

    def d(t):
        return None if t is None else t.double()

    def rows(t):
        t = d(t)
        return t if t is None or t.dim() == 1 else t[0] if t.shape[0] == 1 else t[group.long()]

    def norm(t, mag, kind, gain, bias):
        """value, magnitude of what makes it up"""
        if kind is None:
            return t, mag
        mean = t.mean(1, keepdim=True) if kind == "layer" else 0.0
        r = 1 / torch.sqrt(((t - mean) ** 2).mean(1, keepdim=True) + eps)
        v, top = (t - mean) * r, (mag + (mag.mean(1, keepdim=True) if kind == "layer" else 0.0)) * r
        top = top + v.abs()   # the root's relative error
        if gain is not None:
            v, top = v * d(gain), top * d(gain).abs()
        if bias is not None:
            v, top = v + d(bias), top + d(bias).abs()
        return v, top

    v, top = rs * d(h), abs(rs) * d(h).abs()
    if y is not None:
        z, zt = norm(d(y), d(y).abs(), post, pg, pb)
        if gate is not None:
            z, zt = z * rows(gate), zt * rows(gate).abs()
        v, top = v + z, top + zt
    u, ut = norm(v, top, pre, g, b)
    if scale is not None:
        u, ut = u * (1 + rows(scale)), ut * (1 + rows(scale).abs())
    if shift is not None:
        u, ut = u + rows(shift), ut + rows(shift).abs()

    def tol(val, mag, dt, steps):
        e = steps * U32 * mag
        return e + (U16 if dt == torch.bfloat16 else U32) * (val.abs() + e) + 1e-30

    return v, tol(v, top, h_dtype, 64), u, tol(u, ut, u_dtype, 128)


def check_norm(rows, dim, post=None, pre="layer", gate=0, mod=0, h="f32", y="bf16", u="bf16", rs=1.0, offset=0.0,
               seed=0, eps=1e-5, bad_alignment=False):
    """gate, mod: 0 none, 1 a vector, more: that many groups."""
    import torch
    from flow_matching_dit_b200 import norm_residual
    t = {"f32": torch.float32, "bf16": torch.bfloat16}
    g = gen(seed + rows * 5 + dim)

    def mat(dt, std, add=0.0):
        extra = 3 if bad_alignment else 0
        return (rnd(g, rows, dim + extra, std=std) + add).to(dt)[:, extra:]

    H, Y = mat(t[h], 3.0, offset), mat(t[y], 1.0, offset) if y else None
    vec = lambda n, std, add=0.0: None if n == 0 else rnd(g, *([n, dim] if n > 1 else [dim]), std=std) + add  # noqa: E731
    pg, pb = (vec(1, 0.2, 1.0), vec(1, 0.2)) if post else (None, None)
    G, B = (vec(1, 0.2, 1.0), vec(1, 0.2)) if pre else (None, None)
    ga, sc, sh = vec(gate, 0.5), vec(mod, 0.2), vec(mod, 0.2)
    groups = max(gate, mod)
    rg = torch.randint(0, groups, (rows,), generator=g, device="cuda", dtype=torch.int32) if groups > 1 else None
    got_h, got_u = norm_residual(H, Y, post=post, post_gain=pg, post_bias=pb, gate=ga, residual_scale=rs, pre=pre,
                                 pre_gain=G, pre_bias=B, scale=sc, shift=sh, row_group=rg, eps=eps, u_dtype=t[u])
    rh, th, ru, tu = norm64(H, Y, post, pg, pb, ga, rs, pre, G, B, sc, sh, rg, eps, t[h], t[u])
    assert got_h.dtype == t[h] and got_u.dtype == t[u]
    within(got_h, rh, th, "h'")
    within(got_u, ru, tu, "u")
    clean()


@pytest.mark.parametrize("rows", [1, 17, 300])
@pytest.mark.parametrize("dim", [1, 2, 7, 8, 31, 40, 255, 256, 264, 1000, 1024, 1337, 2048, 4096, 4097, 5000, 8192,
                                 8200, 16384])
def test_norm_sizes(rows, dim):
    check_norm(rows, dim, post="layer", pre="rms", gate=1, mod=1)


@pytest.mark.parametrize("dim", [3, 5, 6, 127, 129, 1022, 1023, 1025, 1337, 2047, 4099, 16381, 16382, 16383])
@pytest.mark.parametrize("h, y, u", [("bf16", "bf16", "bf16"), ("f32", "bf16", "f32")])
def test_norm_widths_that_shift_the_rows(dim, h, y, u):
    """Rows that begin at every offset from an aligned address, with few rows and with many."""
    for rows in (9, 1300 if dim < 5000 else 300):
        check_norm(rows, dim, "rms", "layer", 1, 1, h=h, y=y, u=u)
    check_norm(40, dim, "layer", "rms", 7, 7, h=h, y=y, u=u)


def test_norm_strides_that_differ_between_the_matrices():
    """One matrix's rows shifted, the others' not: no common layout, value by value."""
    import torch
    from flow_matching_dit_b200 import norm_residual
    g = gen(5)
    wide = rnd(g, 50, 517)
    y = rnd(g, 50, 512, dtype=torch.bfloat16)
    for h in (wide[:, :512], wide[:, 1:513], wide[:, 4:516]):
        out_h, out_u = torch.zeros(50, 515, device="cuda")[:, 3:], torch.zeros(50, 514, device="cuda", dtype=torch.bfloat16)[:, :512]
        want = norm_residual(h.contiguous(), y, pre="layer")
        got = norm_residual(h, y, pre="layer", out_h=out_h, out_u=out_u)
        for a, b in zip(got, want):   # the sums run in another order
            assert torch.allclose(a.float(), b.float(), rtol=2 ** -8, atol=1e-6)
    clean()


@pytest.mark.parametrize("post", [None, "layer", "rms"])
@pytest.mark.parametrize("pre", [None, "layer", "rms"])
@pytest.mark.parametrize("gate, mod", [(0, 0), (1, 0), (0, 1), (5, 5), (1, 3), (3, 1)])
def test_norm_forms(post, pre, gate, mod):
    check_norm(57, 264, post, pre, gate, mod, rs=0.7)


@pytest.mark.parametrize("h", ["f32", "bf16"])
@pytest.mark.parametrize("y", ["f32", "bf16", None])
@pytest.mark.parametrize("u", ["f32", "bf16"])
@pytest.mark.parametrize("bad_alignment", [False, True])
def test_norm_types(h, y, u, bad_alignment):
    check_norm(33, 520, "rms" if y else None, "layer", 1 if y else 0, 2, h, y, u, rs=1.25, bad_alignment=bad_alignment)


def test_norm_of_a_large_mean_keeps_its_digits():
    """Deviations of 1e-3 of the mean: the variance may not be a difference of two large sums."""
    check_norm(64, 1024, None, "layer", offset=3000.0, y=None, u="f32")
    check_norm(64, 1001, "layer", "layer", offset=3000.0, y="f32", u="f32")


def test_norm_many_rows_and_long_offsets():
    """More rows than one pass of the grid, and rows beyond 2^31 elements."""
    import torch
    from flow_matching_dit_b200 import norm_residual
    check_norm(40000, 64, "rms", "rms", gate=7, mod=7)
    rows, dim = 140000, 16384   # 2.3e9 elements
    big = torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda")
    big[-3:] = rnd(gen(1), 3, dim, dtype=torch.bfloat16)
    out = torch.empty_like(big)
    _, u = norm_residual(big, pre="rms", eps=0.25, out_u=out)
    ref = big[-3:].double()
    ref = ref / torch.sqrt((ref ** 2).mean(1, keepdim=True) + 0.25)
    within(u[-3:], ref, U16 * ref.abs() + 64 * U32 * ref.abs())
    assert not u[:-3].any()
    clean()


def test_norm_in_place_and_outputs_left_out():
    import torch
    from flow_matching_dit_b200 import norm_residual
    g = gen(4)
    h, y = rnd(g, 50, 264), rnd(g, 50, 264, dtype=torch.bfloat16)
    want_h, want_u = norm_residual(h, y, pre="layer")
    same, none = norm_residual(h, y)
    assert none is None and torch.equal(same, want_h)
    h1 = h.clone()
    got, u = norm_residual(h1, None, pre="rms")
    assert got is h1 and torch.equal(h1, h)
    y1 = y.clone()
    got, u = norm_residual(h1, y1, pre="layer", out_h=h1, out_u=y1)
    assert got is h1 and u is y1 and torch.equal(h1, want_h) and torch.equal(y1, want_u)
    got, u = norm_residual(h, residual_scale=0.5)
    assert u is None and torch.equal(got, h * 0.5)
    clean()


def test_norm_bad_groups_are_reported_and_their_rows_are_nan():
    import torch
    from flow_matching_dit_b200 import _lib, norm_residual, op_status
    g = gen(5)
    h, gate = rnd(g, 6, 256), rnd(g, 3, 256)
    y = rnd(g, 6, 256, dtype=torch.bfloat16)
    rg = torch.tensor([0, 3, 2, -1, 1, 2147483647], dtype=torch.int32, device="cuda")
    got, u = norm_residual(h, y, gate=gate, pre="rms", row_group=rg)
    bad = torch.tensor([False, True, False, True, False, True], device="cuda")
    assert torch.isnan(got[bad]).all() and torch.isnan(u[bad]).all()
    assert torch.isfinite(got[~bad]).all() and torch.isfinite(u[~bad]).all()
    assert op_status() == _lib.GDIT_EDEVICE
    assert op_status() == 0


def test_norm_refusals():
    import torch
    from flow_matching_dit_b200 import norm_residual
    h = torch.zeros(4, 64, device="cuda")
    y = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    for kw, err in ((dict(gate=torch.zeros(2, 64, device="cuda")), ValueError),          # no row_group
                    (dict(pre="batch"), ValueError),
                    (dict(pre="layer", pre_gain=torch.zeros(63, device="cuda")), ValueError),
                    (dict(pre="layer", pre_gain=torch.zeros(64)), TypeError),
                    (dict(pre_gain=torch.zeros(64, device="cuda")), ValueError),
                    (dict(post_gain=torch.zeros(64, device="cuda")), ValueError),
                    (dict(u_dtype=torch.float16), TypeError),
                    (dict(out_h=y), TypeError),
                    (dict(scale=torch.zeros(2, 64, device="cuda"), shift=torch.zeros(3, 64, device="cuda"),
                          row_group=torch.zeros(4, device="cuda", dtype=torch.int32)), ValueError)):
        with pytest.raises(err):
            norm_residual(h, y, **kw)
    with pytest.raises(ValueError):
        norm_residual(h, y[:3])
    with pytest.raises(ValueError):
        norm_residual(h, post="rms")
    with pytest.raises(ValueError):
        norm_residual(h)
    a, b = norm_residual(h[:0], y[:0], pre="rms")
    assert a.shape == b.shape == (0, 64)


# ---------------------------------------------------------------------------------------------- attention

def attention64(q, k, v, ql, kl, ks, causal, scale):
    """(out, its tolerance, lse, its tolerance) in 64 bits, sequence by sequence; ks: first key of each."""
    import torch
    heads, kv_heads, dim = q.shape[1], k.shape[1], q.shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    ltol = torch.zeros_like(lse)
    at = 0
    for nq, nk, k0 in zip(ql, kl, ks):
        if nq and nk:
            kk = k[k0:k0 + nk].double().repeat_interleave(heads // kv_heads, 1).transpose(0, 1)
            vv = v[k0:k0 + nk].double().repeat_interleave(heads // kv_heads, 1).transpose(0, 1)
            qq = q[at:at + nq].double().transpose(0, 1)
            s = qq @ kk.transpose(1, 2) * scale
            e = (dim / 16 + 16) * 2.0 ** -23 * abs(scale) * (qq.abs() @ kk.abs().transpose(1, 2)).amax(-1)
            if causal:
                i = torch.arange(nq, device="cuda")[:, None] + (nk - nq)
                s = s.masked_fill(torch.arange(nk, device="cuda")[None] > i, -math.inf)
            l = torch.logsumexp(s, -1)
            p = torch.exp(s - l.clamp_min(-1e300)[..., None])
            o = p @ vv
            mag = p @ vv.abs()
            out[at:at + nq] = o.transpose(0, 1)
            lse[at:at + nq] = l.t()
            t = mag * (U16 + 2.0 ** -16 + 2 * e[..., None])
            tol[at:at + nq] = (t + U16 * (o.abs() + t)).transpose(0, 1)
            ltol[at:at + nq] = (e + 2.0 ** -16 + 4 * U32 * l.abs().nan_to_num(posinf=0)).t()
        at += nq
    return out, tol + 1e-30, lse, ltol + 1e-30


def check_attention(ql, kl=None, heads=4, kv_heads=2, dim=128, causal=True, slot=None, fused=False, seed=0, std=1.0,
                    scale=None, extra_q=0, garbage=float("nan"), max_q=None, max_k=None):
    """kl None: the queries' lengths.  slot: keys in slots of that many rows, filled with `garbage` behind each length.
    extra_q: rows behind the last sequence, which stay as they were."""
    import torch
    from flow_matching_dit_b200 import attention
    kl = list(ql) if kl is None else kl
    g = gen(seed + sum(ql) * 3 + sum(kl) + heads + dim)
    bf = torch.bfloat16
    tq = sum(ql) + extra_q
    if slot is None:
        ks = [int(x) for x in np.cumsum([0] + list(kl))]
        tk = ks[-1] + (extra_q if fused else 5)
    else:
        ks = [i * slot for i in range(len(kl) + 1)]
        tk = ks[-1]
    if fused:
        assert tq == tk
        qkv = rnd(g, tq, heads + 2 * kv_heads, dim, std=std, dtype=bf)
        q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
    else:
        q, k, v = (rnd(g, n, h, dim, std=std, dtype=bf) for n, h in ((tq, heads), (tk, kv_heads), (tk, kv_heads)))
    used = torch.zeros(tk, dtype=torch.bool, device="cuda")
    for k0, n in zip(ks, kl):
        used[k0:k0 + n] = True
    if not fused:
        k[~used] = garbage
        v[~used] = garbage
    cu = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cq, ck = cu([int(x) for x in np.cumsum([0] + list(ql))]), cu(ks)
    out = torch.full((tq, heads, dim), 7.0, dtype=bf, device="cuda")
    sc = dim ** -0.5 if scale is None else scale
    mq, mk = max(ql) if max_q is None else max_q, max(kl) if max_k is None else max_k
    got, lse = attention(q, k, v, cq, ck, max_q=mq, max_k=mk, causal=causal, scale=scale,
                         k_len=cu(kl) if slot is not None else None, out=out, return_lse=True)
    assert got is out
    n = sum(ql)
    assert (out[n:] == 7.0).all()
    ref, tol, rl, tl = attention64(q[:n], k, v, ql, kl, ks, causal, sc)
    within(out[:n], ref, tol, "out")
    within(lse[:n], rl, tl, "lse")
    clean()
    return q, k, v, cq, ck, out, lse


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 511, 700])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_lengths(n, causal):
    check_attention([n], causal=causal)


@pytest.mark.parametrize("dim", [8, 16, 24, 32, 40, 64, 72, 80, 96, 104, 120, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_widths(dim, causal):
    check_attention([70, 3, 300], dim=dim, causal=causal)


@pytest.mark.parametrize("heads, kv_heads", [(1, 1), (2, 1), (3, 1), (5, 1), (7, 1), (8, 1), (14, 2), (16, 16),
                                             (20, 4), (32, 4), (36, 3), (48, 1), (128, 1)])
def test_attention_head_groups(heads, kv_heads):
    check_attention([37, 260], heads=heads, kv_heads=kv_heads, dim=64)
    check_attention([1, 1, 1], [200, 1, 513], heads=heads, kv_heads=kv_heads, dim=64)


@pytest.mark.parametrize("ql", [[0, 5, 0, 0, 130, 1, 0], [1] * 70, [0, 0, 9], [600, 200, 333, 417, 599, 1, 2, 256]])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_ragged_batches(ql, causal):
    check_attention(ql, causal=causal, extra_q=6, heads=6, kv_heads=2, dim=64)
    check_attention(ql, causal=causal, extra_q=6, fused=True, heads=2, kv_heads=2)


@pytest.mark.parametrize("ql, kl", [
    ([5, 60, 128], [100, 700, 129]), ([1, 2, 3], [1000, 128, 3]), ([130], [2000]), ([64, 64], [64, 4096]),
    ([4, 9, 200, 30], [0, 5, 120, 30]),      # no keys at all; fewer keys than queries: the first queries see none
    ([16] * 9, [0, 1, 15, 16, 17, 127, 128, 129, 300]), ([300, 1], [40, 0]),
])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_pieces_and_empty_rows(ql, kl, causal):
    check_attention(ql, kl, causal=causal)
    check_attention(ql, kl, causal=causal, slot=max(kl) + 3, dim=64)


@pytest.mark.parametrize("kl", [[1], [7], [128], [129], [5000], [3, 4096, 0, 77, 1024, 1025], [33] * 40, [70000]])
@pytest.mark.parametrize("heads, kv_heads, dim", [(4, 4, 64), (8, 2, 128), (7, 1, 72)])
def test_attention_single_token(kl, heads, kv_heads, dim):
    check_attention([1] * len(kl), kl, heads=heads, kv_heads=kv_heads, dim=dim, slot=max(kl) + 1)


@pytest.mark.parametrize("batch", [255, 256, 257, 700])
def test_attention_many_sequences(batch):
    """Single tokens of more sequences than are taken by falling length, and of as many."""
    kl = [int(x) for x in np.random.RandomState(batch).randint(0, 300, batch)]
    check_attention([1] * batch, kl, 4, 2, 64, slot=300)
    check_attention([i % 3 for i in range(batch)], [min(i % 3, n) + n for i, n in enumerate(kl)], 2, 1, 64)


@pytest.mark.parametrize("heads, kv_heads", [(16, 1), (17, 1), (32, 1), (64, 1), (65, 1), (128, 1), (96, 2)])
@pytest.mark.parametrize("nq", [1, 4])
def test_attention_wide_groups(heads, kv_heads, nq):
    """Tiles of 16, 64 and 128 rows, full and nearly empty."""
    check_attention([nq] * 3, [700, nq, 129 + nq], heads, kv_heads, 64, slot=705)


@pytest.mark.parametrize("heads, kv_heads, dim", [(2, 1, 128), (7, 1, 64), (12, 4, 80), (5, 5, 40)])
@pytest.mark.parametrize("ql, kl", [([300], [5000]), ([70, 1, 64], [3000, 400, 64]), ([129], [129]), ([65, 0, 200], [65, 7, 300])])
def test_attention_few_tiles(heads, kv_heads, dim, ql, kl):
    """Too few tiles for the SMs: parts of the keys, joined over clusters."""
    for causal in (True, False):
        check_attention(ql, kl, heads, kv_heads, dim, causal)


@pytest.mark.parametrize("nq", [2, 3, 5, 8, 16, 33])
def test_attention_few_tokens(nq):
    """The tokens of a draft, checked in one call."""
    check_attention([nq, 1, 0, nq], [1000, 64, 50, nq], heads=4, kv_heads=1, slot=1024, dim=64)


@pytest.mark.parametrize("garbage", [float("nan"), float("inf"), -3.0e38])
def test_attention_what_lies_outside_a_sequence_does_not_matter(garbage):
    check_attention([50, 3], [50, 140], slot=300, garbage=garbage)
    check_attention([1, 1], [50, 140], slot=300, garbage=garbage)


def test_attention_values_of_another_sequence_do_not_leak():
    import torch
    from flow_matching_dit_b200 import attention
    for nq in (100, 1):
        q, k, v, cq, ck, out, lse = check_attention([nq, nq, nq], [100, 90, 110], extra_q=0)
        k2, v2 = k.clone(), v.clone()
        k2[100:190], v2[100:190] = float("nan"), float("inf")
        got, l2 = attention(q, k2, v2, cq, ck, max_q=nq, max_k=110, return_lse=True)
        keep = torch.tensor([True] * nq + [False] * nq + [True] * nq, device="cuda")
        assert torch.equal(got[keep], out[keep]) and torch.equal(l2[keep], lse[keep])
    clean()


@pytest.mark.parametrize("std, scale", [(1.0, 0.0), (1.0, -0.3), (6.0, None), (30.0, None), (1.0, 20.0), (1e-3, None)])
def test_attention_scores_of_all_sizes(std, scale):
    """Flat, sharp and negative scales; scores of thousands."""
    check_attention([300, 40], std=std, scale=scale, dim=64)
    check_attention([1, 1], [900, 40], std=std, scale=scale, dim=64)


@pytest.mark.parametrize("nq, nk", [(2048, 2048), (4096, 4096), (513, 6000)])
def test_attention_long(nq, nk):
    check_attention([nq], [nk], heads=2, kv_heads=1, dim=128)


def test_attention_upper_bounds_may_be_loose():
    import torch
    a = check_attention([30, 200], max_q=200, max_k=200)[5]
    b = check_attention([30, 200], max_q=5000, max_k=9000)[5]
    within(a, b.double(), 2 * U16 * b.double().abs() + U16)
    a = check_attention([1, 1], [30, 200], max_q=1, max_k=200)[5]
    b = check_attention([1, 1], [30, 200], max_q=1, max_k=100000)[5]
    within(a, b.double(), 2 * U16 * b.double().abs() + U16)


def test_attention_in_place_of_q():
    import torch
    from flow_matching_dit_b200 import attention
    for ql, kl in (([300, 77], [300, 77]), ([1, 1], [300, 77])):
        q, k, v, cq, ck, out, _ = check_attention(ql, kl, heads=6, kv_heads=2)
        assert attention(q, k, v, cq, ck, max_q=max(ql), max_k=max(kl), out=q) is q
        assert torch.equal(q, out)
    clean()


def test_attention_long_cache_offsets():
    """A cache whose elements pass 2^31: the last slots are read at 64-bit offsets."""
    import torch
    from flow_matching_dit_b200 import attention
    slot, b, kv, dim = 70000, 36, 8, 128   # 2.6e9 elements each
    k = torch.zeros(b * slot, kv, dim, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    g = gen(3)
    kl = [200 + i for i in range(b)]
    for i in (0, b - 1):
        k[i * slot:i * slot + kl[i]] = rnd(g, kl[i], kv, dim, dtype=torch.bfloat16)
        v[i * slot:i * slot + kl[i]] = rnd(g, kl[i], kv, dim, dtype=torch.bfloat16)
    ck = torch.arange(0, (b + 1) * slot, slot, dtype=torch.int32, device="cuda")
    for nq in (1, 150):
        q = rnd(g, b * nq, 16, dim, dtype=torch.bfloat16)
        cq = torch.arange(0, (b + 1) * nq, nq, dtype=torch.int32, device="cuda")
        out = attention(q, k, v, cq, ck, max_q=nq, max_k=max(kl),
                        k_len=torch.tensor(kl, dtype=torch.int32, device="cuda"))
        for i in (0, b - 1):
            ref, tol, _, _ = attention64(q[i * nq:(i + 1) * nq], k[i * slot:], v[i * slot:], [nq], [kl[i]], [0], True,
                                         dim ** -0.5)
            within(out[i * nq:(i + 1) * nq], ref, tol, f"slot {i}")
    clean()


@pytest.mark.parametrize("nq", [1, 40])
def test_attention_bad_offsets_are_reported_and_skipped(nq):
    """A length above max_q or max_k, offsets past the tensors, k_len past its slot: the good sequences are computed."""
    import torch
    from flow_matching_dit_b200 import _lib, attention, op_status
    g = gen(8)
    q = rnd(g, 3 * nq, 2, 64, dtype=torch.bfloat16)
    k, v = (rnd(g, 120, 1, 64, dtype=torch.bfloat16) for _ in range(2))
    cu = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    good_q, good_k = cu(0, nq, 2 * nq, 3 * nq), cu(0, 40, 80, 120)
    ref = attention(q, k, v, good_q, good_k, max_q=nq, max_k=40)
    assert op_status() == 0
    fill = lambda: torch.full_like(q, 5.0)  # noqa: E731
    for cq, ck, kw in ((cu(0, nq, 2 * nq, 3 * nq + 1), good_k, {}), (good_q, cu(0, 40, 80, 121), {}),
                       (good_q, good_k, dict(k_len=cu(40, 40, 41))), (good_q, good_k, dict(k_len=cu(40, 40, -1))),
                       (good_q, cu(0, 40, 80, 2147483647), {}), (cu(0, nq, 2 * nq, -2147483647), good_k, {})):
        out = attention(q, k, v, cq, ck, max_q=nq, max_k=40, out=fill(), **kw)
        assert op_status() == _lib.GDIT_EDEVICE
        assert torch.equal(out[:2 * nq], ref[:2 * nq]) and (out[2 * nq:] == 5.0).all()
    out = attention(q, k, v, good_q, cu(0, 40, 79, 120), max_q=nq, max_k=40, out=fill())   # 41 keys, at most 40
    assert op_status() == _lib.GDIT_EDEVICE
    assert torch.equal(out[:nq], ref[:nq]) and (out[2 * nq:] == 5.0).all()
    assert op_status() == 0


def test_attention_refusals():
    import torch
    from flow_matching_dit_b200 import GditError, attention
    q = torch.zeros(8, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(8, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    ok = dict(max_q=8, max_k=8)
    for args, err in (((q.float(), k, k, cu, cu), TypeError), ((q, k[:, :, :32], k, cu, cu), ValueError),
                      ((q, k, k[:7], cu, cu), ValueError), ((q, k, k, cu.long(), cu), TypeError),
                      ((q, k, k, cu, cu[:1]), ValueError), ((q, k, k, cu.cpu(), cu), TypeError),
                      ((q[:, :3], k, k, cu, cu), GditError), ((q[0], k, k, cu, cu), ValueError)):
        with pytest.raises(err):
            attention(*args, **ok)
    with pytest.raises(GditError):
        attention(q, k, k, cu, cu, max_q=-1, max_k=8)
    with pytest.raises(ValueError):
        attention(q, k, k, cu, cu, out=q[:, :2], **ok)
    empty = attention(q[:0], k[:0], k[:0], cu[:1], cu[:1], **ok)
    assert empty.shape == (0, 4, 64)
    out, lse = attention(q, k[:0], k[:0], cu, torch.zeros_like(cu), return_lse=True, **ok)   # no key anywhere
    assert not out.any() and torch.isinf(lse).all()


# ---------------------------------------------------------------------------------------------- together

def block(x, w, cu, n, heads, kv_heads, dim, norm, lin, att):
    """One transformer block on the residual stream x over packed sequences."""
    h, u = norm(x, None, pre="layer", pre_gain=w["g1"], pre_bias=w["b1"])
    qkv = lin(u, w["qkv"], w["qkv_b"]).view(-1, heads + 2 * kv_heads, dim)
    o = att(qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:], cu, cu, max_q=n, max_k=n)
    y = lin(o.reshape(x.shape[0], -1), w["o"], w["o_b"])
    h, u = norm(h, y, post="rms", post_gain=w["g2"], gate=w["gate"], pre="rms", pre_gain=w["g3"])
    f = lin(u, w["f1"], w["f1_b"], activation="gelu")
    return lin(f, w["f2"], w["f2_b"], residual=h, out_dtype=x.dtype)


def block_inputs(lens, width, heads, kv_heads, dim, seed=0):
    import torch
    g = gen(seed)
    bf = torch.bfloat16
    x = rnd(g, sum(lens), width)
    mat = lambda n, k: rnd(g, n, k, std=k ** -0.5, dtype=bf)  # noqa: E731
    vec = lambda n, add=0.0: rnd(g, n, std=0.1) + add  # noqa: E731
    w = dict(g1=vec(width, 1), b1=vec(width), qkv=mat((heads + 2 * kv_heads) * dim, width),
             qkv_b=vec((heads + 2 * kv_heads) * dim), o=mat(width, heads * dim), o_b=vec(width), g2=vec(width, 1),
             gate=vec(width, 0.5), g3=vec(width, 1), f1=mat(4 * width, width), f1_b=vec(4 * width),
             f2=mat(width, 4 * width), f2_b=vec(width))
    cu = torch.tensor([int(c) for c in np.cumsum([0] + list(lens))], dtype=torch.int32, device="cuda")
    return x, w, cu


def block64(x, w, lens, heads, kv_heads, dim):
    import torch
    w = {k: t.double() for k, t in w.items()}

    def norm(h, y, post=None, post_gain=None, gate=None, pre=None, pre_gain=None, pre_bias=None):
        one = torch.float64
        v, _, u, _ = norm64(h, y, post, post_gain, None, gate, 1.0, pre, pre_gain, pre_bias, None, None, None, 1e-5, one, one)
        return v, u

    def lin(a, m, b, activation="none", residual=None, out_dtype=None):
        z = act64(a @ m.t() + b, activation)
        return z if residual is None else z + residual

    def att(q, k, v, cu, *_, **__):
        ks = [int(c) for c in np.cumsum([0] + list(lens))]
        return attention64(q, k, v, lens, lens, ks, True, dim ** -0.5)[0]

    return block(x.double(), w, None, max(lens), heads, kv_heads, dim, norm, lin, att)


@pytest.mark.parametrize("lens, width, heads, kv_heads, dim", [
    ([33, 200, 1, 97], 256, 4, 2, 64), ([300], 512, 4, 1, 128), ([17] * 40, 384, 6, 6, 64),
])
def test_block_of_the_operators(lens, width, heads, kv_heads, dim):
    """Seven calls as a block makes them, eagerly, then captured and replayed on other inputs.  About ten roundings to
    bf16 (each 2^-9 of its value on average) lie between x and what the block adds to it: 2 % of that is out of reach."""
    import torch
    from flow_matching_dit_b200 import attention, linear, norm_residual
    x, w, cu = block_inputs(lens, width, heads, kv_heads, dim)
    run = lambda t: block(t, w, cu, max(lens), heads, kv_heads, dim, norm_residual, linear, attention)  # noqa: E731
    got, ref = run(x), block64(x, w, lens, heads, kv_heads, dim)
    rel = lambda a, b, base: float((a.double() - b).norm() / (b - base).norm())  # noqa: E731
    assert rel(got, ref, x.double()) < 2e-2
    clean()
    graph, static = torch.cuda.CUDAGraph(), x.clone()
    with torch.cuda.graph(graph):
        out = run(static)
    for seed in (5, 6):
        x2 = block_inputs(lens, width, heads, kv_heads, dim, seed)[0]
        static.copy_(x2)
        graph.replay()
        assert torch.equal(out, run(x2))
    clean()


def test_two_streams_at_once():
    """Two streams run blocks side by side, each many times: no state is shared between calls."""
    import torch
    from flow_matching_dit_b200 import attention, linear, norm_residual
    cases = [([33, 200, 1, 97], 256, 4, 2, 64), ([300, 20], 512, 4, 1, 128)]
    made = [block_inputs(*c, seed=i) for i, c in enumerate(cases)]

    def run(c, m):
        lens, width, heads, kv_heads, dim = c
        return block(m[0], m[1], m[2], max(lens), heads, kv_heads, dim, norm_residual, linear, attention)

    want = [run(c, m) for c, m in zip(cases, made)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(run(cases[i], made[i]))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(t, w) for t in g)
    clean()


def test_captured_graphs_side_by_side():
    """Two captured graphs replay on two streams at once, again and again, with new inputs: nothing is shared."""
    import torch
    from flow_matching_dit_b200 import attention, linear, norm_residual
    g = gen(11)
    bf = torch.bfloat16
    cu = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = [rnd(g, 4096, 2, 128, dtype=bf) for _ in range(2)]
    w1, w2, gain = rnd(g, 1024, 1024, std=0.03, dtype=bf), rnd(g, 1024, 1024, std=0.03, dtype=bf), rnd(g, 1024)
    cq, ck, kl = cu(0, 1, 2), cu(0, 2048, 4096), cu(2048, 1500)

    def step(x):
        h, u = norm_residual(x, None, pre="rms", pre_gain=gain, u_dtype=bf)
        q = linear(u, w1, activation="silu").view(2, 8, 128)
        o = attention(q, *cache, cq, ck, max_q=1, max_k=2048, k_len=kl).view(2, 1024)
        return linear(o, w2, residual=h, out_dtype=torch.float32)

    xs = [[rnd(g, 2, 1024) for _ in range(5)] for _ in range(2)]
    want = [[step(x) for x in row] for row in xs]
    streams, graphs = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for st in streams:
        x = torch.zeros(2, 1024, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            y = step(x)
        graphs.append((graph, x, y))
    got = [[], []]
    for i in range(5):
        for s, (st, (graph, x, y)) in enumerate(zip(streams, graphs)):
            with torch.cuda.stream(st):
                x.copy_(xs[s][i])
                graph.replay()
                got[s].append(y.clone())
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, r) for p, r in zip(a, b))
    clean()


def test_binding_refusals():
    import torch
    from flow_matching_dit_b200 import attention, linear, norm_residual
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    q, cu = x.view(8, 1, 64), torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    for f, err in ((lambda: linear(x, 1), TypeError), (lambda: linear(x, None), TypeError),
                   (lambda: linear(x, x, activation=3), ValueError), (lambda: linear(x, x, out_dtype="bf16"), TypeError),
                   (lambda: linear(x, x, torch.zeros(8, dtype=torch.float64, device="cuda")), TypeError),
                   (lambda: linear(x, x, torch.zeros(16, device="cuda")[::2]), TypeError),
                   (lambda: linear(x, x, stream="0"), TypeError),
                   (lambda: norm_residual(x, eps="no", pre="rms"), TypeError), (lambda: norm_residual(x, x, gate=3.0), TypeError),
                   (lambda: norm_residual(x, x, row_group=torch.zeros(8, device="cuda")), TypeError),
                   (lambda: norm_residual(x, x, pre="rms", eps=-1.0), RuntimeError),
                   (lambda: attention(q, q, q, cu, cu, max_q=1 << 40, max_k=8), ValueError),
                   (lambda: attention(q, q, q, cu, cu, max_q=1.5, max_k=8), TypeError),
                   (lambda: attention(q, q, q, cu, cu, max_q=8, max_k=8, scale="x"), TypeError),
                   (lambda: attention(q, q, q, cu, cu, max_q=8, max_k=8, k_len=cu), ValueError),
                   (lambda: attention(q, q, q, cu[:0], cu, max_q=8, max_k=8), ValueError)):
        with pytest.raises(err):
            f()
    clean()


def test_first_calls_of_a_process_inside_a_capture():
    """No set-up call is needed: every kernel's first call may be a captured one."""
    import subprocess
    import sys
    code = """
import torch
from flow_matching_dit_b200 import attention, linear, norm_residual, op_status
bf = torch.bfloat16
g = torch.Generator(device="cuda").manual_seed(0)
r = lambda *s: torch.randn(*s, generator=g, device="cuda")
x, w, wide = r(3, 1024).to(bf), r(512, 1024).to(bf), r(2048, 1024).to(bf)
h, y = r(40, 513), r(40, 513).to(bf)
q, kv, cq, ck = r(2, 8, 128).to(bf), r(6000, 2, 128).to(bf), torch.tensor([0, 1, 2]), torch.tensor([0, 3000, 6000])
p, cp = r(500, 8, 64).to(bf), torch.tensor([0, 200, 500])
cq, ck, cp = (t.int().cuda() for t in (cq, ck, cp))
def calls():
    return [linear(x, w), linear(wide, wide, activation="gelu"), *norm_residual(h, y, post="rms", pre="layer"),
            attention(q, kv, kv, cq, ck, max_q=1, max_k=3000), attention(p, p[:, :4], p[:, 4:], cp, cp, max_q=300, max_k=300)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = calls()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, calls())) and op_status() == 0
print("fine")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def test_on_a_stream_of_its_own_and_by_handle():
    import torch
    from flow_matching_dit_b200 import linear, op_status
    g = gen(12)
    x, w = (rnd(g, 64, 256, dtype=torch.bfloat16) for _ in range(2))
    want = linear(x, w)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    out = torch.zeros_like(want)
    linear(x, w, out=out, stream=st.cuda_stream)
    st.synchronize()
    assert torch.equal(out, want) and op_status(stream=st.cuda_stream) == 0


def test_same_bits_every_time():
    import torch
    from flow_matching_dit_b200 import attention, linear
    g = gen(2)
    bf = torch.bfloat16
    for m, n, k in ((1, 1024, 4096), (40, 520, 2048), (700, 1024, 1024)):
        x, w = rnd(g, m, k, dtype=bf), rnd(g, n, k, dtype=bf)
        first = linear(x, w, out_dtype=torch.float32)
        assert all(torch.equal(first, linear(x, w, out_dtype=torch.float32)) for _ in range(10))
    k, v = (rnd(g, 5000, 2, 128, dtype=bf) for _ in range(2))
    cu = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for nq in (1, 400):
        q = rnd(g, 2 * nq, 8, 128, dtype=bf)
        args = (q, k, v, cu(0, nq, 2 * nq), cu(0, 1900, 5000))
        first = attention(*args, max_q=nq, max_k=3100)
        assert all(torch.equal(first, attention(*args, max_q=nq, max_k=3100)) for _ in range(10))
    clean()
