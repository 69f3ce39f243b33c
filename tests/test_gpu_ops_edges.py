"""The operators where their layouts, values or callers are unusual, against
the 64-bit forms and with the tolerances of test_gpu_ops."""

import pytest

from tests.gpu_util import require_gpu
from tests.test_gpu_ops import clean, gen, norm64, rnd, within

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


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
