"""The activations' derivatives in tlg_act_backward_mx at the ends of their range: saved values that
decode to infinity, the negative side of GELU where the derivative is small, and the identity."""

import numpy as np
import pytest
import torch

from oracle import mx

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "gelu", "silu", "gelu_tanh"]


@pytest.fixture(scope="module")
def tlg():
    import tiled_dense_gemm_tlg_b200 as t
    return t


def saved(z):
    codes, scale = mx.quantize(z, "e4m3")
    return torch.from_numpy(mx.pack(codes, "e4m3")).cuda(), torch.from_numpy(mx.tile_scales(scale, 255)).cuda()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("typ", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cols", [64, 300, 2048])
def test_largest_inputs(tlg, act, typ, cols):
    """The type's largest value is saved as 2^128, which fp32 reads back as infinity; the derivative
    there is 1, and on the negative side 0 (1 for the identity)."""
    rows = 40
    z = torch.zeros((rows, cols), dtype=typ)
    z[1::2, 0::3] = torch.finfo(typ).max
    z[1::2, 1::3] = -torch.finfo(typ).max
    Y, Q, S = tlg.tlg_act_forward_mx(z.cuda(), act)
    assert torch.isinf(tlg.tlg_mx_dequantize(Q, S, cols, format="e4m3", out="f32")).any()
    dy = torch.randint(-8, 9, (rows, cols), generator=torch.Generator().manual_seed(cols)).to(typ)
    dz, db = tlg.tlg_act_backward_mx(dy.cuda(), Q, S, act)
    zf = z.double()
    at_zero = {"none": 1.0, "relu": 0.0}.get(act, 0.5)
    slope = torch.where(zf > 0, 1.0, torch.where(zf < 0, 1.0 if act == "none" else 0.0, at_zero))
    want = dy.double() * slope
    # |dY| <= 8 times the derivative's error, and a rounding of 4 or less
    bound = 8e-6 + 4 * torch.finfo(typ).eps / 2
    assert ((dz.double().cpu() - want).abs() <= bound).all()
    # sums of multiples of 1/2, each term within 8e-6
    assert ((db.double().cpu() - want.sum(dim=0)).abs() <= rows * 8e-6 + rows * 2.0 ** -24 * 8 * rows).all()


def test_gelu_slope_keeps_relative_accuracy(tlg):
    """Saved values of three mantissa bits come back exactly.  The derivative's fit is within 1e-5
    of it, relatively, on [-12, -2] (checked on the CPU with its roundings); the hardware's exp2 and
    reciprocal add at most 2^-22 each."""
    v = np.array([-2, -2.5, -3, -3.5, -4, -4.5, -5, -5.5, -6, -6.5, -7, -8, -9, -10, -12])
    Q, S = saved(np.repeat(v[:, None], 96, axis=1))
    dy = torch.full((len(v), 96), 1024.0, device="cuda")
    dz = tlg.tlg_act_backward_mx(dy, Q, S, "gelu")[0].double().cpu().numpy() / 1024
    want = mx.slope("gelu", v)[:, None]
    assert (np.abs(dz / want - 1) < 2e-5).all(), np.abs(dz / want - 1).max(axis=1)
    v = np.array([-14, -100, -1e30])  # further out it is 0 to fp32's smallest numbers
    Q, S = saved(np.repeat(v[:, None], 96, axis=1))
    dz = tlg.tlg_act_backward_mx(dy[:3], Q, S, "gelu")[0]
    assert (dz.abs() < 1e-37).all()


@pytest.mark.parametrize("typ", [torch.float32, torch.float16, torch.bfloat16])
def test_identity_passes_the_gradient(tlg, typ):
    """The identity's derivative is 1 whatever Z holds, a NaN block included."""
    z = np.random.default_rng(0).standard_normal((33, 200))
    z[5, 40] = np.nan
    Q, S = saved(z)
    dy = torch.randn((33, 200), device="cuda").to(typ)
    dz, _ = tlg.tlg_act_backward_mx(dy, Q, S, "none")
    assert torch.equal(dz, dy)
