"""How exact the weight gradient of the root-mean-square norm is: the sum over the rows of dY * H * rstd, against 64 bits.

Tolerance, of the 2-norm of the error over all columns relative to that of the result: a rounding to fp32 has a
root-mean-square error of at most 2^-24 / sqrt(3) = 3.4e-8 of the value.  Every term has two, which in a sum of random
signs is 3.4e-8 sqrt(2) of the result.  A CTA adds its rows in fp32, the sum so far of n rows being sqrt(n) terms: over a
chain of r rows sqrt(2 + .. + r) 3.4e-8 terms, which is 3.4e-8 sqrt((r + 1) / 2) of sqrt(r) terms.  The CTAs' sums are
added in 64 bits and rounded once more: 3.4e-8.  In quadrature 3.4e-8 sqrt(3 + (r + 1) / 2); r is 4 at 1000 x 3001 and at
most 8 in what follows."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(1000, 3001), (1000, 4096), (2000, 512), (1100, 9000)])
def test_weight_gradient(rows, cols):
    import tiled_dense_gemm_tlg_b200 as tlg

    gen = torch.Generator(device="cuda").manual_seed(1)
    dY, H = (torch.randn((rows, cols), generator=gen, device="cuda") for _ in range(2))
    w = torch.ones(cols, device="cuda")
    rstd = torch.rand(rows, generator=gen, device="cuda") + 0.5
    _, dweight = tlg.tlg_rmsnorm_backward(dY, H, w, rstd)
    want = (dY.double() * H.double() * rstd.double()[:, None]).sum(dim=0)
    error = ((dweight.double() - want).norm() / want.norm()).item()
    assert error <= 2.0 ** -24 / 3 ** 0.5 * (3 + (8 + 1) / 2) ** 0.5, error
