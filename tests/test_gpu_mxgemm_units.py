"""tlg_gemm_mxfp4 with several tiles to a unit: the accumulators and ring phases, the columns that
the 256-wide accumulators share, the pieces that change warps from tile to tile, the bias loaded for
the next tile, and the output box used again, all of which a unit's first tile does not reach."""

import numpy as np
import pytest
import torch

from oracle import mx
from test_gpu_mxgemm import Out, TILES, TYPES, check, operand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tlg():
    import tiled_dense_gemm_tlg_b200 as t
    yield t
    rc, code = t.tlg_device_error()
    assert rc == 0, hex(code)


# Rows, columns and K of each tile's problem: 20 tiles and more, ragged, so that one to four units
# take 5 tiles or more each, with an even and an odd number of them.
SIZES = {64: (300, 449, 300), 128: (600, 513, 1300), 192: (820, 897, 300), 256: (1000, 1100, 1300)}


@pytest.mark.parametrize("units", [1, 2, 3, 4])
@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("cg,bn", TILES)
def test_many_tiles_to_a_unit(tlg, cg, bn, typ, units):
    M, N, K = SIZES[bn]
    assert -(-M // (128 * cg)) * -(-N // bn) >= 5 * units
    A, SA, a = operand(M, K, "exact", M)
    B, SB, b = operand(N, K, "exact", N)
    z = a @ b.T
    g = np.random.default_rng(units)
    bias = torch.from_numpy(g.integers(-64, 65, N) / 16).to(torch.bfloat16 if typ == "bf16" else torch.float16).cuda()
    R = torch.from_numpy(g.integers(-64, 65, (M, N)) / 16).to(TYPES[typ])
    cfg = {"cta_group": cg, "block_n": bn, "max_ctas": units * cg}
    for lead, extra in ((0, 0), (8, 8), (1, 1)):
        # Every sum is a multiple of 1/16 below 2^20: the only rounding is the last one.
        o = Out(M, N, TYPES[typ], lead, extra)
        tlg.tlg_gemm_mxfp4(A, SA, B, SB, C=o.view, out=typ, config=cfg)
        check(o.view, z, 0.0, typ)
        assert o.guards_kept()
        r = Out(M, N, TYPES[typ], lead, extra, R)
        want = np.maximum(z + bias.double().cpu().numpy(), 0) + R.double().numpy()
        for c in (o, r):  # into another matrix, then in place
            tlg.tlg_gemm_mxfp4(A, SA, B, SB, bias=bias, activation="relu", residual=r.view, C=c.view, out=typ, config=cfg)
            check(c.view, want, 0.0, typ)
            assert c.guards_kept()
        tlg.tlg_gemm_mxfp4(A, SA, B, SB, bias=bias, C=o.view, out=typ, config=cfg)
        check(o.view, z + bias.double().cpu().numpy(), 0.0, typ)
        assert o.guards_kept()


@pytest.mark.parametrize("cg,bn", TILES)
@pytest.mark.parametrize("raster", [1, 3, 64])
def test_raster_groups(tlg, cg, bn, raster):
    M, N, K = SIZES[bn]
    A, SA, a = operand(M, K, "exact", 1)
    B, SB, b = operand(N, K, "exact", 2)
    for units in (2, 5):
        C = tlg.tlg_gemm_mxfp4(A, SA, B, SB, out="f32", config={"cta_group": cg, "block_n": bn, "max_ctas": units * cg,
                                                                "raster_group": raster})
        assert np.array_equal(C.cpu().numpy(), a @ b.T)


@pytest.mark.parametrize("act", ["gelu", "silu", "gelu_tanh"])
@pytest.mark.parametrize("cg,bn", TILES)
def test_activations_over_many_tiles(tlg, cg, bn, act):
    """A unit's tiles one after the other give the bits that one tile to a unit gives."""
    M, N, K = SIZES[bn]
    A, SA, _ = operand(M, K, "exact", 3)
    B, SB, _ = operand(N, K, "exact", 4)
    SA, SB = ((s.int() - 3).clamp(min=0).to(torch.uint8) for s in (SA, SB))
    for typ in TYPES:
        bias = torch.randn(N, device="cuda").to(torch.bfloat16 if typ == "bf16" else torch.float16)
        R = torch.randn((M, N), device="cuda").to(TYPES[typ])
        run = lambda **cfg: tlg.tlg_gemm_mxfp4(A, SA, B, SB, bias=bias, activation=act, residual=R, out=typ,
                                               config={"cta_group": cg, "block_n": bn, **cfg})
        want = run()
        assert torch.isfinite(want).all()
        for units in (1, 3):
            assert torch.equal(run(max_ctas=units * cg), want)
