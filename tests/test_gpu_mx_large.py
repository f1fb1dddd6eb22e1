"""The MX row kernels at sizes where a warp takes several pieces of a row and a column's sum comes
from many partial sums, against the fp64 reference."""

import numpy as np
import pytest
import torch

from oracle import mx
from test_gpu_mx import TYPES, Strided, bits, check_mx, saved, values, y_bound

pytestmark = pytest.mark.gpu

SHAPES = [(4096, 1024), (3000, 1032)]


@pytest.fixture(scope="module")
def tlg():
    import tiled_dense_gemm_tlg_b200 as t
    return t


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("act", ["relu", "gelu", "silu", "gelu_tanh"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward_with_sums(tlg, typ, act, rows, cols):
    rng = np.random.default_rng(rows + cols)
    Q, S, z = saved(rng.standard_normal((rows, cols)) * 2.5)
    dy = torch.from_numpy(rng.standard_normal((rows, cols))).to(TYPES[typ])
    d64 = dy.double().numpy()
    slope = mx.slope(act, z)
    want = d64 * slope
    half = torch.finfo(TYPES[typ]).eps / 2
    fn = np.abs(d64) * (1e-6 + 2.0 ** -23 * np.abs(slope))  # the slope, and one fp32 product
    bound = half * np.abs(want) * (1 + 1e-5) + fn + (2.0 ** -25 if typ == "f16" else 0.0)
    # every term's error, and the additions, whose chains are shorter than the plain one of `rows`
    sum_bound = fn.sum(axis=0) + (rows + 16) * 2.0 ** -24 * np.abs(want).sum(axis=0)
    first = None
    for lead, extra in ((0, 0), (8, 8), (1, 1)):
        m, o = Strided(dy, lead, extra), Strided(torch.zeros_like(dy), lead, extra)
        dz, db = tlg.tlg_act_backward_mx(m.view, Q, S, act, dZ=o.view)
        assert (np.abs(dz.double().cpu().numpy() - want) <= bound).all()
        assert (np.abs(db.double().cpu().numpy() - want.sum(axis=0)) <= sum_bound).all()
        assert m.guards_kept() and o.guards_kept()
        first = dz.clone() if first is None else first
        dz2, db2 = tlg.tlg_act_backward_mx(m.view, Q, S, act, dZ=m.view)  # in place
        assert torch.equal(bits(dz2), bits(first)) and torch.equal(db2, db) and m.guards_kept()


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_both_ways_and_back(tlg, typ, fmt, rows, cols):
    x = values(rows, cols, TYPES[typ], seed=cols)
    codes, scale = mx.quantize(x.double().numpy(), fmt)
    want = torch.from_numpy(mx.decode(codes, scale, fmt)[:, :cols]).float().to(TYPES[typ])
    for op, stored in (("N", x), ("T", x.t().contiguous())):
        Q, S = tlg.tlg_mx_quantize(stored.cuda(), format=fmt, op=op)
        check_mx(Q, S, codes, scale, fmt)
    assert torch.equal(bits(tlg.tlg_mx_dequantize(Q, S, cols, format=fmt, out=typ)), bits(want.cuda()))


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(tlg, typ, rows, cols):
    z = (torch.randn((rows, cols), generator=torch.Generator().manual_seed(rows)) * 3).clamp(-12, 12).to(TYPES[typ])
    codes, scale = mx.quantize(z.double().numpy(), "e4m3")
    for act in ("gelu", "silu"):
        want = mx.activate(act, z.double().numpy())
        Y, Q, S = tlg.tlg_act_forward_mx(z.cuda(), act)
        check_mx(Q, S, codes, scale, "e4m3")
        assert (np.abs(Y.double().cpu().numpy() - want) <= y_bound(act, typ, want, z.double().numpy())).all()


@pytest.mark.parametrize("odd", [0, 1])
def test_row_offsets_past_32_bits(tlg, odd):
    """Every matrix in rows so far apart that the last ones lie past 2^31 elements and 2^32 bytes."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB of free device memory")
    rows, cols = 5, 300
    ld = (1 << 31) // 4 + 64 + odd
    far = lambda dtype, ld, cols: torch.empty((rows * ld,), dtype=dtype, device="cuda").view(rows, ld)[:, :cols]
    x, y = far(torch.float16, ld, cols), far(torch.float16, ld, cols)
    q = far(torch.uint8, (1 << 30) + 64, 320)
    z = torch.randn((rows, cols), device="cuda").half()
    x.copy_(z)
    Y, Q, S = tlg.tlg_act_forward_mx(z, "gelu")
    S.zero_(), tlg.tlg_act_forward_mx(z, "gelu", Q=Q, S=S)
    s = torch.zeros_like(S)
    tlg.tlg_act_forward_mx(x, "gelu", Y=y, Q=q, S=s)
    assert torch.equal(y, Y) and torch.equal(q, Q) and torch.equal(s, S)
    tlg.tlg_mx_dequantize(q, s, cols, format="e4m3", out="f16", X=y)
    assert torch.equal(y, tlg.tlg_mx_dequantize(Q, S, cols, format="e4m3", out="f16"))
    want, db = tlg.tlg_act_backward_mx(z, Q, S, "gelu")
    got, db2 = tlg.tlg_act_backward_mx(x, q, s, "gelu", dZ=y)
    assert torch.equal(y, want) and torch.equal(db, db2)
