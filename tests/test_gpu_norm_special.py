"""GPU tests of the root-mean-square norm on rows that are not finite, or whose sum of squares is not: what the formula
gives in fp32, in Y and in every block of its microscaled forms."""

import numpy as np
import pytest
import torch

from oracle import mx

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
COLS = 328  # ten blocks and a part of one


@pytest.fixture(scope="module")
def tlg():
    import tiled_dense_gemm_tlg_b200 as t
    return t


def rows_of(typ):
    """Finite rows, 0 and 5, around two with a NaN, one with infinities, and one that is so by its sum alone."""
    X = torch.randn((6, COLS), generator=torch.Generator().manual_seed(1)).to(TYPES[typ])
    R = torch.randn((6, COLS), generator=torch.Generator().manual_seed(2)).to(TYPES[typ])
    X[1, 70] = float("nan")
    X[2, 33], R[2, 300] = float("inf"), float("-inf")
    X[3, 5], R[3, 5] = float("inf"), float("-inf")  # a NaN in H
    if typ != "f16":
        X[4] = 3e19  # finite, its square is not
    return X, R


@pytest.mark.parametrize("typ", list(TYPES))
def test_values(tlg, typ):
    X, R = rows_of(typ)
    w = torch.ones(COLS, dtype=TYPES[typ])
    Y, H, rstd = (t.cpu() for t in tlg.tlg_rmsnorm_forward(X.cuda(), w.cuda(), residual=R.cuda()))
    assert torch.isnan(Y[[1, 3]]).all() and torch.isnan(rstd[[1, 3]]).all()
    there = torch.isinf(H[2])
    assert there.nonzero().flatten().tolist() == [33, 300] and rstd[2] == 0
    assert torch.isnan(Y[2, there]).all() and (Y[2, ~there] == 0).all()
    if typ != "f16":
        assert rstd[4] == 0 and (Y[4] == 0).all()
    assert torch.isfinite(Y[[0, 5]]).all() and (rstd[[0, 5]] > 0).all()


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("typ", list(TYPES))
def test_every_block(tlg, typ, fmt):
    X, R = rows_of(typ)
    w = torch.ones(COLS, dtype=TYPES[typ])
    Q, S, _, rstd = tlg.tlg_rmsnorm_forward_mx(X.cuda(), w.cuda(), residual=R.cuda(), format=fmt)
    back = tlg.tlg_mx_dequantize(Q, S, COLS, format=fmt, out="f32").cpu()
    scales = S.cpu().numpy()[mx.scale_index(6, 12)]  # to a multiple of four blocks
    assert torch.isnan(back[[1, 3]]).all() and (scales[[1, 3], :11] == 255).all()
    broken = np.zeros(11, dtype=bool)
    broken[[33 // 32, 300 // 32]] = True
    assert (scales[2, :11][broken] == 255).all() and (scales[2, :11][~broken] == 0).all()
    columns = torch.from_numpy(np.repeat(broken, 32)[:COLS])
    assert torch.isnan(back[2, columns]).all() and (back[2, ~columns] == 0).all()
    if typ != "f16":
        assert (back[4] == 0).all() and rstd[4] == 0
    assert torch.isfinite(back[[0, 5]]).all() and (scales[:, 11] == 0).all()
