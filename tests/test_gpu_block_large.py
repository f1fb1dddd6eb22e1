"""The operators around the linear layers where element offsets pass 32 bits: rows far apart in buffers of
several GB.  References in 64 bits, tolerances as in the operators' own tests."""

import pytest
import torch

from test_gpu_gemv_q4 import check as check_q4
from test_gpu_gemv_q4 import make
from test_gpu_grouped import backward as grouped_backward
from test_gpu_grouped import check, forward, offsets_of, operands
from test_gpu_norm import backward as norm_backward
from test_gpu_norm import check as check_norm
from test_gpu_norm import f32_error, near, rows_of
from test_gpu_norm import forward as norm_forward

pytestmark = pytest.mark.gpu

FAR = 2 ** 31 + 2 ** 20  # elements between the first and the last row, at least


@pytest.fixture(scope="module")
def tlg():
    import tiled_dense_gemm_tlg_b200 as t
    yield t
    torch.cuda.empty_cache()


def spread(host, odd=0):
    """The rows (or matrices) of `host` so far apart that the last begins past 2^31 elements."""
    rows, cols = host.shape[0], host[0].numel()
    ld = (FAR // (rows - 1) + 63) // 64 * 64 + odd
    buf = torch.empty((rows - 1) * ld + cols + 64, dtype=host.dtype, device="cuda")
    view = torch.as_strided(buf, (rows, *host.shape[1:]), (ld, *host.stride()[1:]))
    view.copy_(host)
    return view


@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("op_b", ["N", "T"])
def test_grouped(tlg, op_b, odd):
    """Far rows of A and C, far matrices of B; odd strides take the plain loads."""
    sizes = [3, 60, 137]
    A, B = operands(1, 200, 72, 136, 3, op_b, torch.float16)
    want, err = forward(A, B, sizes, 0, op_b, "none")
    a, b, c = spread(A, odd), spread(B, odd), spread(torch.zeros((200, 136), dtype=torch.float16), odd)
    tlg.tlg_gemm_grouped(a, b, offsets_of(sizes).cuda(), op_b=op_b, C=c)
    check(c.contiguous(), want, err, torch.float16)
    del b
    want, err = grouped_backward(A, c.cpu(), sizes, 0, op_b)
    db = spread(torch.zeros(want.shape, dtype=torch.float16))
    tlg.tlg_gemm_grouped_dw(a, c, offsets_of(sizes).cuda(), op_b=op_b, dB=db)
    check(db.contiguous(), want, err, torch.float16)


@pytest.mark.parametrize("odd", [0, 1, 2])
def test_norm(tlg, odd):
    X, R = rows_of(1, 300, 264, torch.bfloat16), rows_of(2, 300, 264, torch.bfloat16)
    w = torch.ones(264, dtype=torch.bfloat16)
    h, rstd, y = norm_forward(X, R, w, 1e-6)
    x = spread(X, odd)
    Y = spread(torch.zeros_like(X), odd)
    _, H, s = tlg.tlg_rmsnorm_forward(x, w.cuda(), residual=R.cuda(), Y=Y)
    near(Y.contiguous(), y, f32_error(264), torch.bfloat16)
    near(s, rstd, f32_error(264), torch.float32)
    want, err, dw, dw_err = norm_backward(R, X, w, s.cpu(), None)
    dX, dweight = tlg.tlg_rmsnorm_backward(R.cuda(), x, w.cuda(), s, dX=Y)
    check_norm(dX.contiguous(), want, err, torch.bfloat16)
    check_norm(dweight, dw, dw_err, torch.float32)


def test_gemv_q4(tlg):
    """Far rows of weights (bytes), of X and of C."""
    X, Q, S, Z = make(1, 3, 300, 200, 64, True, torch.float16)
    q, x, c = spread(Q, 0), spread(X), spread(torch.zeros((3, 300), dtype=torch.float16))
    tlg.tlg_gemv_q4(x, q, S.cuda(), Z.cuda(), group=64, C=c)
    check_q4(c.contiguous(), X, Q, S, Z, 64, torch.float16)


def test_many_rows(tlg):
    """More rows than a grid dimension other than x holds, most of them in one group."""
    rows = 70000
    A, B = operands(3, rows, 64, 64, 3, "N", torch.bfloat16)
    sizes = [66000, 0, 4000]
    want, err = forward(A, B, sizes, 0, "N", "none")
    check(tlg.tlg_gemm_grouped(A.cuda(), B.cuda(), offsets_of(sizes).cuda()), want, err, torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    h, rstd, y = norm_forward(A, None, w, 1e-6)
    Y, _, s = tlg.tlg_rmsnorm_forward(A.cuda(), w.cuda())
    near(Y, y, f32_error(64), torch.bfloat16)
    want, err, dw, dw_err = norm_backward(A, A, w, s.cpu(), None)
    dX, dweight = tlg.tlg_rmsnorm_backward(A.cuda(), A.cuda(), w.cuda(), s)
    check_norm(dX, want, err, torch.bfloat16)
    check_norm(dweight, dw, dw_err, torch.float32)
    X, Q, S, _ = make(4, 1, 70000, 64, 32, False, torch.float16)
    check_q4(tlg.tlg_gemv_q4(X.cuda(), Q.cuda(), S.cuda(), group=32), X, Q, S, None, 32, torch.float16)
