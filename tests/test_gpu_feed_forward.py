"""The operators as a feed-forward block runs them: norm, experts' products, an activation with its input
saved in 8 bits, and the whole way back; and the serving forms, with weights in 4 bits.

The references take each operator's input as the GPU left it, so that a step's tolerance is that operator's own
(derived in its own test); the gradients of the whole block are checked against differences of the block in 64 bits,
where the 8-bit checkpoint is left out of the comparison by an activation that does not read it."""

import pytest
import torch

from oracle import mx
from test_gpu_gemv_q4 import make, weights
from test_gpu_grouped import backward as grouped_backward
from test_gpu_grouped import check, forward, offsets_of
from test_gpu_norm import check as check_norm
from test_gpu_norm import backward as norm_backward

pytestmark = pytest.mark.gpu

SIZES = [100, 0, 37, 63]
ROWS, D, F = 200, 256, 384


@pytest.fixture(scope="module")
def tlg():
    import tiled_dense_gemm_tlg_b200 as t
    return t


def block(tlg, X, R, w, W1, W2, off, act):
    """The experts' feed-forward block in front of a residual stream: what training keeps, and the output."""
    Y, H, rstd = tlg.tlg_rmsnorm_forward(X, w, residual=R)
    Z = tlg.tlg_gemm_grouped(Y, W1, off, op_b="T")
    A, Q, S = tlg.tlg_act_forward_mx(Z, act)
    return tlg.tlg_gemm_grouped(A, W2, off, op_b="T"), (Y, H, rstd, Z, A, Q, S)


def block_backward(tlg, dO, dH, kept, w, W1, W2, off, act):
    Y, H, rstd, Z, A, Q, S = kept
    dA = tlg.tlg_gemm_grouped(dO, W2, off, op_b="N")
    dW2 = tlg.tlg_gemm_grouped_dw(A, dO, off, op_b="T", out="f32")
    dZ, _ = tlg.tlg_act_backward_mx(dA, Q, S, act, bias_grad=False)
    dY = tlg.tlg_gemm_grouped(dZ, W1, off, op_b="N")
    dW1 = tlg.tlg_gemm_grouped_dw(Y, dZ, off, op_b="T", out="f32")
    dX, dw = tlg.tlg_rmsnorm_backward(dY, H, w, rstd, dH=dH)
    return dX, dw, dW1, dW2, (dA, dZ, dY)


def tensors(dtype):
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g)
    return [t.to(dtype) for t in (r(ROWS, D), r(ROWS, D), 1 + 0.1 * r(D), r(4, F, D) / D ** 0.5, r(4, D, F) / F ** 0.5,
                                  r(ROWS, D), r(ROWS, D))]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_training_step(tlg, dtype):
    X, R, w, W1, W2, dO, dH = (t.cuda() for t in tensors(dtype))
    off = offsets_of(SIZES).cuda()
    out, kept = block(tlg, X, R, w, W1, W2, off, "silu")
    Y, H, rstd, Z, A, Q, S = (t.cpu() for t in kept)
    for got, a, b in ((Z, Y, W1), (out, A, W2)):
        want, err = forward(a, b.cpu(), SIZES, 0, "T", "none")
        check(got, want, err, dtype)
    dX, dw, dW1, dW2, mid = block_backward(tlg, dO, dH, kept, w, W1, W2, off, "silu")
    dA, dZ, dY = (t.cpu() for t in mid)
    want, err = forward(dO.cpu(), W2.cpu(), SIZES, 0, "N", "none")
    check(dA, want, err, dtype)
    z = torch.from_numpy(mx.decode(mx.unpack(Q.numpy(), "e4m3"), S.numpy()[mx.scale_index(ROWS, F // 32)], "e4m3")[:, :F])
    slope = torch.sigmoid(z) * (1 + z * torch.sigmoid(-z))
    check(dZ, dA.double() * slope, 2e-6 * dA.double().abs(), dtype)
    want, err = forward(dZ, W1.cpu(), SIZES, 0, "N", "none")
    check(dY, want, err, dtype)
    for got, a, d in ((dW2, A, dO.cpu()), (dW1, Y, dZ)):
        want, err = grouped_backward(a, d, SIZES, 0, "T")
        check(got, want, err, torch.float32)
    want, err, dw_want, dw_err = norm_backward(dY, H, w.cpu(), rstd, dH.cpu())
    check_norm(dX, want, err, dtype)
    check_norm(dw, dw_want, dw_err, torch.float32)


def test_gradients_of_the_block_against_differences(tlg):
    """The whole way forward and back without an activation, whose 8-bit checkpoint then does not matter: the gradient
    along a direction against a central difference of the block in 64 bits.  The 16-bit steps between round to 2^-11
    each; a directional derivative sums thousands of such errors of either sign, and stays within 1 % of the
    sum's size by far."""
    X, R, w, W1, W2, dO, dH = (t.cuda() for t in tensors(torch.float16))
    off = offsets_of(SIZES).cuda()
    _, kept = block(tlg, X, R, w, W1, W2, off, "none")
    dX, dw, dW1, dW2, _ = block_backward(tlg, dO, dH, kept, w, W1, W2, off, "none")

    def value(X, w, W1, W2):
        h = X + R.double().cpu()
        y = h / torch.sqrt((h * h).mean(dim=1, keepdim=True) + 1e-6) * w
        total = (h * dH.double().cpu()).sum()
        r = 0
        for g, s in enumerate(SIZES):
            total = total + ((y[r:r + s] @ W1[g].t() @ W2[g].t()) * dO[r:r + s].double().cpu()).sum()
            r += s
        return total

    at = [t.double().cpu() for t in (X, w, W1, W2)]
    for i, grad in enumerate((dX, dw, dW1, dW2)):
        grad = grad.double().cpu()
        direction = grad / grad.norm()
        h = 1e-4
        up, down = ([t + s * h * direction if j == i else t for j, t in enumerate(at)] for s in (1, -1))
        slope = (value(*up) - value(*down)) / (2 * h)
        assert abs(slope - grad.norm()) < 0.01 * grad.norm(), i


def test_training_step_in_a_graph(tlg):
    X, R, w, W1, W2, dO, dH = (t.cuda() for t in tensors(torch.bfloat16))
    off = offsets_of(SIZES).cuda()
    step = lambda: block_backward(tlg, dO, dH, block(tlg, X, R, w, W1, W2, off, "gelu")[1], w, W1, W2, off, "gelu")[:4]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    off.copy_(offsets_of([20, 80, 0, 100]))
    X.mul_(0.75)
    graph.replay()
    want = step()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("tokens", [1, 3, 20])
def test_serving_with_4_bit_weights(tlg, tokens):
    """A decoding step: the norm into the integer 4-bit layers, the activation and the residual in their epilogues; and
    the norm's own 4-bit output into the microscaled product."""
    X, Q1, S1, Z1 = make(2, tokens, F, D, 64, True, torch.float16)
    _, Q2, S2, _ = make(3, tokens, D, F, 128, False, torch.float16)
    S1, S2 = S1 / 16, S2 / 16
    w = torch.ones(D, dtype=torch.float16)
    q1, s1, z1, q2, s2, x = (t.cuda() for t in (Q1, S1, Z1, Q2, S2, X))
    Y, H, _ = tlg.tlg_rmsnorm_forward(x, w.cuda(), residual=x)
    A = tlg.tlg_gemv_q4(Y, q1, s1, z1, group=64, activation="gelu_tanh")
    out = tlg.tlg_gemv_q4(A, q2, s2, group=128, residual=H)
    y, h, a = (t.double().cpu() for t in (Y, H, A))
    # fp32 sums as in the operator's own test, the activation's slope (at most 1.13) and stated error, the stored half unit
    W1, W2 = weights(Q1, S1, Z1, D, 64), weights(Q2, S2, None, F, 128)
    u = y @ W1.t()
    want = u * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (u + 0.044715 * u ** 3))
    err = 1.13 * (D + 16) * 2.0 ** -23 * (y.abs() @ W1.abs().t()) + 2.0 ** -18 * (1 + want.abs())
    assert ((a - want).abs() <= err + 2.0 ** -11 * want.abs()).all()
    want = a @ W2.t() + h
    err = (F + 16) * 2.0 ** -23 * (a.abs() @ W2.abs().t()) + 2.0 ** -24 * want.abs()
    assert ((out.double().cpu() - want).abs() <= err + 2.0 ** -11 * want.abs() + 2.0 ** -24).all()
    W = torch.randn((F, D), generator=torch.Generator().manual_seed(4)).half().cuda()
    Wq, Ws = tlg.tlg_mx_quantize(W)
    Yq, Ys, _, _ = tlg.tlg_rmsnorm_forward_mx(x, w.cuda(), residual=x, format="e2m1")
    C = tlg.tlg_gemm_mxfp4(Yq, Ys, Wq, Ws, out="f32").double()
    a, b = (tlg.tlg_mx_dequantize(q, s, D, out="f32").double() for q, s in ((Yq, Ys), (Wq, Ws)))
    assert ((C - a @ b.t()).abs() <= D * 2.0 ** -23 * (a.abs() @ b.abs().t())).all()
