"""GPU tests of the products with integer 4-bit weights against the formula in 64 bits.

Tolerances: products of q - z (4 bits and a sign) with a 16-bit X are exact in fp32; sums of K terms, the
groups' scales and the warps' sums in fp32 are off by at most (K + 16) 2^-23 times the sum of the terms'
magnitudes; the stored type adds half a unit, the activation its stated error."""

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def tlg():
    import tiled_dense_gemm_tlg_b200 as t
    return t


def make(seed, m, n, k, group, zero_points, dtype):
    g = torch.Generator().manual_seed(seed)
    groups = -(-k // group)
    X = torch.randn((m, k), generator=g).to(dtype)
    Q = torch.randint(0, 256, (n, -(-k // 32) * 16), generator=g, dtype=torch.uint8)
    S = ((torch.rand((n, groups), generator=g) + 0.5) * torch.exp2(torch.randint(-6, 1, (n, groups), generator=g).float())).to(dtype)
    Z = torch.randint(0, 16, (n, groups), generator=g, dtype=torch.uint8) if zero_points else None
    return X, Q, S, Z


def weights(Q, S, Z, k, group):
    c = torch.arange(k)
    q = (Q[:, c // 2].int() >> (4 * (c % 2)).int()) & 15
    z = 8 if Z is None else Z.int()[:, c // group]
    return (q - z).double() * S.double()[:, c // group]


def check(got, X, Q, S, Z, group, dtype, bias=None, act=None, residual=None):
    X = X.double()
    k = X.shape[1]
    W = weights(Q, S, Z, k, group)
    want = X @ W.t()
    err = (k + 16) * 2.0 ** -23 * (X.abs() @ W.abs().t())
    if bias is not None:
        want = want + bias.double()
        err = err + 2.0 ** -24 * want.abs()
    if act is not None:
        want = act(want)
        err = err * 1.13 + 2.0 ** -18 * (1 + want.abs()) + (0.15 * 2.0 ** -10 * want.abs() if dtype != torch.float32 else 0)
    if residual is not None:
        want = want + residual.double()
        err = err + 2.0 ** -24 * want.abs()
    fi = torch.finfo(dtype)
    bad = (got.double().cpu() - want).abs() > err + want.abs() * fi.eps / 2 + fi.tiny * fi.eps
    assert got.shape == want.shape and torch.isfinite(got).all() and not bad.any(), (bad.nonzero()[:4], got.cpu()[bad][:4], want[bad][:4])


def cuda(*t):
    return [x if x is None else x.cuda() for x in t]


@pytest.mark.parametrize("typ,out", [("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("group", [32, 64, 128, 512])
@pytest.mark.parametrize("zero_points", [False, True])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 16, 128), (1, 100, 1000), (2, 17, 333), (3, 4100, 264), (8, 33, 2048),
                                   (9, 70, 700), (16, 130, 96), (33, 50, 520)])
def test_product(tlg, m, n, k, zero_points, group, typ, out):
    X, Q, S, Z = make(1, m, n, k, group, zero_points, TYPES[typ])
    x, q, s, z = cuda(X, Q, S, Z)
    check(tlg.tlg_gemv_q4(x, q, s, z, group=group, out=out), X, Q, S, Z, group, TYPES[out])


@pytest.mark.parametrize("m,n", [(1, 5000), (4, 5000), (8, 9999), (12, 9999), (16, 9700)])
def test_wide_weights(tlg, m, n):
    """Rows of weights enough for the larger tiles."""
    X, Q, S, Z = make(2, m, n, 400, 64, True, torch.bfloat16)
    x, q, s, z = cuda(X, Q, S, Z)
    check(tlg.tlg_gemv_q4(x, q, s, z, group=64), X, Q, S, Z, 64, torch.bfloat16)


@pytest.mark.parametrize("k,group", [(4096 + 40, 32), (9000, 32), (17000, 128), (33000, 256)])
@pytest.mark.parametrize("m", [1, 9])
def test_long_rows(tlg, m, k, group):
    """More groups than have their scales in shared memory at a time."""
    X, Q, S, Z = make(3, m, 40, k, group, True, torch.float16)
    x, q, s, z = cuda(X, Q, S, Z)
    check(tlg.tlg_gemv_q4(x, q, s, z, group=group, out="f32"), X, Q, S, Z, group, torch.float32)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu", "gelu_tanh"])
@pytest.mark.parametrize("typ,out", [("f16", "f16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("m", [1, 10])
def test_epilogue(tlg, m, typ, out, act):
    fn = {"none": None, "relu": lambda v: v.clamp(min=0), "gelu": lambda v: v * torch.special.ndtr(v),
          "silu": lambda v: v * torch.sigmoid(v),
          "gelu_tanh": lambda v: v * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (v + 0.044715 * v ** 3))}[act]
    X, Q, S, Z = make(4, m, 200, 256, 128, False, TYPES[typ])
    S = (S.float() / 16).to(TYPES[typ])
    g = torch.Generator().manual_seed(5)
    bias, res = torch.randn(200, generator=g).to(TYPES[typ]), torch.randn((m, 200), generator=g).to(TYPES[out])
    x, q, s, b, r = cuda(X, Q, S, bias, res)
    got = tlg.tlg_gemv_q4(x, q, s, bias=b, activation=act, residual=r, out=out)
    check(got, X, Q, S, None, 128, TYPES[out], bias, fn, res)
    tlg.tlg_gemv_q4(x, q, s, bias=b, activation=act, residual=r, C=r, out=out)  # in the residual's place
    assert torch.equal(r, got)


@pytest.mark.parametrize("lead,extra", [(0, 0), (1, 3), (2, 2), (8, 8)])
@pytest.mark.parametrize("m,n,k", [(1, 20, 333), (5, 33, 1000), (18, 40, 77)])
def test_strides(tlg, m, n, k, lead, extra):
    """X, C and Q inside larger buffers; elements past K hold anything."""
    X, Q, S, Z = make(6, m, n, k, 32, True, torch.float16)
    xb = torch.full((lead + m * (k + extra) + 8,), float("nan"), dtype=torch.float16, device="cuda")
    x = xb[lead:lead + m * (k + extra)].view(m, k + extra)[:, :k]
    x.copy_(X)
    qb = torch.full((n, Q.shape[1] + 32), 255, dtype=torch.uint8, device="cuda")
    q = qb[:, :Q.shape[1]]
    q.copy_(Q)
    cb = torch.full((lead + m * (n + extra) + 8,), -77.0, dtype=torch.float16, device="cuda")
    c = cb[lead:lead + m * (n + extra)].view(m, n + extra)[:, :n]
    s, z = cuda(S, Z)
    tlg.tlg_gemv_q4(x, q, s, z, group=32, C=c)
    check(c, X, Q, S, Z, 32, torch.float16)
    left = cb.clone()
    left[lead:lead + m * (n + extra)].view(m, n + extra)[:, :n] = -77
    assert (left == -77).all()


def test_empty(tlg):
    X, Q, S, _ = make(7, 3, 16, 64, 32, False, torch.float16)
    bias = torch.arange(16).half()
    x, q, s, b = cuda(X, Q, S, bias)
    got = tlg.tlg_gemv_q4(x[:, :0], q[:, :0], s[:, :0], group=32, bias=b)
    assert torch.equal(got.cpu(), bias.expand(3, -1))
    assert tlg.tlg_gemv_q4(x[:0], q, s, group=32).shape == (0, 16)
    assert tlg.tlg_gemv_q4(x, q[:0], s[:0], group=32).shape == (3, 0)


def test_nan_and_infinity_stay_in_their_row(tlg):
    X, Q, S, _ = make(8, 4, 48, 256, 64, False, torch.bfloat16)
    X[1, 7], X[2, 200] = float("nan"), float("inf")
    S[5, 1] = float("nan")
    x, q, s = cuda(X, Q, S)
    got = tlg.tlg_gemv_q4(x, q, s, group=64)
    assert torch.isnan(got[1]).all() and not torch.isfinite(got[2]).any() and torch.isnan(got[:, 5]).all()
    keep = [n for n in range(48) if n != 5]
    fine = got[[0, 3]][:, keep]
    check(fine, X[[0, 3]], Q[keep], S[keep], None, 64, torch.bfloat16)


def test_streams_and_graphs(tlg):
    X, Q, S, Z = make(9, 2, 3000, 512, 128, True, torch.float16)
    x, q, s, z = cuda(X, Q, S, Z)
    C = torch.empty((2, 3000), dtype=torch.float16, device="cuda")
    tlg.tlg_gemv_q4(x, q, s, z, C=C)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tlg.tlg_gemv_q4(x, q, s, z, C=C)
    x.mul_(2)
    graph.replay()
    check(C, X * 2, Q, S, Z, 128, torch.float16)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [tlg.tlg_gemv_q4(x, q, s, z, stream=t) for _ in range(5) for t in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, C) for o in outs)
