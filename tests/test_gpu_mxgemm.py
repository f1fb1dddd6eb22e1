"""GPU tests of tlg_gemm_mxfp4, the product of 4-bit MX matrices, against fp64 numpy on the
decoded operands.

Two kinds of inputs.  "exact": scales within four binades, so every product is a multiple of
2^-4 and every sum below 2^20 (K <= 2000): each partial sum is an fp32 number, and the fp32
result must equal the fp64 one.  "wide": scales over 31 binades; an fp32 sum of K products
whose every step rounds or truncates by at most one unit of a partial sum no larger than
sum |a b| is within K 2^-23 sum |a b|.  On top come one rounding of the stored type
(eps / 2 relative) and the epilogue's stated errors."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import mx

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TILES = [(1, 64), (1, 128), (2, 192), (2, 256)]
SHAPES = [(1, 1, 1), (1, 8, 32), (3, 65, 33), (128, 64, 256), (129, 129, 257), (200, 333, 1000), (257, 400, 2000),
          (512, 768, 512), (5, 1000, 700), (300, 17, 96)]


@pytest.fixture(scope="module")
def tlg():
    import tiled_dense_gemm_tlg_b200 as t
    yield t
    rc, code = t.tlg_device_error()
    assert rc == 0, hex(code)


def operand(rows, K, kind, seed):
    """(Q, S, fp64 values): random codes, padding codes 0, padding rows' scales 0xFF (never used)."""
    g = np.random.default_rng(seed)
    blocks = -(-K // 32)
    codes = g.integers(0, 16, (rows, blocks * 32)).astype(np.uint8)
    codes[:, K:] = 0
    lo, hi = (126, 129) if kind == "exact" else (112, 143)
    scale = g.integers(lo, hi, (rows, blocks)).astype(np.uint8)
    Q = torch.from_numpy(mx.pack(codes, "e2m1")).cuda()
    S = torch.from_numpy(mx.tile_scales(scale, fill=255)).cuda()
    return Q, S, mx.decode(codes, scale, "e2m1")[:, :K]


class Out:
    """A C (or residual) inside a guarded buffer, `lead` elements in, rows `ld` apart."""

    def __init__(self, rows, cols, dtype, lead=0, extra=0, host=None):
        self.ld = cols + extra
        self.buf = torch.full((lead + rows * self.ld + 128,), float("nan"), dtype=dtype, device="cuda")
        self.view = self.buf[lead:lead + rows * self.ld].view(rows, self.ld)[:, :cols]
        mask = torch.ones_like(self.buf, dtype=torch.bool)
        mask[lead:lead + rows * self.ld].view(rows, self.ld)[:, :cols] = False
        self.mask = mask
        if host is not None:
            self.view.copy_(host)

    def guards_kept(self):
        return bool(torch.isnan(self.buf[self.mask]).all())


def accumulation_bound(a, b, kind):
    return 0.0 if kind == "exact" else a.shape[1] * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)


def check(C, want, err, typ):
    """want: fp64 before the last rounding; err: bound of the error before it."""
    info = torch.finfo(TYPES[typ])
    tiny = 2.0 ** -25 if typ == "f16" else 0.0
    got = C.double().cpu().numpy()
    if typ == "f16":
        want, got = np.clip(want, -1e6, 1e6), np.clip(got, -1e6, 1e6)
        fits = np.abs(want) + err < 65504
        assert np.isfinite(got[fits]).all()
        want, got, err = want[fits], got[fits], (err[fits] if np.ndim(err) else err)
    half = 0.0 if typ == "f32" and np.ndim(err) == 0 else info.eps / 2
    bound = err + half * (np.abs(want) + err) + tiny
    worst = np.abs(got - want) - bound
    assert (worst <= 0).all(), (worst.max(), np.unravel_index(worst.argmax(), worst.shape))


@pytest.mark.parametrize("cg,bn", TILES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_is_exact(tlg, cg, bn, M, N, K):
    A, SA, a = operand(M, K, "exact", M + N)
    B, SB, b = operand(N, K, "exact", K + 1)
    for typ, lead, extra in (("f32", 0, 0), ("f32", 1, 3), ("f16", 8, 8), ("bf16", 1, 1)):
        o = Out(M, N, TYPES[typ], lead, extra)
        tlg.tlg_gemm_mxfp4(A, SA, B, SB, C=o.view, out=typ, config={"cta_group": cg, "block_n": bn})
        check(o.view, a @ b.T, 0.0, typ)
        assert o.guards_kept()


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 31, 32])
@pytest.mark.parametrize("N,K", [(1, 32), (100, 257), (128, 1024), (300, 2000), (1111, 555)])
def test_few_rows_are_exact(tlg, M, N, K):
    A, SA, a = operand(M, K, "exact", M + N)
    B, SB, b = operand(N, K, "exact", K + 1)
    num_kb = -(-K // 256)
    for ks in (0, 1, 2, 4, 8):
        if ks > num_kb:
            with pytest.raises(tlg.TlgError):
                tlg.tlg_gemm_mxfp4(A, SA, B, SB, config={"k_split": ks})
            continue
        for typ, lead, extra in (("f32", 1, 3), ("f16", 0, 0), ("bf16", 1, 1)):
            o = Out(M, N, TYPES[typ], lead, extra)
            tlg.tlg_gemm_mxfp4(A, SA, B, SB, C=o.view, out=typ, config={"k_split": ks})
            check(o.view, a @ b.T, 0.0, typ)
            assert o.guards_kept()


@pytest.mark.parametrize("M", [1, 5, 16, 32])
@pytest.mark.parametrize("typ", list(TYPES))
def test_few_rows_epilogue_is_the_tiles(tlg, M, typ):
    """Few rows run a kernel of their own; with exact sums its results are those of the tiles, to the bit."""
    N, K = 700, 1024
    A, SA, _ = operand(M, K, "exact", M)
    B, SB, _ = operand(N, K, "exact", 9)
    SB = (SB.int() - 6).clamp(min=0).to(torch.uint8)
    bias = torch.randn(N, device="cuda").to(torch.bfloat16 if typ == "bf16" else torch.float16)
    R = torch.randn(M, N, device="cuda").to(TYPES[typ])
    for act in ("none", "relu", "gelu", "silu", "gelu_tanh"):
        want = tlg.tlg_gemm_mxfp4(A, SA, B, SB, bias=bias, activation=act, residual=R, out=typ,
                                  config={"cta_group": 1, "block_n": 64})
        got = tlg.tlg_gemm_mxfp4(A, SA, B, SB, bias=bias, activation=act, residual=R, out=typ)
        assert tlg.tlg_choose_config_mxfp4(M, N, K, typ)["block_n"] in (16, 32)
        assert torch.equal(got, want), act
        C = R.clone()
        tlg.tlg_gemm_mxfp4(A, SA, B, SB, bias=bias, activation=act, residual=C, C=C, out=typ)
        assert torch.equal(C, want), act


@pytest.mark.parametrize("M,N,K", SHAPES + [(2, 4096, 4096), (16, 2048, 8192), (40, 777, 3001)])
def test_product_automatic_tile_wide_scales(tlg, M, N, K):
    A, SA, a = operand(M, K, "wide", M + 3 * N)
    B, SB, b = operand(N, K, "wide", K + 7)
    for typ in TYPES:
        o = Out(M, N, TYPES[typ], 8, 8)
        tlg.tlg_gemm_mxfp4(A, SA, B, SB, C=o.view, out=typ)
        check(o.view, a @ b.T, accumulation_bound(a, b, "wide"), typ)
        assert o.guards_kept()


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu", "gelu_tanh"])
@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("cg,bn", TILES + [(0, 0)])
def test_fused_epilogue(tlg, act, typ, cg, bn):
    for M, N, K in ((7, 200, 96), (300, 333, 256)):
        A, SA, a = operand(M, K, "exact", M)
        B, SB, b = operand(N, K, "exact", N)
        SA = (SA.int() - 2).clamp(min=0).to(torch.uint8)  # values small enough for the activation to matter
        SB = (SB.int() - 2).clamp(min=0).to(torch.uint8)
        g = np.random.default_rng(M)
        bdt = torch.bfloat16 if typ == "bf16" else torch.float16
        bias = torch.from_numpy(g.standard_normal(N)).to(bdt).cuda()
        R = torch.from_numpy(g.standard_normal((M, N))).to(TYPES[typ]).cuda()
        z = a @ b.T / 16
        for use_bias, use_r, inplace, lead, extra in ((1, 1, 0, 8, 8), (1, 0, 0, 1, 1), (0, 1, 1, 0, 0), (0, 0, 0, 0, 0),
                                                      (1, 1, 1, 1, 3)):
            x = z + (bias.double().cpu().numpy() if use_bias else 0)
            want = mx.activate(act, x)
            fn = {"gelu": 3e-7 if typ == "f32" else 0.15 * np.maximum(np.abs(want) * 2.0 ** -10, 2.0 ** -24),
                  "silu": 2e-6 * (1 + np.abs(x)), "gelu_tanh": 2e-6 * (1 + np.abs(x))}.get(act, 0.0)
            # the bias and residual additions: one fp32 rounding each; the activations' slope is below 1.13
            fn = fn + 2.0 ** -24 * (1.2 * np.abs(x) + np.abs(want) + 6)
            if use_r:
                want = want + R.double().cpu().numpy()
            o = Out(M, N, TYPES[typ], lead, extra, R if inplace else None)
            res = (o.view if inplace else R) if use_r else None
            tlg.tlg_gemm_mxfp4(A, SA, B, SB, bias=bias if use_bias else None, activation=act, residual=res, C=o.view,
                               out=typ, config={"cta_group": cg, "block_n": bn} if cg else None)
            check(o.view, want, fn, typ)
            assert o.guards_kept()


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("cg,bn", TILES)
@pytest.mark.parametrize("N,lead,extra", [(330, 0, 0), (330, 2, 0), (330, 1, 1), (336, 0, 0), (331, 0, 5), (335, 8, 1),
                                          (47, 2, 3)])
def test_residuals_of_any_alignment(tlg, typ, cg, bn, N, lead, extra):
    """Base and rows aligned to 16, 4 or 2 bytes, and ends inside 16 and 4 bytes; C has another layout,
    and then the residual's.  Inputs are small multiples of 1/64, so the only rounding is the last."""
    M, K = 270, 96
    A, SA, a = operand(M, K, "exact", N)
    B, SB, b = operand(N, K, "exact", lead + 1)
    R = torch.from_numpy(np.random.default_rng(extra).integers(-64, 65, (M, N)) / 64).to(TYPES[typ])
    r = Out(M, N, TYPES[typ], lead, extra, R)
    want = a @ b.T + R.double().numpy()
    for o in (Out(M, N, TYPES[typ], 8, 8), r):
        tlg.tlg_gemm_mxfp4(A, SA, B, SB, residual=r.view, C=o.view, out=typ, config={"cta_group": cg, "block_n": bn})
        check(o.view, want, 0.0, typ)
        assert o.guards_kept()


def test_nan_scale_reaches_its_row_and_column_only(tlg):
    M, N, K = 150, 210, 300
    for cg, bn in TILES + [(0, 0)]:
        A, SA, a = operand(M, K, "exact", 1)
        B, SB, b = operand(N, K, "exact", 2)
        SA[int(mx.scale_index(M, 12)[140, 9])] = 255
        SB[int(mx.scale_index(N, 12)[7, 0])] = 255
        C = tlg.tlg_gemm_mxfp4(A, SA, B, SB, out="f32", config={"cta_group": cg, "block_n": bn} if cg else None)
        C = C.cpu().numpy()
        want = a @ b.T
        want[140, :] = np.nan
        want[:, 7] = np.nan
        assert np.array_equal(C, want, equal_nan=True)


def test_empty_k_and_empty_output(tlg):
    lib = tlg.raw_library()
    bias = torch.randn(70, device="cuda").half()
    R = torch.randn(5, 70, device="cuda").half()
    C = torch.empty(5, 70, dtype=torch.float16, device="cuda")
    epi = tlg.tlg_fused_epilogue(bias.data_ptr(), 1, R.data_ptr(), 70)
    st = torch.cuda.current_stream().cuda_stream
    assert lib.tlg_gemm_mxfp4(5, 70, 0, None, 0, None, None, 0, None, ctypes.byref(epi), C.data_ptr(), 70, 1, None,
                              st) == 0
    assert torch.equal(C, (bias.float().clamp(min=0) + R.float()).half())
    empty = [torch.empty((n, 0), dtype=torch.uint8, device="cuda") for n in (5, 70)]
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    for typ, b in (("f16", bias), ("f32", bias), ("bf16", bias.bfloat16())):
        got = tlg.tlg_gemm_mxfp4(empty[0], none, empty[1], none, bias=b, activation="relu", out=typ)
        assert torch.equal(got, b.float().clamp(min=0).to(TYPES[typ]).expand(5, 70))
    A, SA, _ = operand(4, 64, "exact", 0)
    assert tlg.tlg_gemm_mxfp4(A[:0], SA, A, SA).shape == (0, 4)


def test_strided_operands(tlg):
    M, N, K = 70, 90, 500
    A, SA, a = operand(M, K, "exact", 5)
    B, SB, b = operand(N, K, "exact", 6)
    bigA = torch.full((M, A.shape[1] + 48), 0x77, dtype=torch.uint8, device="cuda")
    bigB = torch.full((N, B.shape[1] + 16), 0x77, dtype=torch.uint8, device="cuda")
    bigA[:, :A.shape[1]] = A
    bigB[:, :B.shape[1]] = B
    C = tlg.tlg_gemm_mxfp4(bigA[:, :A.shape[1]], SA, bigB[:, :B.shape[1]], SB, out="f32")
    assert np.array_equal(C.cpu().numpy(), a @ b.T)


def test_a_layer_forward_and_backward_in_four_bits(tlg):
    """The operators as a training step uses them: quantise, product with bias, activation with an
    8-bit checkpoint, its backward pass, and both backward products on transposed quantisations.
    Each step is compared with fp64 on the values the step was given."""
    tok, d_in, d_out = 200, 320, 480
    g = torch.Generator().manual_seed(0)
    X = torch.randn((tok, d_in), generator=g).half().cuda()
    W = (torch.randn((d_out, d_in), generator=g) / 18).half().cuda()
    bias = torch.randn((d_out,), generator=g).half().cuda()
    dY = torch.randn((tok, d_out), generator=g).half().cuda()

    def val(Q, S, cols, fmt="e2m1"):
        return tlg.tlg_mx_dequantize(Q, S, cols, format=fmt, out="f32").double().cpu().numpy()

    X4, W4 = tlg.tlg_mx_quantize(X), tlg.tlg_mx_quantize(W)
    x, w = val(*X4, d_in), val(*W4, d_in)
    Z = tlg.tlg_gemm_mxfp4(*X4, *W4, bias=bias)
    check(Z, x @ w.T + bias.double().cpu().numpy(), accumulation_bound(x, w, "wide") + 2.0 ** -22, "f16")
    Y, Q, S = tlg.tlg_act_forward_mx(Z, "gelu")
    dZ, db = tlg.tlg_act_backward_mx(dY, Q, S, "gelu")
    d = dY.double().cpu().numpy()
    want = d * mx.slope("gelu", val(Q, S, d_out, "e4m3"))
    check(dZ, want, 2e-6 * np.abs(d), "f16")
    assert np.abs(db.double().cpu().numpy() - want.sum(axis=0)).max() < 2e-6 * np.abs(d).sum(axis=0).max()
    dZ4 = tlg.tlg_mx_quantize(dZ)
    Wt4 = tlg.tlg_mx_quantize(W, op="T")  # d_in x d_out
    dX = tlg.tlg_gemm_mxfp4(*dZ4, *Wt4)
    p, q = val(*dZ4, d_out), val(*Wt4, d_out)
    check(dX, p @ q.T, accumulation_bound(p, q, "wide"), "f16")
    dZt4, Xt4 = tlg.tlg_mx_quantize(dZ, op="T"), tlg.tlg_mx_quantize(X, op="T")
    dW = tlg.tlg_gemm_mxfp4(*dZt4, *Xt4, out="f32")
    p, q = val(*dZt4, tok), val(*Xt4, tok)
    check(dW, p @ q.T, accumulation_bound(p, q, "wide"), "f32")
    # 4 bits and 8 bits, against the layer in fp64: the quantised products stay near it
    exact_dw = (d * mx.slope("gelu", Z.double().cpu().numpy())).T @ X.double().cpu().numpy()
    rel = np.linalg.norm(dW.double().cpu().numpy() - exact_dw) / np.linalg.norm(exact_dw)
    assert rel < 0.25  # two E2M1 operands, each element off by at most 1/4 of itself or 1/8 of its block's top


def test_single_rows_of_any_stride(tlg):
    A, SA, a = operand(1, 500, "exact", 3)
    B, SB, b = operand(1, 500, "exact", 4)
    wide = [torch.zeros((1, 400), dtype=torch.uint8, device="cuda") for _ in range(2)]
    wide[0][:, :256], wide[1][:, :256] = A, B
    views = [w[:, :256].as_strided((1, 256), (7, 1)) for w in wide]
    for cfg in (None, {"cta_group": 1, "block_n": 64}):
        C = tlg.tlg_gemm_mxfp4(views[0], SA, views[1], SB, out="f32", config=cfg)
        assert np.array_equal(C.cpu().numpy(), a @ b.T)


@pytest.mark.parametrize("M,N,K", [(20, 300, 1500), (700, 500, 1024)])
def test_two_calls_at_once(tlg, M, N, K):
    A, SA, a = operand(M, K, "exact", 1)
    B, SB, b = operand(N, K, "exact", 2)
    want = torch.from_numpy(a @ b.T).cuda()
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(tlg.tlg_gemm_mxfp4(A, SA, B, SB, out="f32"))
    torch.cuda.synchronize()
    assert all(torch.equal(c.double(), want) for c in got)


def test_streams_and_graphs(tlg):
    A, SA, a = operand(100, 512, "exact", 1)
    B, SB, b = operand(300, 512, "exact", 2)
    want = a @ b.T
    C = tlg.tlg_gemm_mxfp4(A, SA, B, SB, out="f32")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        C2 = tlg.tlg_gemm_mxfp4(A, SA, B, SB, out="f32")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        C3 = tlg.tlg_gemm_mxfp4(A, SA, B, SB, out="f32")
    C3.zero_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for x in (C, C2, C3):
        assert np.array_equal(x.cpu().numpy(), want)


def test_configurations(tlg):
    M, N, K = 1000, 900, 300
    A, SA, a = operand(M, K, "exact", 1)
    B, SB, b = operand(N, K, "exact", 2)
    for req in ({"max_ctas": 3}, {"raster_group": 1}, {"raster_group": 64, "cta_group": 2}):
        got = tlg.tlg_choose_config_mxfp4(M, N, K, request=req)
        assert all(got[k] == v for k, v in req.items() if k != "max_ctas")
        assert np.array_equal(tlg.tlg_gemm_mxfp4(A, SA, B, SB, out="f32", config=req).cpu().numpy(), a @ b.T)
    for req in ({"block_n": 96}, {"split_k": 2}, {"cta_group": 3}, {"raster_group": 65}, {"overlap_prev": 2}):
        with pytest.raises(tlg.TlgError):
            tlg.tlg_gemm_mxfp4(A, SA, B, SB, config=req)
