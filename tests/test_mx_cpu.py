"""CPU-side checks of the microscaled (MX) operators: the reference against hand-worked
values, the C interface's refusals (made before any CUDA call) and the binding's."""

import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import mx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def tlg():
    import tiled_dense_gemm_tlg_b200 as t
    return t


# ------------------------------------------------------------------ the reference


def test_e2m1_worked_values():
    # amax 7: scale 2^(2 - 2) = 1; 7 saturates at 6; ties go to the even code
    x = np.zeros((1, 32))
    x[0, :12] = [7, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5.1, -0.2, 0.26, -0.0]
    codes, scale = mx.quantize(x, "e2m1")
    assert scale[0, 0] == 127
    assert mx.decode(codes, scale, "e2m1")[0, :12].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -6, 0, 0.5, 0]
    assert codes[0, 11] == 8  # the sign of a zero stays


def test_e4m3_worked_values():
    # 449 / 448 > 1: the scale steps to 2; 448 itself keeps 1
    for amax, byte in ((448.0, 127), (449.0, 128), (447.0, 127), (224.5, 127), (224.0, 126)):
        x = np.zeros((1, 32))
        x[0, 0] = amax
        assert mx.quantize(x, "e4m3")[1][0, 0] == byte, amax
    x[0, :5] = [448, 17, 18, 2.0 ** -10, 3 * 2.0 ** -10]  # 17 and 2^-10 tie (even below), 3 * 2^-10 ties up
    codes, scale = mx.quantize(x, "e4m3")
    assert mx.decode(codes, scale, "e4m3")[0, :5].tolist() == [448, 16, 18, 0, 2 * 2.0 ** -9]
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(mx.E4M3, t)


def test_scale_limits():
    x = np.zeros((4, 32))
    x[1, 3], x[2, 0], x[3, 31] = np.inf, np.nan, 2.0 ** -140
    for fmt in ("e2m1", "e4m3"):
        codes, scale = mx.quantize(x, fmt)
        assert scale[:, 0].tolist() == [0, 255, 255, 0]
        v = mx.decode(codes, scale, fmt)
        assert (v[0] == 0).all() and np.isnan(v[1:3]).all()


def test_scale_layout_is_a_permutation():
    for rows, cols in ((1, 1), (129, 200), (256, 512), (300, 33)):
        blocks = -(-cols // 32)
        idx = mx.scale_index(-(-rows // 128) * 128, -(-blocks // 4) * 4)
        assert np.array_equal(np.sort(idx.ravel()), np.arange(mx.scale_bytes(rows, cols)))
    assert mx.scale_index(128, 4)[33, 2] == 16 + 4 + 2


def test_slopes_match_differences():
    x = np.linspace(-6, 6, 2401)
    x = x[np.abs(x) > 1e-3]
    h = 1e-5
    for act in ("none", "relu", "gelu", "silu", "gelu_tanh"):
        d = (mx.activate(act, x + h) - mx.activate(act, x - h)) / (2 * h)
        assert np.abs(d - mx.slope(act, x)).max() < 1e-8, act


def test_gelu_slope_coefficients_are_the_fit():
    import importlib.util
    import re

    csrc = os.path.join(ROOT, "tiled_dense_gemm_tlg_b200", "csrc")
    spec = importlib.util.spec_from_file_location("fit_gelu_slope", os.path.join(csrc, "fit_gelu_slope.py"))
    fit = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(fit)
    src = open(os.path.join(csrc, "tlg_mx_device.cuh")).read()
    n, vals = re.search(r"gelu_slope_coef\(int k\).*?c\[(\d+)\] = \{([^}]*)\}", src, flags=re.S).groups()
    kernel = np.array([float(v.strip().rstrip("f")) for v in vals.split(",")], dtype=np.float32)
    assert int(n) == fit.DEGREE + 1 == kernel.size
    assert np.abs(kernel - fit.fit()).max() < 1e-6  # the fit itself, to what a linear solver repeats
    x = np.linspace(-12, 12, 960001).astype(np.float32)
    assert np.abs(fit.gelu_slope_f32(x, kernel) - fit.gelu_slope_exact(x)).max() < 2e-7


# ------------------------------------------------------------------ refusals of the C interface

A = 1 << 20  # fake, aligned addresses: the checks never dereference them


def test_mx_size(tlg):
    assert tlg.tlg_mx_size("e2m1", 1, 1) == (16, 512)
    assert tlg.tlg_mx_size("e4m3", 129, 129) == (160, 2 * 2 * 512)
    assert tlg.tlg_mx_size("e2m1", 0, 0) == (0, 0)
    lib = tlg.raw_library()
    q, s = ctypes.c_int64(5), ctypes.c_size_t(5)
    assert lib.tlg_mx_size(2, 1, 1, ctypes.byref(q), ctypes.byref(s)) == tlg.TLG_ERR_INVALID_ARG
    assert lib.tlg_mx_size(0, -1, 1, ctypes.byref(q), ctypes.byref(s)) == tlg.TLG_ERR_INVALID_ARG
    assert lib.tlg_mx_size(0, 2 ** 31, 1, ctypes.byref(q), ctypes.byref(s)) == tlg.TLG_ERR_UNSUPPORTED
    assert lib.tlg_mx_size(0, 1, 1, None, ctypes.byref(s)) == tlg.TLG_ERR_INVALID_ARG
    assert (q.value, s.value) == (0, 0)


def test_quantize_refusals(tlg):
    f = tlg.raw_library().tlg_mx_quantize

    def call(fmt=0, rows=8, cols=64, op=0, type=1, X=A, ldx=64, Q=2 * A, ldq=32, S=3 * A):
        return f(fmt, rows, cols, op, type, X, ldx, Q, ldq, S, None)

    bad, align, unsup = tlg.TLG_ERR_INVALID_ARG, tlg.TLG_ERR_ALIGNMENT, tlg.TLG_ERR_UNSUPPORTED
    assert call(fmt=2) == bad and call(type=3) == bad and call(op=2) == bad
    assert call(rows=-1) == bad and call(cols=2 ** 31) == unsup
    assert call(X=None) == bad and call(Q=None) == bad and call(S=None) == bad
    assert call(ldx=63) == bad and call(ldq=16) == bad
    assert call(op=1, ldx=7) == bad  # X is cols x rows: ldx >= rows
    assert call(X=A + 1) == align and call(type=0, X=A + 2) == align
    assert call(Q=2 * A + 8) == align and call(ldq=40) == align and call(S=3 * A + 4) == align
    assert call(Q=A + 16) == bad and call(S=A + 64) == bad  # an output over the input
    assert call(S=2 * A + 32) == bad  # scales over elements
    assert call(rows=2 ** 30, ldx=2 ** 36) == unsup
    assert call(ldq=40) == align and call(rows=1, ldq=40) != align  # a single row's stride does not matter
    assert call(rows=0, X=None, Q=None, S=None) == tlg.TLG_OK
    assert call(cols=0, X=None, Q=None, S=None) == tlg.TLG_OK


def test_dequantize_refusals(tlg):
    f = tlg.raw_library().tlg_mx_dequantize

    def call(fmt=1, rows=8, cols=64, Q=A, ldq=64, S=3 * A, type=1, X=2 * A, ldx=64):
        return f(fmt, rows, cols, Q, ldq, S, type, X, ldx, None)

    bad, align = tlg.TLG_ERR_INVALID_ARG, tlg.TLG_ERR_ALIGNMENT
    assert call(fmt=-1) == bad and call(type=7) == bad and call(ldq=48) == bad and call(ldx=10) == bad
    assert call(X=A) == bad and call(X=3 * A) == bad
    assert call(X=2 * A + 1) == align and call(Q=A + 2) == align
    assert call(rows=0) == tlg.TLG_OK


def test_activation_refusals(tlg):
    lib = tlg.raw_library()

    def fwd(rows=8, cols=64, act=2, type=1, Z=A, ldz=64, Y=2 * A, ldy=64, Q=3 * A, ldq=64, S=4 * A):
        return lib.tlg_act_forward_mx(rows, cols, act, type, Z, ldz, Y, ldy, Q, ldq, S, None)

    bad, align = tlg.TLG_ERR_INVALID_ARG, tlg.TLG_ERR_ALIGNMENT
    assert fwd(act=5) == bad and fwd(act=-1) == bad and fwd(type=3) == bad
    assert fwd(Y=A + 2) == bad and fwd(Y=A, ldy=72) == bad  # over Z, but not Z itself
    assert fwd(Q=2 * A) == bad and fwd(S=A) == bad and fwd(ldq=32) == bad
    assert fwd(Y=2 * A + 1) == align and fwd(rows=0) == tlg.TLG_OK

    def bwd(rows=8, cols=64, act=2, type=1, dY=A, lddy=64, Q=3 * A, ldq=64, S=4 * A, dZ=2 * A, lddz=64, db=None,
            ws=None, n=0):
        return lib.tlg_act_backward_mx(rows, cols, act, type, dY, lddy, Q, ldq, S, dZ, lddz, db, ws, n, None)

    assert bwd(act=9) == bad and bwd(dZ=3 * A) == bad and bwd(dZ=A + 2) == bad and bwd(lddy=8) == bad
    assert bwd(db=5 * A + 2) == align and bwd(ws=5 * A + 16, n=64) == align
    assert bwd(db=2 * A) == bad and bwd(ws=A, n=256) == bad and bwd(db=5 * A, ws=5 * A, n=4096) == bad
    assert bwd(cols=0) == tlg.TLG_OK and bwd(rows=0) == tlg.TLG_OK  # no dbias: nothing to write
    n = ctypes.c_size_t(3)
    assert lib.tlg_act_backward_mx_workspace_size(8, 8, 4, ctypes.byref(n)) == bad and n.value == 0
    assert lib.tlg_act_backward_mx_workspace_size(8, 8, 1, None) == bad


def test_product_refusals(tlg):
    lib = tlg.raw_library()

    def call(M=8, N=8, K=64, Am=A, lda=32, SA=2 * A, B=3 * A, ldb=32, SB=4 * A, epi=None, C=5 * A, ldc=8, out=1):
        return lib.tlg_gemm_mxfp4(M, N, K, Am, lda, SA, B, ldb, SB, ctypes.byref(epi) if epi else None, C, ldc, out,
                                  None, None)

    E = tlg.tlg_fused_epilogue
    bad, align, unsup = tlg.TLG_ERR_INVALID_ARG, tlg.TLG_ERR_ALIGNMENT, tlg.TLG_ERR_UNSUPPORTED
    assert call(M=-1) == bad and call(out=3) == bad and call(K=2 ** 31) == unsup and call(M=2 ** 31 - 300, N=2 ** 20) == unsup
    assert call(Am=None) == bad and call(SB=None) == bad and call(C=None) == bad
    assert call(lda=16) == bad and call(ldb=31) == bad and call(ldc=7) == bad
    assert call(lda=40) == align and call(B=3 * A + 8) == align and call(SA=2 * A + 8) == align
    assert call(C=5 * A + 1) == align and call(C=5 * A + 2, out=0) == align
    assert call(C=A) == bad and call(C=4 * A) == bad  # C over A, over B's scales
    assert call(epi=E(None, 5, None, 0)) == bad and call(epi=E(6 * A + 1, 0, None, 0)) == align
    assert call(epi=E(5 * A, 0, None, 0)) == bad and call(epi=E(None, 0, 5 * A, 16)) == bad
    assert call(epi=E(None, 0, 6 * A, 7)) == bad and call(epi=E(None, 0, 6 * A + 1, 8)) == align
    assert call(M=0) == tlg.TLG_OK and call(N=0) == tlg.TLG_OK
    assert lib.tlg_choose_config_mxfp4(8, 8, 8, 1, None) == bad


def test_product_binding_refusals(tlg):
    Q, S = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    with pytest.raises(ValueError):
        tlg.tlg_gemm_mxfp4(Q, S, Q[:, :16], S)
    with pytest.raises(ValueError):
        tlg.tlg_gemm_mxfp4(Q[:, :24], S, Q[:, :24], S)
    with pytest.raises(ValueError):
        tlg.tlg_gemm_mxfp4(Q, S[:256], Q, S)
    with pytest.raises(ValueError):
        tlg.tlg_gemm_mxfp4(Q, S, Q, S, out="bf16", bias=torch.zeros(4, dtype=torch.float16))
    with pytest.raises(ValueError):
        tlg.tlg_gemm_mxfp4(Q, S, Q, S, residual=torch.zeros((4, 4)))
    with pytest.raises(ValueError):
        tlg.tlg_gemm_mxfp4(Q, S, Q, S, activation="swish")
    with pytest.raises(tlg.TlgError):
        tlg.tlg_gemm_mxfp4(Q, S, Q, S)


def test_binding_refusals(tlg):
    X = torch.zeros((4, 40), dtype=torch.float16)
    Q, S = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    with pytest.raises(ValueError):
        tlg.tlg_mx_quantize(X, format="e3m2")
    with pytest.raises(TypeError):
        tlg.tlg_mx_quantize(X.double())
    with pytest.raises(ValueError):
        tlg.tlg_mx_quantize(X, Q=Q[:, :16], S=S)  # 40 columns are two blocks
    with pytest.raises(ValueError):
        tlg.tlg_mx_quantize(X, Q=Q, S=S[:100])
    with pytest.raises(ValueError):
        tlg.tlg_mx_dequantize(Q, S, 65)
    with pytest.raises(ValueError):
        tlg.tlg_mx_dequantize(Q, S, 40, out="f64")
    with pytest.raises(ValueError):
        tlg.tlg_act_forward_mx(X, "swish")
    with pytest.raises(ValueError):
        tlg.tlg_act_backward_mx(X, Q, S, "gelu")  # e4m3 rows of 40 columns are 64 bytes
    with pytest.raises(tlg.TlgError):  # no CPU fallback
        tlg.tlg_mx_quantize(X, Q=Q, S=S)


def test_workspace_must_be_contiguous(tlg):
    """A broadcast tensor has more elements than bytes behind it."""
    X = torch.zeros((4, 40), dtype=torch.float16)
    Q, S = torch.zeros((4, 64), dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    for workspace in (torch.zeros(1).expand(1 << 20), torch.zeros(1 << 12)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            tlg.tlg_act_backward_mx(X, Q, S, "gelu", workspace=workspace)


def test_choose_config_refusals(tlg):
    lib, bad = tlg.raw_library(), tlg.TLG_ERR_INVALID_ARG
    cfg, E = tlg.tlg_config(), tlg.tlg_fused_epilogue
    assert lib.tlg_choose_config_mxfp4_fused(8, 8, 8, None, 1, None) == bad
    assert lib.tlg_choose_config_mxfp4_fused(8, -8, 8, None, 1, ctypes.byref(cfg)) == bad
    assert lib.tlg_choose_config_mxfp4_fused(8, 8, 8, ctypes.byref(E(None, 9, None, 0)), 1, ctypes.byref(cfg)) == bad
    with pytest.raises(ValueError):
        tlg.tlg_choose_config_mxfp4_fused(8, 8, 8, activation="swish")


@pytest.mark.parametrize("op", ["transpose", "", "TN", None, 1])
def test_quantize_refuses_other_ops(tlg, op):
    with pytest.raises(ValueError, match="op"):
        tlg.tlg_mx_quantize(torch.zeros((4, 40), dtype=torch.float16), op=op)
