"""What the operators around the linear layers refuse, on the host and before any CUDA call: products
grouped by expert, the root-mean-square norm and the products with 4-bit weights."""

import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B, C, O, X = (1 << 20) * 16, (1 << 20) * 32, (1 << 20) * 48, (1 << 20) * 64, (1 << 20) * 80  # fake, far apart


@pytest.fixture(scope="module")
def tlg():
    import importlib.util

    spec = importlib.util.spec_from_file_location("tlg_build", os.path.join(ROOT, "tiled_dense_gemm_tlg_b200", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.build()
    import tiled_dense_gemm_tlg_b200 as t
    return t


INVALID, ALIGNMENT, UNSUPPORTED, OK = 1, 2, 3, 0


def grouped(tlg, rows=8, n=16, k=32, groups=3, offsets=O, typ=1, a=A, lda=32, op=0, b=B, ldb=16, stride=512, act=0, c=C,
            ldc=16, out=1):
    return tlg.raw_library().tlg_gemm_grouped(rows, n, k, groups, offsets, typ, a, lda, op, b, ldb, stride, act, c, ldc,
                                              out, None)


def test_grouped_refusals(tlg):
    for bad in (dict(rows=-1), dict(groups=-1), dict(typ=0), dict(typ=7), dict(out=2), dict(out=5), dict(op=2),
                dict(act=9), dict(offsets=None), dict(a=None), dict(b=None), dict(c=None), dict(lda=31), dict(ldb=15),
                dict(ldc=15), dict(stride=-8), dict(c=A), dict(c=B + 2 * 512 * 2), dict(c=O)):
        assert grouped(tlg, **bad) == INVALID, bad
    for bad in (dict(a=A + 1), dict(b=B + 1), dict(c=C + 1), dict(offsets=O + 2), dict(c=C + 2, out=0)):
        assert grouped(tlg, **bad) == ALIGNMENT, bad
    for bad in (dict(groups=1025), dict(rows=2 ** 31), dict(n=2 ** 31), dict(k=2 ** 31), dict(lda=2 ** 37),
                dict(stride=2 ** 39), dict(rows=2 ** 31 - 300, n=2 ** 31 - 300, ldb=2 ** 31, ldc=2 ** 31)):
        assert grouped(tlg, **bad) in (UNSUPPORTED, INVALID), bad
    assert grouped(tlg, op=1, ldb=31) == INVALID  # N x K needs K
    for empty in (dict(rows=0, a=None, c=None), dict(n=0, c=None), dict(groups=0, offsets=None)):
        assert grouped(tlg, **empty) == OK, empty


def grouped_dw(tlg, rows=8, n=16, k=32, groups=3, offsets=O, typ=1, a=A, lda=32, d=B, ldd=16, op=0, db=C, lddb=16,
               stride=512, out=1):
    return tlg.raw_library().tlg_gemm_grouped_dw(rows, n, k, groups, offsets, typ, a, lda, d, ldd, op, db, lddb, stride,
                                                 out, None)


def test_grouped_dw_refusals(tlg):
    for bad in (dict(rows=-1), dict(typ=0), dict(out=2), dict(op=5), dict(offsets=None), dict(a=None), dict(d=None),
                dict(db=None), dict(lda=31), dict(ldd=15), dict(lddb=15), dict(stride=511), dict(stride=0),
                dict(db=A), dict(db=B), dict(db=O), dict(op=1, lddb=31)):
        assert grouped_dw(tlg, **bad) == INVALID, bad
    for bad in (dict(a=A + 1), dict(d=B + 1), dict(db=C + 1), dict(offsets=O + 1)):
        assert grouped_dw(tlg, **bad) == ALIGNMENT, bad
    assert grouped_dw(tlg, groups=2000) == UNSUPPORTED
    for empty in (dict(n=0, db=None), dict(k=0), dict(groups=0)):
        assert grouped_dw(tlg, **empty) == OK, empty


def forward(tlg, rows=4, cols=64, typ=2, x=A, ldx=64, r=B, ldr=64, w=O, eps=1e-6, h=C, ldh=64, y=X, ldy=64, rstd=None):
    return tlg.raw_library().tlg_rmsnorm_forward(rows, cols, typ, x, ldx, r, ldr, w, eps, h, ldh, y, ldy, rstd, None)


def test_norm_refusals(tlg):
    nan, inf = float("nan"), float("inf")
    for bad in (dict(rows=-1), dict(typ=3), dict(eps=-1e-6), dict(eps=nan), dict(eps=inf), dict(x=None), dict(w=None),
                dict(y=None), dict(ldx=63), dict(ldr=63), dict(ldh=63), dict(ldy=63), dict(h=X), dict(y=C + 2),
                dict(h=A + 2 * 64), dict(y=A, ldy=65), dict(h=O), dict(rstd=C), dict(rstd=A)):
        assert forward(tlg, **bad) == INVALID, bad
    for bad in (dict(x=A + 1), dict(r=B + 1), dict(w=O + 1), dict(h=C + 1), dict(y=X + 1), dict(rstd=O + 4098)):
        assert forward(tlg, **bad) == ALIGNMENT, bad
    assert forward(tlg, typ=0, x=A + 2) == ALIGNMENT
    assert forward(tlg, cols=16385, ldx=20000, ldr=20000, ldh=20000, ldy=20000) == UNSUPPORTED
    assert forward(tlg, rows=0, x=None, y=None) == OK and forward(tlg, cols=0) == OK
    mx = tlg.raw_library().tlg_rmsnorm_forward_mx
    args = [4, 64, 2, A, 64, None, 0, O, 1e-6, None, 0, 1, C, 64, X, None, None]
    for i, v, want in ((11, 2, INVALID), (11, -1, INVALID), (12, None, INVALID), (14, None, INVALID), (13, 48, INVALID),
                       (12, C + 8, ALIGNMENT), (13, 72, ALIGNMENT), (14, X + 4, ALIGNMENT), (12, A, INVALID), (14, C, INVALID)):
        bad = list(args)
        bad[i] = v
        assert mx(*bad) == want, (i, v)


def backward(tlg, rows=4, cols=64, typ=2, dy=A, lddy=64, h=B, ldh=64, w=O, rstd=O + 4096, dh=None, lddh=64, dx=C,
             lddx=64, dw=X, ws=X + (1 << 20), size=1 << 20):
    return tlg.raw_library().tlg_rmsnorm_backward(rows, cols, typ, dy, lddy, h, ldh, w, rstd, dh, lddh, dx, lddx, dw, ws,
                                                  size, None)


def test_norm_backward_refusals(tlg):
    for bad in (dict(rows=-1), dict(typ=4), dict(dy=None), dict(h=None), dict(w=None), dict(rstd=None), dict(dx=None),
                dict(lddy=63), dict(lddh=63, dh=A), dict(dx=B), dict(dx=A + 2), dict(dx=A, lddx=80), dict(dx=O),
                dict(dw=A), dict(dw=C), dict(ws=A), dict(ws=C), dict(dw=X, ws=X)):
        assert backward(tlg, **bad) == INVALID, bad
    for bad in (dict(dy=A + 1), dict(dx=C + 1), dict(rstd=O + 4097), dict(dw=X + 2), dict(ws=X + (1 << 20) + 16)):
        assert backward(tlg, **bad) == ALIGNMENT, bad
    assert backward(tlg, cols=16385) == UNSUPPORTED
    n = ctypes.c_size_t(5)
    size = tlg.raw_library().tlg_rmsnorm_backward_workspace_size
    assert size(4, 64, 9, ctypes.byref(n)) == INVALID and n.value == 0
    assert size(4, 20000, 2, ctypes.byref(n)) == UNSUPPORTED and size(4, 64, 2, None) == INVALID
    assert size(0, 64, 2, ctypes.byref(n)) == OK and n.value == 0


def gemv(tlg, m=2, n=32, k=256, typ=1, x=A, ldx=256, q=B, ldq=128, s=O, z=None, group=64, epi=None, c=C, ldc=32, out=1):
    e = ctypes.byref(tlg.tlg_fused_epilogue(*epi)) if epi is not None else None
    return tlg.raw_library().tlg_gemv_q4(m, n, k, typ, x, ldx, q, ldq, s, z, group, e, c, ldc, out, None)


def test_gemv_refusals(tlg):
    for bad in (dict(m=-1), dict(typ=0), dict(out=2), dict(group=0), dict(group=16), dict(group=48), dict(group=-64),
                dict(x=None), dict(q=None), dict(s=None), dict(c=None), dict(ldx=255), dict(ldq=112), dict(ldc=31),
                dict(c=A), dict(c=B), dict(c=O), dict(z=C), dict(epi=(None, 9, None, 0)), dict(epi=(None, 0, C + 64, 32)),
                dict(epi=(C, 0, None, 0)), dict(epi=(None, 0, X, 31))):
        assert gemv(tlg, **bad) == INVALID, bad
    for bad in (dict(x=A + 1), dict(q=B + 8), dict(ldq=136), dict(s=O + 1), dict(c=C + 1), dict(epi=(X + 1, 0, None, 0))):
        assert gemv(tlg, **bad) == ALIGNMENT, bad
    for bad in (dict(k=2 ** 31), dict(group=2 ** 32), dict(ldq=2 ** 37)):
        assert gemv(tlg, **bad) == UNSUPPORTED, bad
    assert gemv(tlg, m=0, x=None) == OK and gemv(tlg, n=0, q=None) == OK


def test_binding_checks(tlg):
    h = torch.zeros
    a, b, off = h((8, 32)).half(), h((3, 32, 16)).half(), h(4, dtype=torch.int32)
    for args, kw, err in (((a, b, off.long()), {}, ValueError), ((a, b[:2], off), {}, ValueError),
                          ((a, b, off), {"op_b": "T"}, ValueError), ((a, b, off), {"op_b": "X"}, ValueError),
                          ((a, b.bfloat16(), off), {}, TypeError), ((a, b, off), {"activation": "tanh"}, ValueError),
                          ((a, b, off), {"out": "f64"}, ValueError), ((a, b.transpose(1, 2), off), {}, ValueError),
                          ((a, b, off), {"C": h((8, 15)).half()}, ValueError), ((a[0], b, off), {}, ValueError),
                          ((a, b[0], off), {}, ValueError)):
        with pytest.raises(err):
            tlg.tlg_gemm_grouped(*args, **kw)
    d = h((8, 16)).half()
    for args, kw, err in (((a, d[:7], off), {}, ValueError), ((a, d.float(), off), {}, TypeError),
                          ((a, d, off), {"dB": h((3, 16, 32)).half()}, ValueError)):
        with pytest.raises(err):
            tlg.tlg_gemm_grouped_dw(*args, **kw)
    x, w = h((4, 64)), h(64)
    for call, err in ((lambda: tlg.tlg_rmsnorm_forward(x, w[:63]), ValueError),
                      (lambda: tlg.tlg_rmsnorm_forward(x, w.half()), ValueError),
                      (lambda: tlg.tlg_rmsnorm_forward(x, w, residual=x[:3]), ValueError),
                      (lambda: tlg.tlg_rmsnorm_forward(x.double(), w), TypeError),
                      (lambda: tlg.tlg_rmsnorm_forward(x.t(), w), ValueError),
                      (lambda: tlg.tlg_rmsnorm_forward_mx(x, w, format="e5m2"), ValueError),
                      (lambda: tlg.tlg_rmsnorm_backward(x, x[:, :32], w, h(4)), ValueError),
                      (lambda: tlg.tlg_rmsnorm_backward(x, x, w, h(3)), ValueError),
                      (lambda: tlg.tlg_rmsnorm_backward(x, x, w, h(4).half()), ValueError),
                      (lambda: tlg.tlg_rmsnorm_backward(x, x, w, h(4), dH=x.half()), ValueError)):
        with pytest.raises(err):
            call()
    X, Q, S = h((2, 256)).half(), h((32, 128), dtype=torch.uint8), h((32, 4)).half()
    for args, kw, err in (((X, Q[:, :64], S), {"group": 64}, ValueError), ((X, Q, S), {"group": 128}, ValueError),
                          ((X, Q, S.float()), {"group": 64}, ValueError), ((X, Q.int(), S), {"group": 64}, ValueError),
                          ((X, Q, S, S), {"group": 64}, ValueError), ((X, Q, S), {"group": 0}, ValueError),
                          ((X, Q, S), {"group": 64, "bias": h(31).half()}, ValueError),
                          ((X, Q, S), {"group": 64, "residual": h((2, 32))}, ValueError)):
        with pytest.raises(err):
            tlg.tlg_gemv_q4(*args, **kw)


def test_cpu_tensors_are_refused(tlg):
    """Rather than read as device memory: the library has no CPU fallback."""
    with pytest.raises(tlg.TlgError):
        tlg.tlg_rmsnorm_forward(torch.zeros((4, 64)), torch.zeros(64))
    with pytest.raises(tlg.TlgError):
        tlg.tlg_gemm_grouped(torch.zeros((8, 32)).half(), torch.zeros((3, 32, 16)).half(), torch.zeros(4, dtype=torch.int32))
