"""GPU tests of the root-mean-square norm, with the residual's addition and microscaled outputs, and of
its backward pass, against the formulas in 64 bits.

Tolerances: in fp32 a row's sum of n squares is off by at most n 2^-24 relative (in fact far less: lanes
sum n / 32 or fewer terms each, then shuffles), rstd by half of that and its own rounding, a product by 2^-24 each, so
the fp32 value of Y is within (n / 64 + 8) 2^-24; the stored type adds half a unit, eps / 2."""

import numpy as np
import pytest
import torch

from oracle import mx

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SHAPES = [(1, 1), (1, 32), (3, 33), (5, 256), (9, 257), (2, 1000), (1, 4096), (7, 4095), (500, 520), (3, 2049), (2, 8192),
          (2, 8200), (1, 16384), (3, 16383)]


@pytest.fixture(scope="module")
def tlg():
    import tiled_dense_gemm_tlg_b200 as t
    return t


def f32_error(cols):
    return (cols / 64 + 8) * 2.0 ** -24


class Strided:
    """A matrix inside a larger buffer: `lead` elements in front, `extra` behind each row."""

    def __init__(self, host, lead=0, extra=0):
        rows, cols = host.shape
        self.buf = torch.full((lead + rows * (cols + extra) + 64,), -77.0, device="cuda").to(host.dtype)
        self.view = self.buf[lead:lead + rows * (cols + extra)].view(rows, cols + extra)[:, :cols]
        self.view.copy_(host)
        self.mask = torch.ones(self.buf.shape, dtype=torch.bool, device="cuda")
        self.mask[lead:lead + rows * (cols + extra)].view(rows, cols + extra)[:, :cols] = False
        self.before = self.buf.clone()

    def guards_kept(self):
        return bool((self.buf[self.mask] == self.before[self.mask]).all())


def rows_of(seed, rows, cols, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * torch.exp2(torch.randint(-4, 5, (rows, 1), generator=g).float()) * scale
    if rows > 2:
        x[1] = 0
    return x.to(dtype)


def forward(X, R, w, eps):
    h = X.double() if R is None else X.double() + R.double()
    rstd = 1 / torch.sqrt((h * h).mean(dim=1) + eps)
    return h, rstd, h * rstd[:, None] * w.double()


def near(got, want, rel, dtype):
    """Within rel of the value's magnitude and half a unit of the stored type (subnormals: half their step)."""
    fi = torch.finfo(dtype)
    bound = want.abs() * (rel + fi.eps / 2) + fi.tiny * fi.eps
    bad = (got.double().cpu() - want).abs() > bound
    assert torch.isfinite(got).all() and not bad.any(), (bad.nonzero()[:4], got.cpu()[bad][:4], want[bad][:4])


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(tlg, rows, cols, residual, typ):
    dt = TYPES[typ]
    X, R = rows_of(1, rows, cols, dt), rows_of(2, rows, cols, dt) if residual else None
    w = (1 + 0.2 * torch.randn(cols, generator=torch.Generator().manual_seed(3))).to(dt)
    eps = 1e-5
    h, rstd, y = forward(X, R, w, eps)
    r = None if R is None else R.cuda()
    Y, H, s = tlg.tlg_rmsnorm_forward(X.cuda(), w.cuda(), residual=r, eps=eps)
    near(s, rstd, f32_error(cols), torch.float32)
    # h in fp32 is off by half a unit of itself, which reaches y
    near(Y, y, f32_error(cols), dt)
    near(H, h, 2.0 ** -24, dt)
    if R is None:
        assert H.data_ptr() and torch.equal(H.cpu(), X)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("lead,extra", [(0, 0), (1, 1), (3, 2), (0, 5), (2, 0)])
@pytest.mark.parametrize("rows,cols", [(1, 5), (6, 77), (40, 515), (3, 5001)])
def test_forward_any_alignment(tlg, rows, cols, lead, extra, typ):
    dt = TYPES[typ]
    X, R = Strided(rows_of(4, rows, cols, dt), lead, extra), Strided(rows_of(5, rows, cols, dt), extra, lead)
    w = Strided((1 + 0.2 * torch.randn((1, cols), generator=torch.Generator().manual_seed(6))).to(dt), lead)
    H, Y = Strided(torch.zeros((rows, cols), dtype=dt), lead, 3), Strided(torch.zeros((rows, cols), dtype=dt), 5, extra)
    h, rstd, y = forward(X.view.cpu(), R.view.cpu(), w.view[0].cpu(), 0.0 if rows < 3 else 1e-6)
    tlg.tlg_rmsnorm_forward(X.view, w.view[0], residual=R.view, eps=0.0 if rows < 3 else 1e-6, H=H.view, Y=Y.view)
    near(Y.view, y, f32_error(cols), dt)
    near(H.view, h, 2.0 ** -24, dt)
    assert H.guards_kept() and Y.guards_kept()
    # the same bits with whole 16-byte accesses
    Y2, H2, _ = tlg.tlg_rmsnorm_forward(X.view.contiguous(), w.view[0].clone(), residual=R.view.contiguous(),
                                        eps=0.0 if rows < 3 else 1e-6)
    assert torch.equal(Y2, Y.view) and torch.equal(H2, H.view)


@pytest.mark.parametrize("cols", [64, 515, 4096, 16384])
@pytest.mark.parametrize("typ", list(TYPES))
def test_forward_in_place(tlg, cols, typ):
    """H in the residual's place and Y in X's, rows more than are taken at once."""
    dt, rows = TYPES[typ], 1500 if cols < 5000 else 400
    X, R, w = rows_of(7, rows, cols, dt).cuda(), rows_of(8, rows, cols, dt).cuda(), torch.ones(cols, dtype=dt).cuda()
    Y, H, s = tlg.tlg_rmsnorm_forward(X, w, residual=R)
    x, r = X.clone(), R.clone()
    tlg.tlg_rmsnorm_forward(x, w, residual=r, H=r, Y=x)
    assert torch.equal(x, Y) and torch.equal(r, H)
    x, r = X.clone(), R.clone()
    tlg.tlg_rmsnorm_forward(x, w, residual=r, H=x, Y=r)
    assert torch.equal(x, H) and torch.equal(r, Y)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("rows,cols", [(1, 1), (2, 31), (130, 96), (5, 257), (3, 4096), (40, 1000), (2, 16384)])
def test_forward_mx(tlg, rows, cols, typ, fmt):
    """The MX output is the quantisation of fp32 values within their error of Y: every element lies
    between the quantisations of Y less and of Y plus that error, in a scale that either bound gives."""
    dt = TYPES[typ]
    X, R = rows_of(9, rows, cols, dt), rows_of(10, rows, cols, dt)
    w = (1 + 0.2 * torch.randn(cols, generator=torch.Generator().manual_seed(11))).to(dt)
    h, rstd, y = forward(X, R, w, 1e-6)
    Q, S, H, s = tlg.tlg_rmsnorm_forward_mx(X.cuda(), w.cuda(), residual=R.cuda(), format=fmt)
    near(s, rstd, f32_error(cols), torch.float32)
    near(H, h, 2.0 ** -24, dt)
    got = tlg.tlg_mx_dequantize(Q, S, cols, format=fmt, out="f32").double().cpu().numpy()
    y, e = y.numpy(), f32_error(cols)
    lo, hi = (mx.decode(*mx.quantize(y * f, fmt), fmt)[:, :cols] for f in (1 - e, 1 + e))
    # where both give one scale the element lies between them; a block whose largest value is next to a power
    # of two may take either scale, each of which is off by at most half its own step
    least, most = np.minimum(lo, hi), np.maximum(lo, hi)
    nb = -(-cols // 32)
    s_lo, s_hi = (mx.quantize(y * f, fmt)[1] for f in (1 - e, 1 + e))
    same = np.repeat(s_lo[:, :nb] == s_hi[:, :nb], 32, axis=1)[:, :cols]
    assert ((got >= least) & (got <= most))[same].all()
    assert same.mean() > 0.9 or cols < 64
    # the bytes past the last block are 0
    got_s = S.cpu().numpy()[mx.scale_index(rows, -(-nb // 4) * 4)]
    assert (got_s[:, nb:] == 0).all()


def test_forward_mx_feeds_the_4_bit_product(tlg):
    """The norm's 4-bit output is what tlg_gemm_mxfp4 takes, and equals quantising Y's fp32 values."""
    X, W = rows_of(12, 20, 512, torch.float32), rows_of(13, 96, 512, torch.bfloat16)
    w = torch.ones(512)
    Q, S, _, _ = tlg.tlg_rmsnorm_forward_mx(X.cuda(), w.cuda(), format="e2m1")
    Y, _, _ = tlg.tlg_rmsnorm_forward(X.cuda(), w.cuda())
    Q2, S2 = tlg.tlg_mx_quantize(Y)
    assert torch.equal(Q, Q2)
    Wq, Ws = tlg.tlg_mx_quantize(W.cuda())
    assert torch.equal(tlg.tlg_gemm_mxfp4(Q, S, Wq, Ws), tlg.tlg_gemm_mxfp4(Q2, S2, Wq, Ws))


@pytest.mark.parametrize("typ", list(TYPES))
def test_special_values(tlg, typ):
    dt = TYPES[typ]
    X = rows_of(14, 6, 200, dt)
    X[2, 5], X[3, 199], X[4] = float("nan"), float("inf"), 0
    w = torch.ones(200, dtype=dt)
    Y, _, s = tlg.tlg_rmsnorm_forward(X.cuda(), w.cuda(), eps=0.0)
    assert torch.isnan(Y[2]).all() and torch.isnan(Y[4]).all()
    assert torch.isnan(Y[3, 199]) and (Y[3, :199] == 0).all() and s[3] == 0
    assert torch.isfinite(Y[[0, 5]]).all()
    Q, S, _, _ = tlg.tlg_rmsnorm_forward_mx(X.cuda(), w.cuda(), eps=0.0)
    back = tlg.tlg_mx_dequantize(Q, S, 200, format="e4m3", out="f32")
    assert torch.isnan(back[2]).all() and torch.isnan(back[4]).all() and torch.isnan(back[3, 192:]).all()
    got_s = S.cpu().numpy()[mx.scale_index(6, 8)]
    assert (got_s[:, 7] == 0).all() and torch.isfinite(back[[0, 5]]).all()


# ------------------------------------------------------------------ backward


def backward(dY, H, w, rstd, dH):
    """dX, dweight and bounds of the fp32 computation: products and sums of magnitudes."""
    dY, H, w, rstd = dY.double(), H.double(), w.double(), rstd.double()[:, None]
    x, g = H * rstd, dY * w
    dot = (g * x).mean(dim=1, keepdim=True)
    dx = rstd * (g - x * dot)
    n = H.shape[1]
    err = rstd * (8 * g.abs() + x.abs() * (n / 64 + 16) * (g * x).abs().mean(dim=1, keepdim=True)) * 2.0 ** -24
    if dH is not None:
        dx = dx + dH.double()
        err = err + 2.0 ** -24 * dx.abs()
    t = dY * x
    # a sum over r rows: at most r terms in a chain, each step half a unit of the partial sum
    return dx, err, t.sum(dim=0), (H.shape[0] + 4) * 2.0 ** -24 * t.abs().sum(dim=0)


def check(got, want, err, dtype):
    fi = torch.finfo(dtype)
    bad = (got.double().cpu() - want).abs() > err + want.abs() * fi.eps / 2 + fi.tiny * fi.eps
    assert torch.isfinite(got).all() and not bad.any(), (bad.nonzero()[:4], got.cpu()[bad][:4], want[bad][:4])


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("stream_grad", [False, True])
@pytest.mark.parametrize("rows,cols", SHAPES + [(1500, 96), (700, 1100)])
def test_backward(tlg, rows, cols, stream_grad, typ):
    dt = TYPES[typ]
    H, dY = rows_of(15, rows, cols, dt), rows_of(16, rows, cols, dt, 0.25)
    dH = rows_of(17, rows, cols, dt, 0.25) if stream_grad else None
    w = (1 + 0.2 * torch.randn(cols, generator=torch.Generator().manual_seed(18))).to(dt)
    rstd = (1 / torch.sqrt((H.double() ** 2).mean(dim=1) + 1e-2)).float()
    want, err, dw, dw_err = backward(dY, H, w, rstd, dH)
    d = None if dH is None else dH.cuda()
    dX, dweight = tlg.tlg_rmsnorm_backward(dY.cuda(), H.cuda(), w.cuda(), rstd.cuda(), dH=d)
    check(dX, want, err, dt)
    check(dweight, dw, dw_err, torch.float32)
    again, none = tlg.tlg_rmsnorm_backward(dY.cuda(), H.cuda(), w.cuda(), rstd.cuda(), dH=d, weight_grad=False)
    assert none is None and torch.equal(again, dX)
    assert torch.equal(tlg.tlg_rmsnorm_backward(dY.cuda(), H.cuda(), w.cuda(), rstd.cuda())[1], dweight)


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("lead,extra", [(1, 1), (3, 2), (0, 5)])
@pytest.mark.parametrize("rows,cols", [(1, 5), (60, 77), (40, 515), (3, 5001)])
def test_backward_any_alignment(tlg, rows, cols, lead, extra, typ):
    dt = TYPES[typ]
    H, dY, dH = (Strided(rows_of(s, rows, cols, dt), lead, extra) for s in (19, 20, 21))
    w = Strided(torch.ones((1, cols), dtype=dt), lead)
    rstd = (1 / torch.sqrt((H.view.double().cpu() ** 2).mean(dim=1) + 1e-2)).float().cuda()
    dX = Strided(torch.zeros((rows, cols), dtype=dt), extra, lead)
    _, dweight = tlg.tlg_rmsnorm_backward(dY.view, H.view, w.view[0], rstd, dH=dH.view, dX=dX.view)
    want, err, dw, dw_err = backward(*(t.cpu() for t in (dY.view, H.view, w.view[0], rstd, dH.view)))
    check(dX.view, want, err, dt)
    check(dweight, dw, dw_err, torch.float32)
    assert dX.guards_kept()
    for at in (dY, dH):  # in place
        clone = [Strided(t.view.cpu(), lead, extra) for t in (dY, dH)]
        into = clone[0] if at is dY else clone[1]
        tlg.tlg_rmsnorm_backward(clone[0].view, H.view, w.view[0], rstd, dH=clone[1].view, dX=into.view)
        assert torch.equal(into.view, dX.view) and into.guards_kept()


def test_backward_against_differences(tlg):
    """Central differences of sum(Y * G) + sum(H * K) in 64 bits, H = X + R and Y its norm."""
    g = torch.Generator().manual_seed(22)
    X, R, G, K = (torch.randn((3, 40), generator=g) for _ in range(4))
    w = 1 + 0.2 * torch.randn(40, generator=g)
    eps = 1e-3
    _, H, rstd = tlg.tlg_rmsnorm_forward(X.cuda(), w.cuda(), residual=R.cuda(), eps=eps)
    dX, dw = (t.double().cpu() for t in tlg.tlg_rmsnorm_backward(G.cuda(), H, w.cuda(), rstd, dH=K.cuda()))

    def value(x, w):
        h, _, y = forward(x, R, w, eps)
        return (y * G.double()).sum() + (h * K.double()).sum()

    x, w, step = X.double(), w.double(), 1e-5
    for t, d, at in [(x, dX, (r, c)) for r in range(3) for c in (0, 7, 39)] + [(w, dw, (c,)) for c in (0, 20, 39)]:
        old = t[at].item()
        t[at] = old + step
        up = value(x, w)
        t[at] = old - step
        down = value(x, w)
        t[at] = old
        # the difference is off by step^2 times a third derivative of about 1; the fp32 gradient by some 2^-22
        assert abs((up - down) / (2 * step) - d[at]) < 3e-5


def test_no_rows(tlg):
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    none = torch.zeros((0, 64), dtype=torch.float16, device="cuda")
    Y, _, s = tlg.tlg_rmsnorm_forward(none, w)
    assert Y.shape == (0, 64) and s.shape == (0,)
    dw = torch.full((64,), 5.0, device="cuda")
    tlg.tlg_rmsnorm_backward(none, none, w, s, dweight=dw)
    assert (dw == 0).all()


def test_streams_graphs_and_workspaces(tlg):
    """Two calls at once with workspaces of their own, and both passes captured and replayed on new rows."""
    rows, cols = 300, 1000
    X, R = (rows_of(s, rows, cols, torch.bfloat16).cuda() for s in (23, 24))
    w = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    Y, H, rstd = tlg.tlg_rmsnorm_forward(X, w, residual=R)
    dX, dw = tlg.tlg_rmsnorm_backward(Y, H, w, rstd, dH=R)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [tlg.tlg_rmsnorm_backward(Y, H, w, rstd, dH=R, stream=s) for _ in range(5) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, dX) and torch.equal(b, dw) for a, b in got)
    ws = tlg.tlg_workspace(tlg.tlg_rmsnorm_backward_workspace_size(rows, cols, "bf16"))
    outs = [torch.empty_like(t) for t in (Y, H, rstd, dX, dw)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tlg.tlg_rmsnorm_forward(X, w, residual=R, Y=outs[0], H=outs[1], rstd=outs[2])
        tlg.tlg_rmsnorm_backward(outs[0], outs[1], w, outs[2], dH=R, dX=outs[3], dweight=outs[4], workspace=ws)
    X.mul_(0.5)
    ws.fill_(255)
    graph.replay()
    Y, H, rstd = tlg.tlg_rmsnorm_forward(X, w, residual=R)
    dX, dw = tlg.tlg_rmsnorm_backward(Y, H, w, rstd, dH=R)
    assert all(torch.equal(a, b) for a, b in zip(outs, (Y, H, rstd, dX, dw)))
