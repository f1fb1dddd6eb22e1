"""GPU tests of the microscaled (MX) elementwise operators against the fp64 reference:
quantisation of a matrix and of its transpose, dequantisation, the activation that saves its
input in 8 bits, and its backward pass.  Quantisation is exact arithmetic, so elements and
scales are compared as bytes; the float outputs' tolerances count one rounding of the stored
type (half a unit, eps / 2 relative) and the stated error of the fp32 function behind it."""

import numpy as np
import pytest
import torch

from oracle import mx

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SHAPES = [(1, 1), (1, 32), (3, 31), (5, 33), (1, 4096), (7, 4095), (128, 128), (129, 257), (200, 1000), (300, 515),
          (33, 2056)]
ACTS = ["none", "relu", "gelu", "silu", "gelu_tanh"]


@pytest.fixture(scope="module")
def tlg():
    import tiled_dense_gemm_tlg_b200 as t
    return t


def values(rows, cols, dtype, seed):
    """Values over several binades, with zero rows, zero blocks, ties and extremes of the type."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * torch.exp2(torch.randint(-6, 7, (rows, 1), generator=g).float())
    x = x.to(dtype).float()
    flat = x.view(-1)
    n = flat.numel()
    ties = torch.tensor([2.5, 3.5, 5.0, 0.25, 0.75, 7.0, 6.5, -0.0, 448.0, 449.0, 17.0])
    for i, v in enumerate(ties):
        if n > 40 * i:
            flat[(37 * i) % n] = v
    if rows > 4:
        x[rows - 2] = 0
    if rows > 8:
        x[4] *= torch.finfo(dtype).tiny  # subnormals
        x[5] = x[5].sign() * torch.finfo(dtype).max
    return x.to(dtype)


class Strided:
    """A matrix inside a larger buffer: `lead` elements in front, rows `ld` apart, filled with a pattern."""

    def __init__(self, host, lead, extra):
        rows, cols = host.shape
        self.ld = cols + extra
        self.buf = torch.full((lead + rows * self.ld + 64,), -77.0, device="cuda").to(host.dtype)
        self.view = self.buf[lead:lead + rows * self.ld].view(rows, self.ld)[:, :cols]
        self.view.copy_(host)
        self.before = self.buf.clone()
        self.mask = torch.ones_like(self.buf, dtype=torch.bool)
        self.mask[lead:lead + rows * self.ld].view(rows, self.ld)[:, :cols] = False

    def guards_kept(self):
        return bool((self.buf[self.mask] == self.before[self.mask]).all())


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def check_mx(Q, S, want_codes, want_scale, fmt):
    rows, blocks = want_scale.shape
    got_s = S.cpu().numpy()[mx.scale_index(rows, -(-blocks // 4) * 4)]
    assert np.array_equal(got_s[:, :blocks], want_scale)
    assert (got_s[:, blocks:] == 0).all()
    codes = mx.unpack(Q.cpu().numpy(), fmt)
    fine = np.repeat(want_scale != 255, 32, axis=1)  # a NaN block's elements do not matter
    assert np.array_equal(codes[fine], want_codes[fine])


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("op", ["N", "T"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_matches_reference(tlg, fmt, typ, op, rows, cols):
    x = values(rows, cols, TYPES[typ], seed=rows * 7 + cols)
    codes, scale = mx.quantize(x.double().numpy(), fmt)
    stored = x.t().contiguous() if op == "T" else x
    for lead, extra in ((0, 0), (8, 8), (1, 3)):
        m = Strided(stored, lead, extra)
        row_bytes, s_bytes = tlg.tlg_mx_size(fmt, rows, cols)
        Qb = torch.full((rows + 1, row_bytes + 16), 0xA5, dtype=torch.uint8, device="cuda")
        Sb = torch.full((s_bytes + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        Q, S = tlg.tlg_mx_quantize(m.view, format=fmt, op=op, Q=Qb[:rows, :row_bytes], S=Sb)
        check_mx(Q, S, codes, scale, fmt)
        assert (Qb[rows] == 0xA5).all() and (Qb[:, row_bytes:] == 0xA5).all()
        kept = np.ones(s_bytes + 64, dtype=bool)  # rows past the last one and the guard stay as they were
        kept[mx.scale_index(rows, -(-scale.shape[1] // 4) * 4)] = False
        assert (Sb.cpu().numpy()[kept] == 0xA5).all()
        assert m.guards_kept() and torch.equal(bits(m.view), bits(stored.cuda()))


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("op", ["N", "T"])
@pytest.mark.parametrize("typ", list(TYPES))
def test_quantize_non_finite_blocks(tlg, fmt, op, typ):
    x = values(40, 200, TYPES[typ], seed=3)
    x[0, 5], x[1, 40], x[2, 199] = float("inf"), float("nan"), -float("inf")
    codes, scale = mx.quantize(x.double().numpy(), fmt)
    assert (scale == 255).sum() == 3
    Q, S = tlg.tlg_mx_quantize((x.t().contiguous() if op == "T" else x).cuda(), format=fmt, op=op)
    check_mx(Q, S, codes, scale, fmt)
    back = tlg.tlg_mx_dequantize(Q, S, 200, format=fmt, out="f32").cpu().double().numpy()
    # rounded once to fp32: the largest fp32 number quantises up to 2^128, which is infinite there
    want = torch.from_numpy(mx.decode(codes, scale, fmt)[:, :200]).float().double().numpy()
    assert np.array_equal(back, want, equal_nan=True)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_dequantize_matches_reference(tlg, fmt, out, rows, cols):
    g = np.random.default_rng(rows + 1000 * cols)
    blocks = -(-cols // 32)
    codes = g.integers(0, 16 if fmt == "e2m1" else 256, (rows, blocks * 32)).astype(np.uint8)
    if fmt == "e4m3":
        codes[codes % 128 == 127] = 3
    scale = g.integers(100, 150, (rows, blocks)).astype(np.uint8)
    scale[0, 0] = 0
    scale[-1, -1] = 255
    want = mx.decode(codes, scale, fmt)[:, :cols]
    want = torch.from_numpy(want).to(torch.float32).to(TYPES[out])  # fp32 holds every value exactly
    Q = torch.from_numpy(mx.pack(codes, fmt)).cuda()
    S = torch.from_numpy(mx.tile_scales(scale, fill=255)).cuda()
    for lead, extra in ((0, 0), (8, 8), (1, 3)):
        m = Strided(torch.zeros((rows, cols), dtype=TYPES[out]), lead, extra)
        tlg.tlg_mx_dequantize(Q, S, cols, format=fmt, out=out, X=m.view)
        assert np.array_equal(m.view.float().cpu().numpy(), want.float().numpy(), equal_nan=True)
        assert m.guards_kept()


# The fp32 functions' stated errors: GELU 3e-7 absolute for an fp32 result, 0.15 fp16 units for a
# 16-bit one; SiLU and tanh GELU 2e-6 (1 + the largest |value|) on [-12, 12]; derivatives 1e-6.
def y_bound(act, typ, want, z):
    half = torch.finfo(TYPES[typ]).eps / 2
    tiny = 2.0 ** -25 if typ == "f16" else 0.0  # half the subnormal spacing
    fn = np.zeros_like(want)
    if act == "gelu":
        fn = np.full_like(want, 3e-7) if typ == "f32" else 0.15 * np.maximum(np.abs(want) * 2.0 ** -10, 2.0 ** -24)
    elif act in ("silu", "gelu_tanh"):
        # the same relative error of the exponential and the reciprocal as on [-12, 12]
        fn = 2e-6 * (1 + np.abs(z))
    return half * (np.abs(want) + fn) + fn + tiny


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("rows,cols", [(1, 1), (7, 4095), (129, 257), (40, 1024)])
def test_act_forward_saves_and_activates(tlg, act, typ, rows, cols):
    g = torch.Generator().manual_seed(rows + cols)
    z = (torch.randn((rows, cols), generator=g) * 3).clamp(-12, 12).to(TYPES[typ])
    codes, scale = mx.quantize(z.double().numpy(), "e4m3")
    want = mx.activate(act, z.double().numpy())
    bound = y_bound(act, typ, want, z.double().numpy())
    for lead, extra in ((0, 0), (1, 3)):
        m, o = Strided(z, lead, extra), Strided(torch.zeros_like(z), lead, extra)
        Y, Q, S = tlg.tlg_act_forward_mx(m.view, act, Y=o.view)
        check_mx(Q, S, codes, scale, "e4m3")
        assert (np.abs(Y.double().cpu().numpy() - want) <= bound).all()
        assert m.guards_kept() and o.guards_kept()
        Y2, Q2, S2 = tlg.tlg_act_forward_mx(m.view, act, Y=m.view)  # in place
        assert torch.equal(bits(Y2), bits(Y)) and torch.equal(Q2, Q)


def saved(z, fill=255):
    codes, scale = mx.quantize(z, "e4m3")
    back = mx.decode(codes, scale, "e4m3")[:, :z.shape[1]]
    return (torch.from_numpy(mx.pack(codes, "e4m3")).cuda(), torch.from_numpy(mx.tile_scales(scale, fill)).cuda(),
            back)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("rows,cols", [(1, 1), (2, 4095), (129, 257), (1000, 515), (300, 1024)])
def test_act_backward_matches_reference(tlg, act, typ, rows, cols):
    rng = np.random.default_rng(rows * 3 + cols)
    Q, S, z = saved(rng.standard_normal((rows, cols)) * 2.5)
    dy = torch.from_numpy(rng.standard_normal((rows, cols))).to(TYPES[typ])
    d64 = dy.double().numpy()
    want = d64 * mx.slope(act, z)
    half = torch.finfo(TYPES[typ]).eps / 2
    fn = np.abs(d64) * (1e-6 + 2.0 ** -23 * np.abs(mx.slope(act, z)))  # the slope, and one fp32 product
    tiny = 2.0 ** -25 if typ == "f16" else 0.0
    bound = half * np.abs(want) * (1 + 1e-5) + fn + tiny
    # the sum: every term's error, and fp32 additions: a column is added in chains of at most
    # rows / 8 + 8 + (splits <= 65535) terms; a bound by the plain chain of `rows` additions covers them
    sum_bound = fn.sum(axis=0) + (rows + 16) * 2.0 ** -24 * np.abs(want).sum(axis=0)
    for lead, extra in ((0, 0), (1, 3)):
        m, o = Strided(dy, lead, extra), Strided(torch.zeros_like(dy), lead, extra)
        dz, db = tlg.tlg_act_backward_mx(m.view, Q, S, act, dZ=o.view)
        assert (np.abs(dz.double().cpu().numpy() - want) <= bound).all()
        assert (np.abs(db.double().cpu().numpy() - want.sum(axis=0)) <= sum_bound).all()
        assert m.guards_kept() and o.guards_kept()
        dz2, none = tlg.tlg_act_backward_mx(m.view, Q, S, act, dZ=m.view, bias_grad=False)  # in place, no sums
        assert none is None and torch.equal(bits(dz2), bits(dz))


def test_act_backward_edges(tlg):
    z = np.zeros((64, 96))
    z[:, 1], z[:, 2], z[:, 3] = 1e30, -1e30, 50
    z[3, 40] = np.nan  # the block of (3, 32..63)
    z[:, 64:] = np.linspace(-200, 200, 32)
    Q, S, back = saved(z)
    dy = torch.ones((64, 96), device="cuda")
    for act in ACTS[1:]:
        dz, _ = tlg.tlg_act_backward_mx(dy, Q, S, act)
        got, want = dz.double().cpu().numpy(), np.nan_to_num(mx.slope(act, np.clip(back, -300, 300)), nan=np.nan)
        assert np.isnan(got[3, 32:64]).all(), act
        got[3, 32:64] = want[3, 32:64] = 0
        assert np.abs(got - want).max() < 1e-6, act
    # an infinite gradient where ReLU is off is dropped
    dz, db = tlg.tlg_act_backward_mx(torch.full((64, 96), float("inf"), device="cuda"), *saved(np.full((64, 96), -1.0))[:2],
                                     "relu")
    assert (dz == 0).all() and (db == 0).all()


def test_zero_sizes(tlg):
    for rows, cols in ((0, 64), (5, 0), (0, 0)):
        X = torch.empty((rows, cols), dtype=torch.float16, device="cuda")
        Q, S = tlg.tlg_mx_quantize(X)
        assert tlg.tlg_mx_dequantize(Q, S, cols).shape == (rows, cols)
        Y, Q, S = tlg.tlg_act_forward_mx(X, "gelu")
        dz, db = tlg.tlg_act_backward_mx(X, Q, S, "gelu", dbias=torch.full((cols,), 3.0, device="cuda"))
        assert dz.shape == (rows, cols) and (db == 0).all()


def test_backward_sums_do_not_depend_on_timing(tlg):
    rng = np.random.default_rng(0)
    Q, S, _ = saved(rng.standard_normal((3000, 700)))
    dy = torch.from_numpy(rng.standard_normal((3000, 700))).cuda().to(torch.bfloat16)
    assert tlg.tlg_act_backward_mx_workspace_size(3000, 700, "bf16") > 0
    first = tlg.tlg_act_backward_mx(dy, Q, S, "silu")[1]
    for _ in range(5):
        assert torch.equal(tlg.tlg_act_backward_mx(dy, Q, S, "silu")[1], first)


def test_streams_and_graphs(tlg):
    z = torch.randn((512, 1500), device="cuda").half()
    dy = torch.randn((512, 1500), device="cuda").half()
    eager = tlg.tlg_act_backward_mx(dy, *tlg.tlg_act_forward_mx(z, "gelu")[1:], "gelu")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        Y, Q, S = tlg.tlg_act_forward_mx(z, "gelu")
        captured = tlg.tlg_act_backward_mx(dy, Q, S, "gelu")
    z2, dy2 = z.clone(), dy.clone()
    z.copy_(torch.randn_like(z)), dy.copy_(torch.randn_like(dy))
    g.replay()
    z.copy_(z2), dy.copy_(dy2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured[0], eager[0]) and torch.equal(captured[1], eager[1])


def test_given_stream(tlg):
    """Outputs and the workspace of a call on a given stream belong to that stream."""
    z = torch.randn((300, 700), device="cuda").half()
    dy = torch.randn((300, 700), device="cuda").half()
    want = tlg.tlg_act_backward_mx(dy, *tlg.tlg_act_forward_mx(z, "silu")[1:], "silu")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        Y, Q, S = tlg.tlg_act_forward_mx(z, "silu", stream=side)
        got = tlg.tlg_act_backward_mx(dy, Q, S, "silu", stream=side.cuda_stream)
        assert torch.cuda.current_stream() != side
        side.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_one_row_of_any_stride(tlg):
    x = torch.randn((3, 4095), device="cuda").half()
    codes, scale = mx.quantize(x[1:2].double().cpu().numpy(), "e4m3")
    wide = torch.zeros((1, 5000), device="cuda").half()
    wide[:, :4095] = x[1]
    for row in (x[1:2], wide[:, :4095], wide[:, :4095].as_strided((1, 4095), (3, 1))):
        Q, S = tlg.tlg_mx_quantize(row, format="e4m3")
        check_mx(Q, S, codes, scale, "e4m3")
        Y, Q, S = tlg.tlg_act_forward_mx(row, "relu")
        check_mx(Q, S, codes, scale, "e4m3")
        assert torch.equal(Y, row.clamp(min=0))


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("cols", [1, 2, 31, 129, 255, 256, 257, 511, 513, 1023, 1025, 2049])
@pytest.mark.parametrize("lead,odd", [(0, 0), (1, 0), (0, 1), (1, 1)])
def test_any_alignment_gives_the_aligned_bits(tlg, typ, cols, lead, odd):
    """Rows that start at any element, and whose neighbours share their words, against the same
    values in 16-byte aligned rows: every element is computed alone, so the bits are the same."""
    rows = 2401 if cols == 1025 else 133  # the many fill the device, and warps take several pieces
    extra = (odd - cols) % 2  # rows an odd or an even number of elements apart, as close as that allows
    x, dy = values(rows, cols, TYPES[typ], cols), values(rows, cols, TYPES[typ], cols + 1)
    flat = [Strided(t, 0, -cols % 8) for t in (x, dy)]
    X, dY = Strided(x, lead, extra), Strided(dy, lead, extra)
    for fmt in ("e2m1", "e4m3"):
        want, got = (tlg.tlg_mx_quantize(t.view, format=fmt) for t in (flat[0], X))
        assert torch.equal(want[0], got[0])
        index = torch.from_numpy(mx.scale_index(rows, -(-want[0].shape[1] // (16 if fmt == "e2m1" else 32) // 4) * 4)).cuda()
        assert torch.equal(want[1][index], got[1][index])
        o = [Strided(torch.zeros_like(x), *at) for at in ((0, -cols % 8), (lead, extra))]
        for t in o:
            tlg.tlg_mx_dequantize(*want, cols, format=fmt, out=typ, X=t.view)
        assert torch.equal(bits(o[0].view), bits(o[1].view)) and o[1].guards_kept()
    y, q, s = tlg.tlg_act_forward_mx(flat[0].view, "silu")
    tlg.tlg_act_forward_mx(X.view, "silu", Y=X.view)  # in place
    assert torch.equal(bits(X.view), bits(y)) and X.guards_kept()
    dz, _ = tlg.tlg_act_backward_mx(flat[1].view, q, s, "silu", bias_grad=False)
    tlg.tlg_act_backward_mx(dY.view, q, s, "silu", dZ=dY.view)
    assert torch.equal(bits(dY.view), bits(dz)) and dY.guards_kept()


def test_calls_on_two_streams_at_once(tlg):
    """Calls that overlap in time, each with a workspace of its own."""
    rng = np.random.default_rng(1)
    Q, S, _ = saved(rng.standard_normal((4096, 2048)))
    dys = [torch.randn((4096, 2048), device="cuda") for _ in range(2)]
    want = [tlg.tlg_act_backward_mx(dy, Q, S, "gelu") for dy in dys]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(4):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(tlg.tlg_act_backward_mx(dys[i], Q, S, "gelu"))
    torch.cuda.synchronize()
    for i in range(2):
        for dz, db in got[i]:
            assert torch.equal(dz, want[i][0]) and torch.equal(db, want[i][1])


def test_workspace_is_checked(tlg):
    dy = torch.ones((3000, 700), device="cuda")
    Q, S, _ = saved(np.zeros((3000, 700)))
    need = tlg.tlg_act_backward_mx_workspace_size(3000, 700, "f32")
    with pytest.raises(tlg.TlgError):
        tlg.tlg_act_backward_mx(dy, Q, S, "gelu", workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")  # its contents do not matter
    dz, db = tlg.tlg_act_backward_mx(dy, Q, S, "gelu", workspace=ws)
    # GELU'(0) = 1/2, computed with an error below 1e-6 (the polynomial's constant is 0.5 - 6e-8); the
    # sum of 3000 of them adds that error 3000 times and rounds at most 3000 times, each time by at
    # most 2^-24 of a partial sum no larger than 1500
    assert ((dz - 0.5).abs() <= 1e-6).all() and (ws[need:] == 0xFF).all()
    assert ((db - 1500).abs() <= 3000 * (1e-6 + 2.0 ** -24 * 1500)).all()


def test_large_row_offsets(tlg):
    # a row stride whose offsets pass 2^31 elements and 2^32 bytes
    ld = (1 << 31) // 4 + 64
    buf = torch.empty((5 * ld,), dtype=torch.float16, device="cuda")
    x = buf.view(5, ld)[:, :100]
    x.copy_(torch.randn((5, 100), device="cuda"))
    codes, scale = mx.quantize(x.double().cpu().numpy(), "e2m1")
    Q, S = tlg.tlg_mx_quantize(x)
    check_mx(Q, S, codes, scale, "e2m1")
    xt = buf.view(5, ld)[:, :100]
    codes, scale = mx.quantize(xt.t().double().cpu().numpy(), "e4m3")
    Q, S = tlg.tlg_mx_quantize(xt, format="e4m3", op="T")
    check_mx(Q, S, codes, scale, "e4m3")
