"""GPU tests of the products grouped by expert and their gradients against plain 64-bit products.

Tolerances: operands are exact in 64 bits, every product of two 16-bit values is exact in fp32, and a
sum of K terms accumulated in fp32 is off by at most K 2^-23 times the sum of the terms' magnitudes (a
truncating adder's step is twice a rounding one's; the order does not matter), so the bound is
computed per element from the magnitudes.  The stored type adds half a unit, eps / 2 relative, and the activation
its stated error."""

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ACTS = ["none", "relu", "gelu", "silu", "gelu_tanh"]
SIZES = [[1], [5, 0, 130], [0, 0, 64, 1, 63], [257, 16, 0, 700], [33] * 40]


@pytest.fixture(scope="module")
def tlg():
    import tiled_dense_gemm_tlg_b200 as t
    yield t
    assert t.tlg_device_error(clear=True) == (0, 0)


def offsets_of(sizes, first=0):
    return torch.tensor([first] + [first + sum(sizes[:i + 1]) for i in range(len(sizes))], dtype=torch.int32)


class Strided:
    """A matrix or a stack of them inside a larger buffer of NaNs: `lead` elements in front, `extra` behind
    each row."""

    def __init__(self, host, lead=0, extra=0):
        rows, cols = host.shape[-2:]
        mats = host.shape[0] if host.dim() == 3 else 1
        self.buf = torch.full((lead + mats * (rows + 1) * (cols + extra) + 64,), float("nan"), device="cuda").to(host.dtype)
        stack = self.buf[lead:lead + mats * (rows + 1) * (cols + extra)].view(mats, rows + 1, cols + extra)[:, :rows, :cols]
        stack.copy_(host.view(mats, rows, cols))
        self.view = stack if host.dim() == 3 else stack[0]
        mask = torch.ones(self.buf.shape, dtype=torch.bool, device="cuda")
        mask[lead:lead + mats * (rows + 1) * (cols + extra)].view(mats, rows + 1, cols + extra)[:, :rows, :cols] = False
        self.mask = mask
        self.before = self.buf.clone()

    def guards_kept(self):
        kind = torch.int32 if self.buf.dtype == torch.float32 else torch.int16
        return torch.equal(self.buf.view(kind)[self.mask], self.before.view(kind)[self.mask])


def activate(act, x):
    if act == "relu":
        return x.clamp(min=0)
    if act == "gelu":
        return x * torch.special.ndtr(x)
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu_tanh":
        return x * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (x + 0.044715 * x ** 3))
    return x


def forward(A, B, sizes, first, op_b, act):
    """(C, the error bound before it is stored) in 64 bits."""
    A, B = A.double(), B.double()
    C = torch.full((A.shape[0], B.shape[2 if op_b == "N" else 1]), float("nan"), dtype=torch.float64)
    E = torch.zeros_like(C)
    r = first
    for g, s in enumerate(sizes):
        b = B[g] if op_b == "N" else B[g].t()
        z = A[r:r + s] @ b
        C[r:r + s] = activate(act, z)
        E[r:r + s] = A.shape[1] * 2.0 ** -23 * (A[r:r + s].abs() @ b.abs())
        r += s
    if act != "none":
        E = E * 1.13 + 2.0 ** -18 * (1 + C.abs())  # the steepest slope, and the fp32 function's own error
    return C, E


def check(got, want, bound, dtype):
    got = got.double().cpu()
    bound = bound + want.abs() * torch.finfo(dtype).eps / 2 + torch.finfo(dtype).tiny * torch.finfo(dtype).eps
    bad = (got - want).abs() > bound
    assert torch.isfinite(got).all() and not bad.any(), (bad.nonzero()[:4], (got - want).abs()[bad][:4], bound[bad][:4])


def operands(seed, rows, k, n, groups, op_b, dtype):
    g = torch.Generator().manual_seed(seed)
    A = torch.randn((rows, k), generator=g).to(dtype)
    B = (torch.randn((groups, k, n) if op_b == "N" else (groups, n, k), generator=g) / max(k, 1) ** 0.5).to(dtype)
    return A, B


@pytest.mark.parametrize("typ,out", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("op_b", ["N", "T"])
@pytest.mark.parametrize("k,n", [(64, 128), (200, 72), (136, 520)])
@pytest.mark.parametrize("sizes", SIZES)
def test_forward(tlg, sizes, k, n, op_b, typ, out):
    A, B = operands(1, sum(sizes), k, n, len(sizes), op_b, TYPES[typ])
    want, err = forward(A, B, sizes, 0, op_b, "none")
    a, b = Strided(A, 8, 8), Strided(B, 16, 8)
    c = Strided(torch.zeros((sum(sizes), n), dtype=TYPES[out]), 4, 4)
    got = tlg.tlg_gemm_grouped(a.view, b.view, offsets_of(sizes).cuda(), op_b=op_b, C=c.view, out=out)
    check(got, want, err, TYPES[out])
    assert c.guards_kept()


@pytest.mark.parametrize("op_b", ["N", "T"])
@pytest.mark.parametrize("lead,extra", [(0, 0), (1, 1), (3, 2), (0, 1)])
@pytest.mark.parametrize("sizes", [[3, 0, 40], [200, 130]])
def test_forward_any_alignment(tlg, sizes, lead, extra, op_b):
    k, n = 77, 131
    A, B = operands(2, sum(sizes), k, n, len(sizes), op_b, torch.bfloat16)
    want, err = forward(A, B, sizes, 0, op_b, "none")
    a, b = Strided(A, lead, extra), Strided(B, lead, extra)
    c = Strided(torch.zeros((sum(sizes), n), dtype=torch.bfloat16), lead, extra)
    tlg.tlg_gemm_grouped(a.view, b.view, offsets_of(sizes).cuda(), op_b=op_b, C=c.view)
    check(c.view, want, err, torch.bfloat16)
    assert c.guards_kept()


@pytest.mark.parametrize("op_b", ["N", "T"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("sizes,k,n", [([1], 4096, 96), ([0, 1, 0], 2056, 300), ([3, 0, 2], 1088, 1000), ([20, 45, 0], 600, 130),
                                       ([1, 1], 520, 4000), ([64, 65], 4000, 200)])
def test_forward_few_rows_and_long_sums(tlg, sizes, k, n, out, op_b):
    """Few tiles, whose sums several CTAs share."""
    A, B = operands(16, sum(sizes), k, n, len(sizes), op_b, torch.bfloat16)
    want, err = forward(A, B, sizes, 0, op_b, "silu")
    c = Strided(torch.zeros((sum(sizes), n), dtype=TYPES[out]), 4, 4)
    tlg.tlg_gemm_grouped(A.cuda(), B.cuda(), offsets_of(sizes).cuda(), op_b=op_b, activation="silu", C=c.view, out=out)
    check(c.view, want, err, TYPES[out])
    assert c.guards_kept()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("typ,out", [("f16", "f16"), ("bf16", "f32"), ("bf16", "bf16")])
def test_forward_activation(tlg, act, typ, out):
    sizes = [70, 300]
    A, B = operands(3, 370, 256, 200, 2, "N", TYPES[typ])
    want, err = forward(A, B, sizes, 0, "N", act)
    got = tlg.tlg_gemm_grouped(A.cuda(), B.cuda(), offsets_of(sizes).cuda(), activation=act, out=out)
    if act == "gelu" and out != "f32":
        err = err + 0.15 * torch.finfo(TYPES["f16"]).eps * want.abs()  # the 16-bit form's stated error
    check(got, want, err, TYPES[out])


@pytest.mark.parametrize("sizes,first,behind", [([40, 0, 25], 7, 9), ([0, 0], 3, 2), ([300], 0, 50)])
def test_rows_outside_the_groups_stay(tlg, sizes, first, behind):
    rows = first + sum(sizes) + behind
    A, B = operands(4, rows, 96, 160, len(sizes), "T", torch.float16)
    A[:first] = float("nan")
    A[rows - behind:] = float("inf")
    C = torch.full((rows, 160), -7.0, dtype=torch.float16, device="cuda")
    tlg.tlg_gemm_grouped(A.cuda(), B.cuda(), offsets_of(sizes, first).cuda(), op_b="T", C=C)
    want, err = forward(A, B, sizes, first, "T", "none")
    inside = slice(first, rows - behind)
    check(C[inside], want[inside], err[inside], torch.float16)
    assert (C[:first] == -7).all() and (C[rows - behind:] == -7).all()


@pytest.mark.parametrize("op_b", ["N", "T"])
@pytest.mark.parametrize("sizes", [[70, 1, 130], [3, 5]])
def test_other_groups_nan_and_infinity_stay_apart(tlg, sizes, op_b):
    """Weights and rows of another group, k past K included, never reach a group's products."""
    k, n = 72, 96
    A, B = operands(5, sum(sizes), k, n, len(sizes), op_b, torch.bfloat16)
    want, err = forward(A, B, sizes, 0, op_b, "none")
    A2, B2 = A.clone(), B.clone()
    A2[:sizes[0]] = float("inf")
    B2[0] = float("nan")
    got = tlg.tlg_gemm_grouped(A2.cuda(), B2.cuda(), offsets_of(sizes).cuda(), op_b=op_b)
    check(got[sizes[0]:], want[sizes[0]:], err[sizes[0]:], torch.bfloat16)


def test_one_matrix_for_all_groups(tlg):
    sizes = [20, 90, 3]
    A, B = operands(6, 113, 64, 136, 1, "N", torch.float16)
    want, err = forward(A, B.expand(3, -1, -1), sizes, 0, "N", "none")
    got = tlg.tlg_gemm_grouped(A.cuda(), B.cuda().expand(3, -1, -1), offsets_of(sizes).cuda())
    check(got, want, err, torch.float16)


@pytest.mark.parametrize("offsets", [[0, 50, 30, 64], [-5, 10, 64, 1 << 30], [64, 0, 0, 0], [70, 80, 90, 100],
                                     [9, 3, 20, 15], [-(1 << 31), 1, (1 << 31) - 1, 7]])
@pytest.mark.parametrize("many", [False, True])
def test_bad_offsets_stay_inside(tlg, offsets, many):
    """Values outside [0, rows] are held to it, and one less than an earlier one counts as that one; also where the
    groups are so many that several warps look at them."""
    rows, k, n = 64, 64, 128
    if many:
        offsets = offsets[:2] * 40 + offsets[2:] + [o - 1 for o in offsets[2:]] * 20
        offsets = [max(o, -(1 << 31)) for o in offsets]
    groups = len(offsets) - 1
    A, B = operands(7, rows, k, n, groups, "N", torch.float16)
    c = Strided(torch.full((rows, n), -7.0, dtype=torch.float16))
    tlg.tlg_gemm_grouped(A.cuda(), B.cuda(), torch.tensor(offsets, dtype=torch.int32).cuda(), C=c.view)
    assert c.guards_kept()
    held = []
    for o in offsets:
        held.append(max(min(max(o, 0), rows), held[-1] if held else 0))
    sizes = [b - a for a, b in zip(held, held[1:])]
    want, err = forward(A, B, sizes, held[0], "N", "none")
    check(c.view[held[0]:held[-1]], want[held[0]:held[-1]], err[held[0]:held[-1]], torch.float16)
    got = c.view.cpu()
    assert (got[:held[0]] == -7).all() and (got[held[-1]:] == -7).all()
    dB = tlg.tlg_gemm_grouped_dw(A.cuda(), A.cuda(), torch.tensor(offsets, dtype=torch.int32).cuda(), out="f32")
    want, err = backward(A, A, sizes, held[0], "N")
    check(dB, want, err, torch.float32)


def test_many_groups(tlg):
    """As many groups as there may be, most of them empty."""
    groups = 1024
    sizes = [(7 * g) % 3 if g % 5 == 0 else 0 for g in range(groups)]
    A, B = operands(8, sum(sizes), 64, 64, groups, "N", torch.float16)
    want, err = forward(A, B, sizes, 0, "N", "none")
    got = tlg.tlg_gemm_grouped(A.cuda(), B.cuda(), offsets_of(sizes).cuda())
    check(got, want, err, torch.float16)
    dB = tlg.tlg_gemm_grouped_dw(A.cuda(), got, offsets_of(sizes).cuda(), out="f32")
    want, err = backward(A, got.cpu(), sizes, 0, "N")
    check(dB, want, err, torch.float32)


def test_empty(tlg):
    A, B = operands(9, 10, 0, 32, 2, "N", torch.float16)
    off = offsets_of([4, 5]).cuda()
    C = torch.full((10, 32), 3.0, dtype=torch.float16, device="cuda")
    tlg.tlg_gemm_grouped(A.cuda(), B.cuda(), off, C=C)
    assert (C[:9] == 0).all() and (C[9:] == 3).all()
    none = torch.zeros((0, 16), dtype=torch.float16, device="cuda")
    assert tlg.tlg_gemm_grouped(none, torch.zeros((2, 16, 8), dtype=torch.float16, device="cuda"), off).shape == (0, 8)
    dB = tlg.tlg_gemm_grouped_dw(none, torch.zeros((0, 24), dtype=torch.float16, device="cuda"), off)
    assert dB.shape == (2, 16, 24) and (dB == 0).all()
    assert tlg.tlg_gemm_grouped(none, none.new_zeros((0, 16, 8)), offsets_of([]).cuda()).shape == (0, 8)


# ------------------------------------------------------------------ weight gradient


def backward(A, dC, sizes, first, op_b):
    A, dC = A.double(), dC.double()
    W, E = [], []
    r = first
    for s in sizes:
        left, right = (A[r:r + s], dC[r:r + s]) if op_b == "N" else (dC[r:r + s], A[r:r + s])
        W.append(left.t() @ right)
        E.append(s * 2.0 ** -23 * (left.abs().t() @ right.abs()))
        r += s
    return torch.stack(W), torch.stack(E)


@pytest.mark.parametrize("typ,out", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("op_b", ["N", "T"])
@pytest.mark.parametrize("k,n", [(64, 128), (200, 72), (136, 520)])
@pytest.mark.parametrize("sizes", SIZES)
def test_weight_gradient(tlg, sizes, k, n, op_b, typ, out):
    g = torch.Generator().manual_seed(10)
    first, behind = 3, 5
    rows = first + sum(sizes) + behind
    A, dC = (torch.randn((rows, c), generator=g).to(TYPES[typ]) for c in (k, n))
    want, err = backward(A, dC, sizes, first, op_b)
    A[:first], dC[first + sum(sizes):] = float("nan"), float("inf")
    a, d = Strided(A, 8, 8), Strided(dC, 16, 8)
    b = Strided(torch.zeros(want.shape, dtype=TYPES[out]), 4, 4)
    got = tlg.tlg_gemm_grouped_dw(a.view, d.view, offsets_of(sizes, first).cuda(), op_b=op_b, dB=b.view, out=out)
    check(got, want, err, TYPES[out])
    assert b.guards_kept()


@pytest.mark.parametrize("op_b", ["N", "T"])
@pytest.mark.parametrize("lead,extra", [(1, 1), (3, 2), (0, 1)])
def test_weight_gradient_any_alignment(tlg, lead, extra, op_b):
    sizes, k, n = [70, 0, 65], 77, 131
    g = torch.Generator().manual_seed(11)
    A, dC = (torch.randn((135, c), generator=g).to(torch.float16) for c in (k, n))
    want, err = backward(A, dC, sizes, 0, op_b)
    a, d = Strided(A, lead, extra), Strided(dC, lead, extra)
    b = Strided(torch.zeros(want.shape, dtype=torch.float16), lead, extra)
    tlg.tlg_gemm_grouped_dw(a.view, d.view, offsets_of(sizes).cuda(), op_b=op_b, dB=b.view)
    check(b.view, want, err, torch.float16)
    assert b.guards_kept()


def test_weight_gradient_keeps_groups_apart(tlg):
    """A group whose rows are all infinite or NaN, and its neighbours, whose last blocks of rows hold its first."""
    sizes, k, n = [100, 37, 91], 136, 264
    g = torch.Generator().manual_seed(12)
    A, dC = (torch.randn((228, c), generator=g).to(torch.bfloat16) for c in (k, n))
    want, err = backward(A, dC, sizes, 0, "N")
    A[100:137], dC[100:137] = float("inf"), float("nan")
    got = tlg.tlg_gemm_grouped_dw(A.cuda(), dC.cuda(), offsets_of(sizes).cuda(), out="f32")
    check(got[0], want[0], err[0], torch.float32)
    check(got[2], want[2], err[2], torch.float32)


def test_gradients_against_differences(tlg):
    """The input and weight gradients of sum(C * G) against central differences of the product in 64 bits."""
    sizes, k, n = [9, 0, 14], 24, 40
    A, B = operands(13, 23, k, n, 3, "T", torch.float16)
    G = torch.randn((23, n), generator=torch.Generator().manual_seed(14)).half()
    off = offsets_of(sizes).cuda()
    dA = tlg.tlg_gemm_grouped(G.cuda(), B.cuda(), off, op_b="N", out="f32").double().cpu()
    dB = tlg.tlg_gemm_grouped_dw(A.cuda(), G.cuda(), off, op_b="T", out="f32").double().cpu()

    def value(a, b):
        return (forward(a, b, sizes, 0, "T", "none")[0] * G.double()).sum()

    a, b, h = A.double(), B.double(), 1e-3
    for x, d, at in ((a, dA, (0, 3)), (a, dA, (22, 23)), (a, dA, (10, 0)), (b, dB, (0, 39, 23)), (b, dB, (2, 0, 5)), (b, dB, (1, 2, 2))):
        old = x[at].item()
        x[at] = old + h
        up = value(a, b)
        x[at] = old - h
        down = value(a, b)
        x[at] = old
        assert abs((up - down) / (2 * h) - d[at]) < 1e-4  # the product is linear in each element


def test_streams_and_graphs(tlg):
    """On a stream of its own, two at once, and captured and replayed with new offsets."""
    sizes, k, n = [100, 28], 128, 256
    A, B = operands(15, 128, k, n, 2, "N", torch.float16)
    a, b, off = A.cuda(), B.cuda(), offsets_of(sizes).cuda()
    C1, C2 = (torch.zeros((128, n), dtype=torch.float16, device="cuda") for _ in range(2))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        tlg.tlg_gemm_grouped(a, b, off, C=C1, stream=s1)
        tlg.tlg_gemm_grouped(a, b, off, C=C2, stream=s2)
    torch.cuda.synchronize()
    want, err = forward(A, B, sizes, 0, "N", "none")
    check(C1, want, err, torch.float16)
    assert torch.equal(C1, C2)
    dB = torch.zeros((2, k, n), dtype=torch.float32, device="cuda")
    tlg.tlg_gemm_grouped_dw(a, C1, off, dB=dB, out="f32")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tlg.tlg_gemm_grouped(a, b, off, C=C1)
        tlg.tlg_gemm_grouped_dw(a, C1, off, dB=dB, out="f32")
    for sizes in ([3, 125], [128, 0], [60, 68]):
        off.copy_(offsets_of(sizes))
        graph.replay()
        want, err = forward(A, B, sizes, 0, "N", "none")
        check(C1, want, err, torch.float16)
        want, err = backward(A, C1.cpu(), sizes, 0, "N")
        check(dB, want, err, torch.float32)
