"""Grouped products with more tiles to a work unit than are worked out in advance (64): every role then finds the others
by itself.  Ragged and empty groups, a few long and most short, and every group is looked at.

References in 64 bits on the GPU.  Tolerances: products of two 16-bit values are exact in fp32, a step of the truncating
sum of 16 of them loses at most five units of 2^-23 of the magnitudes added so far, so a sum of K terms at most
5 (K / 16 + 1) 2^-23 times the sum of magnitudes; the stored type adds half a unit."""

import pytest
import torch

pytestmark = pytest.mark.gpu

LISTED = 64


@pytest.fixture(scope="module")
def tlg():
    import tiled_dense_gemm_tlg_b200 as t
    yield t
    assert t.tlg_device_error(clear=True) == (0, 0)
    torch.cuda.empty_cache()


def offsets_of(sizes):
    return torch.tensor([0, *torch.tensor(sizes).cumsum(0).tolist()], dtype=torch.int32, device="cuda")


def normal(seed, shape, dtype):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def check(got, left, right):
    want, size = left.double() @ right.double(), left.double().abs() @ right.double().abs()
    fi = torch.finfo(got.dtype)
    bound = 5 * (left.shape[1] / 16 + 1) * 2.0 ** -23 * size + want.abs() * fi.eps / 2 + fi.tiny * fi.eps
    bad = (got.double() - want).abs() > bound
    assert torch.isfinite(got).all() and not bad.any(), (bad.nonzero()[:4], got[bad][:4], want[bad][:4])


def units(pair_or_per_sm):
    """Work units at most: pairs of SMs, or CTAs to an SM."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return sms // 2 if pair_or_per_sm == "pair" else sms * pair_or_per_sm


def tiles_of(sizes, rows, lanes, n):
    return sum(-(-s // rows) for s in sizes) * -(-n // lanes)


# rows of the groups, k, n, tile rows and columns, units: the pairs, the small tiles, the plain loads
FORWARD = {"pairs": ([400, 0, 31, 700, 1, 256, 257, 650], 64, 102440, 256, 256, "pair"),
           "small": ([(7 * g) % 4 for g in range(1023)] + [70], 64, 5000, 64, 128, 2),
           "plain": ([130, 0, 3, 65, 300, 1, 128, 129, 64], 63, 110001, 128, 128, 1)}


@pytest.mark.parametrize("name", list(FORWARD))
def test_forward(tlg, name):
    """B_g is a window of one matrix, g rows further down, so that a wrong group shows."""
    sizes, k, n, rows, lanes, per = FORWARD[name]
    assert tiles_of(sizes, rows, lanes, n) > (LISTED + 1) * units(per)
    groups = len(sizes)
    A, W = normal(1, (sum(sizes), k), torch.bfloat16), normal(2, (n + groups, k), torch.bfloat16)
    B = W.as_strided((groups, n, k), (k, k, 1))
    got = tlg.tlg_gemm_grouped(A, B, offsets_of(sizes), op_b="T")
    r = 0
    for g, s in enumerate(sizes):
        if s:
            check(got[r:r + s], A[r:r + s], B[g].t())
        r += s


# of all groups: columns of A and dC, and the tile
GRADIENT = {"pairs": (296, 616, 256, "pair"), "plain": (129, 643, 128, 1)}


@pytest.mark.parametrize("op_b", ["N", "T"])
@pytest.mark.parametrize("name", list(GRADIENT))
def test_weight_gradient(tlg, name, op_b):
    k, n, tile, per = GRADIENT[name]
    sizes = [0] * 1024
    for g in (0, 1, 5, 300, 301, 302, 640, 641, 900, 1022, 1023):
        sizes[g] = 1 + (37 * g) % 200
    sizes[302], sizes[900] = 64, 128
    assert len(sizes) * -(-k // tile) * -(-n // tile) > (LISTED + 1) * units(per)
    A, dC = normal(3, (sum(sizes), k), torch.float16), normal(4, (sum(sizes), n), torch.float16)
    got = tlg.tlg_gemm_grouped_dw(A, dC, offsets_of(sizes), op_b=op_b)
    r = 0
    for g, s in enumerate(sizes):
        if s:
            left, right = (A, dC) if op_b == "N" else (dC, A)
            check(got[g], left[r:r + s].t(), right[r:r + s])
        r += s
    empty = torch.tensor([g for g, s in enumerate(sizes) if s == 0], device="cuda")
    assert (got[empty] == 0).all()
