"""The time limits of the grouped products' waits: the weight gradient clears what a group's last block of rows holds of
the next group, and the warp that does so waits only where a group has such a block.  Whole blocks of a long group in
front of it are not held against that wait; and where a wait does run out, the call reports it and ends, and the next
one is right.

The group in front has 1501 blocks of 64 rows and 14 tiles to a work unit, some 9 ms; the limit is 2 ms, which is
a thousand times what any other wait takes, and what copies that are under way need to land."""

import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

SIZES, WIDTH = [64 * 1501, 5], 8192


@pytest.fixture(scope="module")
def tlg():
    import tiled_dense_gemm_tlg_b200 as t
    assert t.tlg_device_error(clear=True) == (0, 0)
    yield t
    assert t.tlg_device_error(clear=True) == (0, 0)
    torch.cuda.empty_cache()


@pytest.fixture
def limit(tlg):
    set_limit = tlg.raw_library().tlg_internal_grouped_wait_limit
    set_limit.argtypes, set_limit.restype = [ctypes.c_uint64, ctypes.c_uint64], None
    yield set_limit
    set_limit(0, 0)


@pytest.fixture(scope="module")
def operands():
    gen = torch.Generator(device="cuda").manual_seed(1)
    A, dC = (torch.randn((sum(SIZES), WIDTH), generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    off = torch.tensor([0, SIZES[0], sum(SIZES)], dtype=torch.int32, device="cuda")
    return A, dC, off


def check(dB, A, dC):
    """The last group whole, some columns of the first: products are exact, a step of the truncating sum of 16 of them
    loses at most five units of 2^-23 of a span's magnitudes so far, and half a unit of a bf16 value."""
    for got, a, d in ((dB[1], A[-SIZES[1]:], dC[-SIZES[1]:]), (dB[0, 4000:4100, 8000:], A[:SIZES[0], 4000:4100], dC[:SIZES[0], 8000:])):
        a, d = a.double(), d.double()
        want, size = a.t() @ d, a.t().abs() @ d.abs()
        bound = (5 * 65 * 2.0 ** -23 + a.shape[0] / 1024 * 2.0 ** -24) * size + 2.0 ** -8 * want.abs() + 1e-30
        assert ((got.double() - want).abs() <= bound).all()


def test_whole_blocks_in_front_of_a_tail(tlg, limit, operands):
    A, dC, off = operands
    limit(2000000, 20000)  # and as much for a k-block as ever
    dB = tlg.tlg_gemm_grouped_dw(A, dC, off)
    assert tlg.tlg_device_error(clear=True) == (0, 0)
    check(dB, A, dC)


def test_a_wait_that_runs_out(tlg, limit, operands):
    A, dC, off = operands
    limit(2000000, 0)
    tlg.tlg_gemm_grouped_dw(A, dC, off)
    rc, code = tlg.tlg_device_error(clear=True)
    assert rc == tlg.TLG_ERR_TIMEOUT and code & 1 and code & (1 << 8), hex(code)
    assert tlg.tlg_device_error(clear=True) == (0, 0)
    limit(0, 0)
    dB = tlg.tlg_gemm_grouped_dw(A, dC, off)
    assert tlg.tlg_device_error(clear=True) == (0, 0)
    check(dB, A, dC)
    C = tlg.tlg_gemm_grouped(dC[-64:], dB, torch.tensor([0, 30, 64], dtype=torch.int32, device="cuda"), op_b="T")
    assert torch.isfinite(C).all() and tlg.tlg_device_error(clear=True) == (0, 0)
