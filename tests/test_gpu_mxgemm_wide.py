"""tlg_gemm_mxfp4 where a row of C passes 2^31 bytes: offsets inside a row need more than 32 bits."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tlg():
    import tiled_dense_gemm_tlg_b200 as t
    yield t
    rc, code = t.tlg_device_error()
    assert rc == 0, hex(code)


@pytest.mark.parametrize("inplace", [False, True])
def test_residual_of_rows_beyond_2_gib(tlg, inplace):
    """Every element of A and B is 1 and K is one block, so C = 32 + residual, exactly; the first
    columns have 2^31 bytes of residual and more behind them."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB of free device memory")
    N = (1 << 29) + 4096
    A = torch.full((1, 16), 0x22, dtype=torch.uint8, device="cuda")
    SA = torch.full((512,), 127, dtype=torch.uint8, device="cuda")
    B = torch.full((N, 16), 0x22, dtype=torch.uint8, device="cuda")
    SB = torch.full((N // 128 * 512,), 127, dtype=torch.uint8, device="cuda")
    R = torch.randint(0, 1000, (1, N), device="cuda", dtype=torch.float32)
    want = R + 32
    C = tlg.tlg_gemm_mxfp4(A, SA, B, SB, residual=R, C=R if inplace else None, out="f32",
                           config={"cta_group": 1, "block_n": 128})
    assert torch.equal(C, want)


@pytest.mark.parametrize("typ", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("M,config", [(20, None), (70, {"cta_group": 1, "block_n": 64}), (300, {"cta_group": 2, "block_n": 256})])
def test_strides_whose_offsets_pass_32_bits(tlg, typ, odd, M, config):
    """C and the residual in rows so far apart that the last rows' elements lie past 2^31 elements and
    2^32 bytes, written by TMA or, where rows are not aligned, by plain stores."""
    if torch.cuda.mem_get_info()[0] < 32 << 30:
        pytest.skip("needs 32 GiB of free device memory")
    N, K = 100, 320
    g = torch.Generator(device="cuda").manual_seed(M)
    A, B = (torch.randint(0, 256, (rows, K // 2), generator=g, device="cuda", dtype=torch.uint8) for rows in (M, N))
    S = torch.full((-(-max(M, N) // 128) * 3 * 512,), 127, dtype=torch.uint8, device="cuda")
    a, b = (tlg.tlg_mx_dequantize(q, S, K, out="f32").double() for q in (A, B))
    ld = ((1 << 31) // (M - 1) + 64) // 8 * 8 + odd
    buf = torch.empty((M * ld,), dtype=typ, device="cuda")
    C = buf.view(M, ld)[:, :N]
    C.copy_(torch.randint(-64, 65, (M, N), generator=g, device="cuda"))
    want = (a @ b.T + C.double()).to(typ)  # multiples of 1/4 below 2^20: one rounding
    out = "f32" if typ == torch.float32 else "bf16"
    tlg.tlg_gemm_mxfp4(A, S, B, S, residual=C, C=C, out=out, config=config)
    assert torch.equal(C, want)
