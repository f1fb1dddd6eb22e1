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
