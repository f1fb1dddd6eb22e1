"""tlg_choose_config_mxfp4 answers what tlg_gemm_mxfp4 runs: the captured call's kernel, grid and
shared memory are those of a call that is given the answer."""

import pytest
import torch

pytestmark = pytest.mark.gpu

SIZES = [(4096, 4096, 1024), (1, 4096, 4096), (16, 1024, 512), (32, 300, 2000), (33, 300, 2000), (200, 700, 96), (512, 2048, 512),
         (700, 700, 700), (2048, 2048, 2048), (1000, 5000, 4096), (2000, 1000, 256)]


@pytest.fixture(scope="module")
def tlg():
    import tiled_dense_gemm_tlg_b200 as t
    return t


def launch_of(call):
    """(kernel, grid, shared memory) of the one kernel that `call` launches."""
    from cuda.bindings import driver as cu

    call()  # the kernel's attributes are set
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    raw = cu.CUgraph(init_value=graph.raw_cuda_graph())
    err, nodes, count = cu.cuGraphGetNodes(raw, 8)
    assert err == 0 and count == 1
    err, p = cu.cuGraphKernelNodeGetParams(nodes[0])
    assert err == 0
    return (int(p.func), int(p.kern)), (p.gridDimX, p.gridDimY, p.gridDimZ), p.sharedMemBytes


def product(tlg, M, N, K, typ, epilogue):
    blocks = -(-K // 32)
    mx = lambda rows: (torch.zeros((rows, blocks * 16), dtype=torch.uint8, device="cuda"),
                       torch.zeros(-(-rows // 128) * -(-blocks // 4) * 512, dtype=torch.uint8, device="cuda"))
    A, B = mx(M), mx(N)
    C = torch.empty((M, N), dtype={"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[typ], device="cuda")
    more = {"residual": torch.zeros_like(C), "activation": "gelu"} if epilogue else {}
    return lambda config=None: tlg.tlg_gemm_mxfp4(*A, *B, C=C, out=typ, config=config, **more)


@pytest.mark.parametrize("M,N,K", SIZES)
def test_the_answer_is_what_runs(tlg, M, N, K):
    for typ in ("f16", "f32"):
        call = product(tlg, M, N, K, typ, False)
        answer = tlg.tlg_choose_config_mxfp4(M, N, K, typ)
        assert launch_of(call) == launch_of(lambda: call(answer))
        assert launch_of(call)[1][0] == answer["max_ctas"]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_the_answer_with_an_epilogue_is_what_runs(tlg, M, N, K):
    for typ in ("f16", "bf16"):
        call = product(tlg, M, N, K, typ, True)
        answer = tlg.tlg_choose_config_mxfp4_fused(M, N, K, activation="gelu", residual=True, out=typ)
        assert launch_of(call) == launch_of(lambda: call(answer))
        assert launch_of(call)[1][0] == answer["max_ctas"]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_the_answer_resolves_to_itself(tlg, M, N, K):
    for typ in ("f32", "bf16"):
        answer = tlg.tlg_choose_config_mxfp4(M, N, K, typ)
        assert tlg.tlg_choose_config_mxfp4(M, N, K, typ, request=answer) == answer
        assert tlg.tlg_choose_config_mxfp4_fused(M, N, K, out=typ) == answer  # an epilogue of nothing
        answer = tlg.tlg_choose_config_mxfp4_fused(M, N, K, bias=True, out=typ)
        assert tlg.tlg_choose_config_mxfp4_fused(M, N, K, bias=True, out=typ, request=answer) == answer


def test_requests_of_the_few_row_kernel(tlg):
    """Its own fields are accepted where they describe it, and refused where they do not."""
    answer = tlg.tlg_choose_config_mxfp4(16, 4096, 4096)
    assert answer["block_n"] == 16 and answer["cta_group"] == 1
    for field, value in (("cta_group", 2), ("stages", 3), ("max_ctas", answer["max_ctas"] - 1), ("block_n", 32),
                         ("k_split", 16), ("k_split", 3)):
        with pytest.raises(tlg.TlgError):
            tlg.tlg_choose_config_mxfp4(16, 4096, 4096, request={**answer, field: value})
    with pytest.raises(tlg.TlgError):  # a tile's name for 33 rows, or the few-row kernel's
        tlg.tlg_choose_config_mxfp4(33, 4096, 4096, request=answer)
    # without its block_n these fields ask for a tile, as before
    for request in ({"cta_group": 1}, {"max_ctas": 10}, {"stages": 5}):
        assert tlg.tlg_choose_config_mxfp4(16, 4096, 4096, request=request)["block_n"] >= 64
