"""How kernels of the library follow one another on a stream, read from the edges of a captured graph on a B200 (nothing of it is run): no
elementwise kernel that stands behind a GEMM and in front of a CTA-pair GEMM is launched early (as a programmatic dependent)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

N = pytest.importorskip("mixture_experts_ffn_11_b200._native")


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def launched_early(calls):
    """For each kernel behind the first of what calls() launches on one stream: whether it is a programmatic dependent of the one before."""
    driver = pytest.importorskip("cuda.bindings.driver")
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        calls()
    raw = driver.CUgraph(graph.raw_cuda_graph())
    err, *_, n = driver.cuGraphGetEdges_v2(raw)
    assert err == driver.CUresult.CUDA_SUCCESS
    err, first, second, data, _ = driver.cuGraphGetEdges_v2(raw, n)
    assert err == driver.CUresult.CUDA_SUCCESS
    follows = {int(a): (int(b), e.type) for a, b, e in zip(first, second, data)}
    assert len(follows) == n  # a chain
    at = (set(follows) - {b for b, _ in follows.values()}).pop()
    early = []
    while at in follows:
        at, kind = follows[at]
        early.append(kind == driver.CUgraphDependencyType.CU_GRAPH_DEPENDENCY_TYPE_PROGRAMMATIC.value)
    return early


def test_the_encoder_between_the_fp8_products():
    M, G, d, f = 40, 2, 128, 256
    new = lambda *s, t=N.E4M3: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    f32, bf = torch.float32, torch.bfloat16
    off = torch.tensor([0, 30, M], dtype=torch.int32, device="cuda")
    src = torch.arange(M, dtype=torch.int32, device="cuda")
    x, xq, xs, h, hq, hs = new(M, d, t=bf), new(M, d), new(1, M, t=f32), new(M, f, t=bf), new(M, f), new(2, M, t=f32)
    wg, sg, wd, sd, y = new(G, 2 * f, d), new(G, 2, 2, 1, t=f32), new(G, d, f), new(G, 1, 2, t=f32), new(M, d, t=bf)

    def products():
        N.fp8_row_quantize(x, src, xq, xs)
        N.grouped_gemm_gateup_fp8(xq, xs, wg, sg, off, h)
        N.fp8_row_quantize(h, None, hq, hs)
        N.grouped_gemm_down_fp8(hq, hs, wd, sd, off, y)

    early = launched_early(lambda: (products(), products()))
    assert early[1::2] == [False] * 3  # the encoders
    assert early[2::2] == [True] * 3   # the products behind them


def test_the_weight_encoder_between_the_fp8_products():
    M, G, d = 40, 2, 128
    new = lambda *s, t=N.E4M3: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    f32, bf = torch.float32, torch.bfloat16
    off = torch.tensor([0, 30, M], dtype=torch.int32, device="cuda")
    w, wq, ws, xq, xs, y = new(G, d, d, t=bf), new(G, d, d), new(G, 1, 1, t=f32), new(M, d), new(1, M, t=f32), new(M, d, t=bf)

    def product():
        N.fp8_block_quantize(w, wq, ws)
        N.grouped_gemm_down_fp8(xq, xs, wq, ws, off, y)

    early = launched_early(lambda: (product(), product(), product()))
    assert early[1::2] == [False] * 2
    assert early[2::2] == [True] * 2
