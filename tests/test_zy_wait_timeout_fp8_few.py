"""The failure path of the e4m3 grouped GEMMs and of the few-token layer's grid barrier on a B200: a wait that nothing ends (the
test hook moe_test_set_wait, 1 ms) must end the kernel with MOE_DEVERR_WAIT_TIMEOUT, and the next call must be right."""
import pytest
import torch

pytestmark = pytest.mark.gpu

N = pytest.importorskip("mixture_experts_ffn_11_b200._native")


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    N.get_device_error()
    yield
    N.test_set_wait(0, False)


def stalled_then_right(call, out):
    call()
    want = out.clone()
    assert N.get_device_error() == 0
    N.test_set_wait(1_000_000, stall=True)
    try:
        call()  # returns: its waits give up after 1 ms
        err = N.get_device_error()  # synchronises
    finally:
        N.test_set_wait(0, stall=False)
    assert err & 0x1 and N.get_device_error() == 0  # reported, then cleared
    out.zero_()
    call()
    torch.cuda.synchronize()
    assert N.get_device_error() == 0 and torch.equal(out, want)


@pytest.mark.parametrize("counts", [[20, 0, 45, 7], [100, 60, 0, 80], [300, 0, 129, 645]])  # tiles of 64, 128 and 256 rows
def test_fp8_products(counts):
    d, f, G, M = 272, 144, len(counts), sum(counts)
    g = torch.Generator(device="cuda").manual_seed(1)
    off = torch.tensor([0] + counts).cumsum(0).int().cuda()
    new = lambda *s: torch.empty(s, dtype=N.E4M3, device="cuda")  # noqa: E731
    rows = lambda K: (new(M, K), torch.empty(N.fp8_blocks(K), M, device="cuda"))  # noqa: E731
    xq, hq = rows(d), rows(f)
    N.fp8_row_quantize(torch.randn(M, d, device="cuda", generator=g).bfloat16(), None, *xq)
    N.fp8_row_quantize(torch.randn(M, f, device="cuda", generator=g).bfloat16(), None, *hq)
    wg, sg = new(2 * G, f, d), torch.empty(2 * G, N.fp8_blocks(f), N.fp8_blocks(d), device="cuda")
    wd, sd = new(G, d, f), torch.empty(G, N.fp8_blocks(d), N.fp8_blocks(f), device="cuda")
    N.fp8_block_quantize(torch.randn(2 * G, f, d, device="cuda", generator=g).bfloat16(), wg, sg)
    N.fp8_block_quantize(torch.randn(G, d, f, device="cuda", generator=g).bfloat16(), wd, sd)
    h, y = torch.zeros(M, f, dtype=torch.bfloat16, device="cuda"), torch.zeros(M, d, dtype=torch.bfloat16, device="cuda")
    wg, sg = wg.view(G, 2 * f, d), sg.view(G, 2, *sg.shape[1:])
    stalled_then_right(lambda: N.grouped_gemm_gateup_fp8(*xq, wg, sg, off, h), h)
    stalled_then_right(lambda: N.grouped_gemm_down_fp8(*hq, wd, sd, off, y), y)


def test_few_tokens():
    T, d, f, E, k = 5, 264, 136, 8, 2
    g = torch.Generator(device="cuda").manual_seed(2)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g) * 0.1  # noqa: E731
    args = (n(T, d).bfloat16(), n(E, d), None, n(E, 2 * f, d).bfloat16(), n(E, d, f).bfloat16(), None, None, k, "topk_softmax",
            torch.empty(T, E, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda"))
    y = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(N.few_tokens_workspace_size(T, d, f, 0, E, k), dtype=torch.uint8, device="cuda")
    stalled_then_right(lambda: N.few_tokens(*args, y, ws), y)
