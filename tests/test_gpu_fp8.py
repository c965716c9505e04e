"""e4m3 operands with a scale per block of 128 on a B200: the encoders bit for bit, the grouped products against sums in 64
bits.

Tolerances (u = 2^-24, h = eps(bf16) / 2): products of two e4m3 values are exact in fp32. A sum of K of them in fp32, in any order, is
off by at most K u of the sum of magnitudes; scales, and the sums over blocks, add under (K / 128 + 3) u of it: E(K) = (1.01 K + 4)
u. silu has a slope of at most 1.1; its fast exponential and divide, and the product with u, are off by under 2^-20 of the
result. What is stored is off by h of its size besides.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

N = pytest.importorskip("mixture_experts_ffn_11_b200._native")

E4M3 = torch.float8_e4m3fn
H = torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    N.get_device_error()
    yield
    torch.cuda.synchronize()
    assert N.get_device_error() == 0


def nb(n):
    return (n + 127) // 128


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def spread(s, n, dim):
    return s.repeat_interleave(128, dim).narrow(dim, 0, n)


def encode(x, top):
    """The definition: 448 x / top in 64 bits (ties stay ties), to e4m3; top spread over x."""
    some = torch.where(top > 0, top, torch.full_like(top, 448.0))
    v = (x.double() * 448.0 / some.double()).clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    q = torch.round(v / step) * step  # to even
    return q.float().to(E4M3), some / torch.full_like(some, 448.0)


def row_tops(x):
    R, K = x.shape
    return torch.nn.functional.pad(x.float(), (0, nb(K) * 128 - K)).view(R, nb(K), 128).abs().amax(2)


def quantize_rows(x, row_src=None, R=None):
    R = x.shape[0] if R is None else R
    K = x.shape[1]
    q = torch.full((R, K), 0x7f, dtype=torch.uint8, device="cuda").view(E4M3)
    s = torch.full((nb(K), R), float("nan"), device="cuda")
    N.fp8_row_quantize(x, row_src, q, s)
    return q, s


def quantize_weights(w):
    G, n, K = w.shape
    q = torch.full((G, n, K), 0x7f, dtype=torch.uint8, device="cuda").view(E4M3)
    s = torch.full((G, nb(n), nb(K)), float("nan"), device="cuda")
    N.fp8_block_quantize(w, q, s)
    return q, s


def bits(q):
    b = q.view(torch.uint8)
    return torch.where(b == 0x80, torch.zeros_like(b), b)  # the two zeros are one value


@pytest.mark.parametrize("R,K", [(1, 16), (3, 128), (7, 144), (33, 2880), (5, 7168), (64, 1024), (2, 4112)])
def test_row_encoder_is_exact(R, K):
    x = torch.randn(R, K, device="cuda", generator=gen(R + K)) * torch.exp(3 * torch.randn(R, K, device="cuda", generator=gen(1)))
    x = x.bfloat16()
    x[0, :16] = 0
    q, s = quantize_rows(x)
    top = row_tops(x)
    want, scale = encode(x, spread(top, K, 1))
    assert torch.equal(bits(q), bits(want))
    assert torch.equal(spread(s.t(), K, 1), scale)


def test_ties_zero_blocks_and_extreme_magnitudes():
    """Tops divisible by 7 make quotients that are exact ties; blocks of zeros; the smallest and largest bf16 magnitudes."""
    x = torch.zeros(8, 256, device="cuda")
    x[0, :128] = 7.0
    x[0, 1:128] = torch.arange(1, 128, device="cuda") / 16.0  # 448 x / 7 = 4 (1 .. 127): many ties
    x[1, 0], x[1, 1:128] = 112.0, torch.arange(1, 128, device="cuda") * 0.0078125
    x[2, 5] = 9.2e-41
    x[3, :] = 3.3e38
    x[4, 0], x[4, 1] = 3.3e38, 1e-38
    x[5, 0], x[5, 1:64] = 1e-38, torch.arange(1, 64, device="cuda") * 1e-40
    x[6, 128:] = -1.0
    x = x.bfloat16()
    q, s = quantize_rows(x)
    top = row_tops(x)
    want, scale = encode(x, spread(top, 256, 1))
    assert torch.equal(bits(q), bits(want))
    assert torch.equal(spread(s.t(), 256, 1), scale)
    assert (s[:, 7] == 1).all()


def test_row_gather_and_bad_rows():
    x = torch.randn(10, 272, device="cuda", generator=gen(3)).bfloat16()
    src = torch.tensor([9, 0, 0, 5, 3, 9, 1], dtype=torch.int32, device="cuda")
    q, s = quantize_rows(x, src, 7)
    q0, s0 = quantize_rows(x)
    assert torch.equal(bits(q), bits(q0)[src.long()]) and torch.equal(s, s0[:, src.long()])
    q, s = quantize_rows(x, torch.tensor([1, -1, 10, 2], dtype=torch.int32, device="cuda"), 4)
    assert N.get_device_error() == 0x8  # flagged, encoded as zeros
    assert (bits(q)[1:3] == 0).all() and torch.equal(bits(q)[3], bits(q0)[2])
    bad = x.clone()
    bad[2, 200] = float("inf")
    bad[4, 3] = float("nan")
    q, s = quantize_rows(bad)
    assert torch.equal(bits(q)[[0, 1, 3]], bits(q0)[[0, 1, 3]])
    assert (q[2, 128:256].float() * s[1, 2]).isnan().all() and q[4, 3].float().isnan()


@pytest.mark.parametrize("G,n,K", [(1, 8, 16), (2, 130, 144), (3, 256, 2880), (1, 2880, 272)])
def test_weight_encoder_is_exact(G, n, K):
    w = (torch.randn(G, n, K, device="cuda", generator=gen(n)) * 0.02).bfloat16()
    w[0, :, :16] *= 30
    q, s = quantize_weights(w)
    top = torch.nn.functional.pad(w.float(), (0, nb(K) * 128 - K, 0, nb(n) * 128 - n))
    top = top.view(G, nb(n), 128, nb(K), 128).abs().amax((2, 4))
    want, scale = encode(w, spread(spread(top, n, 1), K, 2))
    assert torch.equal(bits(q), bits(want))
    assert torch.equal(spread(spread(s, n, 1), K, 2), scale)


def problem(counts, d, f, seed, lead=0):
    """Rows and weights with their values; `lead` rows before the first group, 3 behind the last."""
    g = gen(seed)
    M = lead + sum(counts) + 3
    off = torch.tensor([lead] + counts, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
    a = torch.randn(M, d, device="cuda", generator=g)
    a[:, ::41] *= 10
    aq, a_s = quantize_rows(a.bfloat16())
    G = len(counts)
    w = (torch.randn(G, 2 * f, d, device="cuda", generator=g) * 0.05).bfloat16()
    wq, ws = quantize_weights(w.view(2 * G, f, d))
    # scales of another origin: any finite ones
    ws = ws * torch.exp(0.5 * torch.randn(ws.shape, device="cuda", generator=g))
    return off, aq, a_s, wq.view(G, 2 * f, d), ws.view(G, 2, nb(f), nb(d))


def down_problem(counts, d, f, seed, lead=0):
    g = gen(seed)
    M = lead + sum(counts) + 3
    off = torch.tensor([lead] + counts, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
    hq, h_s = quantize_rows(torch.randn(M, f, device="cuda", generator=g).bfloat16())
    wq, ws = quantize_weights((torch.randn(len(counts), d, f, device="cuda", generator=g) * 0.05).bfloat16())
    return off, hq, h_s, wq, ws


def sums(q, s, lo, hi, w):
    """(sum, sum of magnitudes) of rows lo..hi with weight w [n, K] in 64 bits."""
    a = q[lo:hi].double() * spread(s[:, lo:hi].t().double(), q.shape[1], 1)
    return a @ w.t(), a.abs() @ w.abs().t()


def fraction(K):
    return (1.01 * K + 4) * 2.0 ** -24


COUNTS = [([1], 16, 16), ([0, 1, 0], 128, 128), ([3, 0, 17, 1], 272, 144), ([5], 2880, 160), ([33, 64, 65, 2], 1040, 400),
          ([300, 0, 127, 1, 256, 257], 512, 272), ([100, 31, 513], 144, 2880), ([64] * 5, 2048, 768), ([1] * 40, 256, 128),
          ([1000], 384, 640)]


@pytest.mark.parametrize("lead", [0, 5])
@pytest.mark.parametrize("counts,d,f", COUNTS)
def test_gateup(counts, d, f, lead):
    off, aq, a_s, wq, ws = problem(counts, d, f, 11, lead)
    M = aq.shape[0]
    h = torch.full((M, f), float("nan"), dtype=torch.bfloat16, device="cuda")
    N.grouped_gemm_gateup_fp8(aq, a_s, wq, ws, off, h)
    o = off.tolist()
    e = fraction(d)
    for g in range(len(counts)):
        lo, hi = o[g], o[g + 1]
        gate, gsize = sums(aq, a_s, lo, hi, wq[g, :f].double() * spread(spread(ws[g, 0].double(), f, 0), d, 1))
        up, usize = sums(aq, a_s, lo, hi, wq[g, f:].double() * spread(spread(ws[g, 1].double(), f, 0), d, 1))
        ref = gate * torch.sigmoid(gate) * up
        bound = 1.1 * e * gsize * (up.abs() + e * usize) + e * usize * (gate.abs() + e * gsize) + (2.0 ** -20 + H * 1.001) * ref.abs()
        err = (h[lo:hi].double() - ref).abs()
        assert (err <= bound + 1e-30).all(), (g, float((err / (bound + 1e-30)).max()))
    assert h[:lead].isnan().all() and h[o[-1]:].isnan().all()  # rows outside the groups are left as they were


@pytest.mark.parametrize("lead", [0, 5])
@pytest.mark.parametrize("counts,d,f", COUNTS)
def test_down(counts, d, f, lead):
    off, hq, h_s, wq, ws = down_problem(counts, d, f, 12, lead)
    M = hq.shape[0]
    y = torch.full((M, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    N.grouped_gemm_down_fp8(hq, h_s, wq, ws, off, y)
    o = off.tolist()
    for g in range(len(counts)):
        lo, hi = o[g], o[g + 1]
        ref, size = sums(hq, h_s, lo, hi, wq[g].double() * spread(spread(ws[g].double(), d, 0), f, 1))
        bound = fraction(f) * size + H * 1.001 * ref.abs()
        err = (y[lo:hi].double() - ref).abs()
        assert (err <= bound + 1e-30).all(), (g, float((err / (bound + 1e-30)).max()))
    assert y[:lead].isnan().all() and y[o[-1]:].isnan().all()


def test_a_row_of_nan_stays_in_its_row():
    off, aq, a_s, wq, ws = problem([40, 3], 272, 144, 13)
    h = torch.empty(46, 144, dtype=torch.bfloat16, device="cuda")
    N.grouped_gemm_gateup_fp8(aq, a_s, wq, ws, off, h)
    clean = h.clone()
    aq[7, 100] = float("nan")
    a_s[1, 41] = float("inf")
    N.grouped_gemm_gateup_fp8(aq, a_s, wq, ws, off, h)
    rest = [r for r in range(43) if r not in (7, 41)]
    assert torch.equal(h[rest], clean[rest]) and h[7].isnan().all() and not h[41].isfinite().any()


def test_same_bits_again_on_a_side_stream_and_in_a_graph():
    off, aq, a_s, wq, ws = problem([70, 0, 300], 1040, 400, 14)
    offd, hq, h_s, wqd, wsd = down_problem([70, 0, 300], 1040, 400, 15)
    h = torch.zeros(373, 400, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(373, 1040, dtype=torch.bfloat16, device="cuda")

    def go(stream=None):
        N.grouped_gemm_gateup_fp8(aq, a_s, wq, ws, off, h, stream)
        N.grouped_gemm_down_fp8(hq, h_s, wqd, wsd, offd, y, stream)

    go()
    want = h.clone(), y.clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    h.zero_()
    y.zero_()
    side.wait_stream(torch.cuda.current_stream())
    go(side)
    side.synchronize()
    assert torch.equal(h, want[0]) and torch.equal(y, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for _ in range(3):
        h.zero_()
        y.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, want[0]) and torch.equal(y, want[1])


def test_bad_offsets_are_flagged():
    off, aq, a_s, wq, ws = problem([4, 4], 128, 128, 16)
    off[1] = 1000
    h = torch.empty(11, 128, dtype=torch.bfloat16, device="cuda")
    N.grouped_gemm_gateup_fp8(aq, a_s, wq, ws, off, h)
    assert N.get_device_error() & 0x4


def test_no_rows():
    off, aq, a_s, wq, ws = problem([0, 0], 128, 128, 17)
    h = torch.full((3, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    N.grouped_gemm_gateup_fp8(aq, a_s, wq, ws, off, h)
    assert (h == 5).all()
    N.grouped_gemm_gateup_fp8(aq[:0], a_s[:, :0].contiguous(), wq, ws, off, h[:0])
    quantize_rows(torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"))


def test_refusals():
    off, aq, a_s, wq, ws = problem([4, 4], 128, 128, 18)
    h = torch.empty(11, 128, dtype=torch.bfloat16, device="cuda")
    ok = dict(aq=aq, a_s=a_s, wq_gateup=wq, ws_gateup=ws, group_offsets=off, h=h)
    for change in ({"aq": aq.view(torch.uint8)}, {"a_s": a_s.t().contiguous()}, {"ws_gateup": ws[:, 0]}, {"h": h.float()},
                   {"group_offsets": off.long()}, {"group_offsets": off.cpu()}, {"wq_gateup": wq.transpose(1, 2)}):
        with pytest.raises(ValueError):
            N.grouped_gemm_gateup_fp8(**{**ok, **change})
    with pytest.raises(N.MoEError):  # rows of 24 bytes
        quantize_rows(torch.zeros(2, 24, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(N.MoEError):  # more rows than x has, and no row_src
        quantize_rows(torch.zeros(2, 32, dtype=torch.bfloat16, device="cuda"), None, 3)
