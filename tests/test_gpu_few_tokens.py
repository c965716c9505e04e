"""The whole layer for few tokens (few_tokens) on a B200, against the layer's formulas in 64 bits.

Tolerances (u = 2^-24, h = eps(bf16) / 2): a fp32 sum of K products, in any order, is off by at most E(K) = (K + 4) u of the sum of
magnitudes; silu has a slope of at most 1.1, its fast exponential and divide and the products behind them are off by under
2^-20 of the result; h_tj and y are each rounded once (h of their size). The bounds below are these, carried through element by
element; besides them the relative Frobenius error stays under the layer's parity bar of 5e-3.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

N = pytest.importorskip("mixture_experts_ffn_11_b200._native")
from mixture_experts_ffn_11_b200 import MoEFFN  # noqa: E402

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


def inputs(T, d, f, E, k, fs=0, bias=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s, std=1.0: torch.randn(*s, device="cuda", generator=g) * std  # noqa: E731
    return {"x": n(T, d).bfloat16(), "w_router": n(E, d, std=0.05), "bias": n(E, std=0.5) if bias else None,
            "w_gateup": n(E, 2 * f, d, std=0.05).bfloat16(), "w_down": n(E, d, f, std=0.05).bfloat16(),
            "w_gateup_shared": n(2 * fs, d, std=0.05).bfloat16() if fs else None,
            "w_down_shared": n(d, fs, std=0.05).bfloat16() if fs else None, "k": k}


def run(st, mode, ws=None, stream=None, out=None):
    T, d = st["x"].shape
    E, f = st["w_down"].shape[0], st["w_down"].shape[2]
    fs = st["w_down_shared"].shape[1] if st["w_down_shared"] is not None else 0
    if ws is None:  # need not be initialised
        ws = torch.full((max(256, N.few_tokens_workspace_size(T, d, f, fs, E, st["k"])),), 255, dtype=torch.uint8, device="cuda")
    if out is None:
        out = {"logits": torch.full((T, E), float("nan"), device="cuda"),
               "topk_idx": torch.full((T, st["k"]), -1, dtype=torch.int32, device="cuda"),
               "topk_w": torch.full((T, st["k"]), float("nan"), device="cuda"),
               "y": torch.full((T, d), float("nan"), dtype=torch.bfloat16, device="cuda")}
    N.few_tokens(st["x"], st["w_router"], st["bias"], st["w_gateup"], st["w_down"], st["w_gateup_shared"], st["w_down_shared"],
                 st["k"], mode, out["logits"], out["topk_idx"], out["topk_w"], out["y"], ws, stream)
    return out


def expert(x, wgu, wd, scale):
    """(y, bound without the rounding of y) of one token through one expert, in 64 bits."""
    f = wd.shape[1]
    e, ef = (x.numel() + 4) * 2.0 ** -24, (wd.shape[1] + 4) * 2.0 ** -24
    g, u = wgu[:f].double() @ x, wgu[f:].double() @ x
    gs, us = wgu[:f].double().abs() @ x.abs(), wgu[f:].double().abs() @ x.abs()
    h = scale * g * torch.sigmoid(g) * u
    dh = scale * (1.1 * e * gs * (u.abs() + e * us) + e * us * (g.abs() + e * gs)) + (2.0 ** -20 + H * 1.001) * h.abs()
    return wd.double() @ h, wd.double().abs() @ (dh + ef * h.abs())


def check(st, mode, got, tokens=None):
    if tokens is not None:  # these rows alone
        st = {**st, "x": st["x"][tokens]}
        got = {name: v[tokens].contiguous() for name, v in got.items()}
    T, d = st["x"].shape
    E, k = st["w_router"].shape[0], st["k"]
    x = st["x"].double()
    # logits
    ref = x @ st["w_router"].double().t()
    size = x.abs() @ st["w_router"].double().abs().t()
    if st["bias"] is not None:
        ref, size = ref + st["bias"].double(), size + st["bias"].double().abs()
    assert ((got["logits"].double() - ref).abs() <= (d + 4) * 2.0 ** -24 * size).all()
    # selection and weights: exactly what the selection gives for these logits
    idx, w = torch.empty_like(got["topk_idx"]), torch.empty_like(got["topk_w"])
    N.topk_from_logits(got["logits"], k, mode, idx, w)
    assert torch.equal(got["topk_idx"], idx) and torch.equal(got["topk_w"], w)
    # layer output, for the selection and weights taken
    num = den = 0.0
    for t in range(T):
        y = torch.zeros(d, dtype=torch.float64, device="cuda")
        bound = torch.zeros_like(y)
        for j in range(k):
            e = int(idx[t, j])
            a, b = expert(x[t], st["w_gateup"][e], st["w_down"][e], float(w[t, j]))
            y, bound = y + a, bound + b
        if st["w_down_shared"] is not None:
            a, b = expert(x[t], st["w_gateup_shared"], st["w_down_shared"], 1.0)
            y, bound = y + a, bound + b
        err = (got["y"][t].double() - y).abs()
        assert (err <= bound + H * 1.001 * (y.abs() + bound) + 1e-30).all(), (t, float((err / (bound + H * y.abs())).max()))
        num, den = num + float((err ** 2).sum()), den + float((y ** 2).sum())
    assert (num / den) ** 0.5 <= 5e-3


CASES = [
    (1, 8, 8, 1, 1, 0), (1, 16, 8, 2, 2, 0), (2, 256, 512, 8, 2, 0), (3, 40, 24, 5, 3, 16), (8, 264, 136, 16, 4, 0),
    (9, 2880, 320, 32, 4, 0), (16, 512, 768, 128, 8, 0), (17, 72, 1032, 7, 7, 8), (32, 1024, 256, 4, 2, 1024),
    (32, 200, 104, 256, 8, 72), (1, 7168, 256, 64, 8, 256), (5, 1000, 2880, 3, 1, 40), (31, 128, 64, 1024, 32, 0),
    (4, 2880, 2880, 8, 4, 0), (32, 64, 64, 1, 1, 0), (24, 4096, 512, 8, 2, 0),
]


@pytest.mark.parametrize("mode", ["topk_softmax", "softmax_topk_renorm", "sigmoid_topk_norm"])
@pytest.mark.parametrize("T,d,f,E,k,fs", CASES)
def test_matches_the_formulas(T, d, f, E, k, fs, mode):
    st = inputs(T, d, f, E, k, fs, bias=T % 2 == 0, seed=T)
    check(st, mode, run(st, mode))


def test_every_token_to_one_expert_and_equal_logits():
    """Equal logits go to the lowest ids; all 32 tokens share the two experts."""
    st = inputs(32, 136, 72, 16, 2, 0, seed=3)
    st["w_router"].zero_()
    got = run(st, "topk_softmax")
    assert (got["topk_idx"] == torch.tensor([0, 1], dtype=torch.int32, device="cuda")).all() and (got["topk_w"] == 0.5).all()
    check(st, "topk_softmax", got)


def test_a_bad_token_stays_its_own():
    st = inputs(6, 264, 136, 16, 4, 64, seed=4)
    clean = run(st, "topk_softmax")
    st["x"][2, 5] = float("nan")
    got = run(st, "topk_softmax")
    rest = [0, 1, 3, 4, 5]
    for name in ("logits", "topk_idx", "topk_w"):
        assert torch.equal(got[name][rest], clean[name][rest]), name
    # The bad token chooses other experts than before, and the order of the down projection's sums follows the batch's active
    # experts: the other rows' sums are the same terms in another order, each within the bounds that hold for any order.
    check(st, "topk_softmax", got, rest)
    assert got["y"][2].isnan().all()


def test_same_bits_again_side_stream_graph_and_two_at_once():
    st = inputs(5, 1032, 520, 32, 4, 64, bias=True, seed=5)
    want = run(st, "topk_softmax")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(10):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(run(st, "topk_softmax"))
    torch.cuda.synchronize()
    for o in got:
        for name in want:
            assert torch.equal(o[name], want[name]), name
    out = run(st, "topk_softmax")
    ws = torch.empty(N.few_tokens_workspace_size(5, 1032, 520, 64, 32, 4), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(st, "topk_softmax", ws, out=out)
    for _ in range(3):
        out["y"].fill_(7)
        ws.fill_(90)
        graph.replay()
    torch.cuda.synchronize()
    for name in want:
        assert torch.equal(out[name], want[name]), name


def test_layer_takes_it_for_few_tokens():
    T, d, f, E, k = 7, 512, 256, 16, 4
    st = inputs(T, d, f, E, k, 128, bias=True, seed=6)
    args = (st["w_router"], st["w_gateup"], st["w_down"], k, "sigmoid_topk_norm", st["bias"], st["w_gateup_shared"],
            st["w_down_shared"])
    plain, few = MoEFFN(*args), MoEFFN(*args, few=True)
    for t in (T, 1, 16):
        x = inputs(t, d, f, E, k, seed=t)["x"]
        a, b = plain(x).clone(), few(x)
        assert torch.equal(few.buf["topk_idx"], plain.buf["topk_idx"])
        assert float((a.double() - b.double()).norm() / a.double().norm()) <= 5e-3
    x = inputs(17, d, f, E, k, seed=9)["x"]  # one more than it takes it for: the separate calls, the same bits
    assert torch.equal(plain(x), few(x))
    y = few.forward(inputs(T, d, f, E, k, seed=1)["x"], train=True)  # training keeps what the backward pass reads
    few.backward(torch.ones_like(y))


def test_refusals():
    st = inputs(4, 64, 64, 8, 2, 0, seed=7)
    with pytest.raises(N.MoEError) as e:
        run(st, "topk_softmax", ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == N.MOE_ERR_WORKSPACE
    with pytest.raises(N.MoEError):
        run(inputs(33, 64, 64, 8, 2), "topk_softmax")
    with pytest.raises(ValueError):
        run(st, "no such mode")
    bad = dict(st)
    bad["w_gateup"] = st["w_gateup"][:, :64]
    with pytest.raises(ValueError):
        run(bad, "topk_softmax")
    out = run(inputs(0, 64, 64, 8, 2), "topk_softmax")  # no tokens
    assert out["y"].shape == (0, 64)
