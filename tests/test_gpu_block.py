"""The operators around the expert layer used together on a B200: MoEFFN with fp8 weights, MoEBlock in a chain, forward and
backward.

Tolerances. A path's bf16 roundings are independent errors of at most h = 2^-8 of a value, 2^-9 in the root mean square; n of them
in a row leave at most sqrt(n) 2^-9 of the result's norm where the path's parts are about as large as their result.

fp8: e4m3 values are at least their binade's base 2^e and 2^(e-3) apart, so a rounding is off by at most q = 2^-3 / sqrt(12) = 0.0361
of the value in the root mean square, and a sum of many products keeps that share of its norm: g and u, from rounded rows and
weights, are off by sqrt(2) q. h = silu(g) u takes u's share as it is and g's times rms(silu'(g)) rms(g) / rms(silu(g)). For g and -g
equally likely, sigmoid(g)^2 + sigmoid(-g)^2 >= 1/2 gives rms(silu(g)) >= rms(g) / 2, and silu'(g) + silu'(-g) = 1 with silu' between -0.1
and 1.1 gives rms(silu') <= sqrt((1.1^2 + 0.1^2) / 2) = 0.78: a factor of at most 1.56. The roundings of h and W_down add q each:
sqrt(2 (1 + 1.56^2) + 2) q = 0.107.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

N = pytest.importorskip("mixture_experts_ffn_11_b200._native")
from mixture_experts_ffn_11_b200 import MoEBlock, MoEFFN  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    N.get_device_error()
    yield
    torch.cuda.synchronize()
    assert N.get_device_error() == 0


def weights(E, d, f, fs=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s, std=0.05: torch.randn(*s, device="cuda", generator=g) * std  # noqa: E731
    return {"w_router": n(E, d), "w_gateup": n(E, 2 * f, d).bfloat16(), "w_down": n(E, d, f).bfloat16(),
            "bias": n(E, std=0.3), "w_gateup_shared": n(2 * fs, d).bfloat16() if fs else None,
            "w_down_shared": n(d, fs).bfloat16() if fs else None}


def off(a, b):
    a, b = a.detach().double(), b.detach().double()
    return float((a - b).norm() / b.norm())


@pytest.mark.parametrize("T,fs", [(1, 0), (5, 160), (300, 0), (1000, 96)])
def test_fp8_layer(T, fs):
    E, d, f, k = 8, 528, 400, 2
    w = weights(E, d, f, fs)
    x = torch.randn(T, d, device="cuda").bfloat16()
    ref = MoEFFN(w["w_router"], w["w_gateup"], w["w_down"], k, "topk_softmax", w["bias"], w["w_gateup_shared"], w["w_down_shared"])
    lay = MoEFFN(w["w_router"], w["w_gateup"], w["w_down"], k, "topk_softmax", w["bias"], w["w_gateup_shared"], w["w_down_shared"],
                 weights="fp8")
    y, want = lay(x), ref(x)
    assert torch.equal(lay.buf["topk_idx"], ref.buf["topk_idx"])
    assert off(y, want) <= 0.107
    # the separate calls, and weights given encoded, give the same bits
    b = lay.buf
    xq = torch.empty(T * k, d, dtype=N.E4M3, device="cuda")
    xs = torch.empty(5, T * k, device="cuda")
    N.fp8_row_quantize(x, b["perm_src"], xq, xs)
    h = torch.empty(T * k, f, dtype=torch.bfloat16, device="cuda")
    N.grouped_gemm_gateup_fp8(xq, xs, *lay.f8["gateup"], b["offsets"], h)
    assert torch.equal(h, b["h"])
    again = MoEFFN(w["w_router"], lay.f8["gateup"], lay.f8["down"], k, "topk_softmax", w["bias"], lay.f8.get("gateup_shared"),
                   lay.f8.get("down_shared"), weights="fp8")
    assert torch.equal(again(x), y)
    twin = lay.sibling()
    assert torch.equal(twin(x), y)
    with pytest.raises(NotImplementedError):
        lay.backward(torch.ones_like(y))


def test_fp8_layer_refuses_what_it_cannot_encode():
    w = weights(2, 24, 16)
    with pytest.raises(N.MoEError):
        MoEFFN(w["w_router"], w["w_gateup"], w["w_down"], 1, weights="fp8")
    with pytest.raises(ValueError):
        MoEFFN(w["w_router"], (w["w_gateup"], w["w_router"]), w["w_down"], 1)


def norm(v, eps=1e-6):
    return v * (v.square().mean(1, keepdim=True) + eps).rsqrt()


def ffn64(x, p, idx, k, mode):
    """The layer in 64 bits with the given selection, differentiable."""
    logits = (x @ p["w_router"].t() + p["bias"]).gather(1, idx)
    w = torch.sigmoid(logits) if mode == "sigmoid_topk_norm" else torch.softmax(logits, 1)
    w = w / w.sum(1, keepdim=True)
    f = p["w_down"].shape[2]
    gu = torch.einsum("td,tknd->tkn", x, p["w_gateup"][idx])
    h = gu[..., :f] * torch.sigmoid(gu[..., :f]) * gu[..., f:]
    return torch.einsum("tk,tkf,tkdf->td", w, h, p["w_down"][idx])


@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,gated", [(1, False), (37, True), (200, True)])
def test_two_blocks_in_a_row(T, gated, res):
    E, d, f, k, alpha, mode = 4, 136, 72, 2, 0.6, "sigmoid_topk_norm"
    g = torch.Generator(device="cuda").manual_seed(T)
    n = lambda *s, std=1.0: torch.randn(*s, device="cuda", generator=g) * std  # noqa: E731
    blocks, raw = [], []
    for i in range(2):
        w = weights(E, d, f, seed=10 + i)
        raw.append({"w_router": w["w_router"], "w_gateup": w["w_gateup"], "w_down": w["w_down"], "bias": w["bias"],
                    "w_in": 1 + n(d, std=0.2), "w_out": 1 + n(d, std=0.2), "gate": n(d).bfloat16() if gated else None})
        ffn = MoEFFN(w["w_router"], w["w_gateup"], w["w_down"], k, mode, w["bias"])
        blocks.append(MoEBlock(ffn, raw[i]["w_in"], raw[i]["w_out"], raw[i]["gate"], alpha))
    r = n(T, d, std=2.0).to(res)
    dout = n(T, d).to(res)
    a, b = blocks
    mid, xn = a(r, next_norm=b.w_in, train=True)
    out = b(mid, xn=xn, train=True)
    # one block alone norms its input itself: the same bits
    alone = MoEBlock(b.ffn.sibling(), raw[1]["w_in"], raw[1]["w_out"], raw[1]["gate"], alpha)
    assert torch.equal(alone(mid), out)
    gb = b.backward(dout)
    ga = a.backward(gb["dr"], gb["dxn"])

    leaf = [{name: v.double().requires_grad_() for name, v in p.items() if v is not None} for p in raw]
    r64 = r.double().requires_grad_()
    v = r64
    for p, blk in zip(leaf, blocks):
        y = ffn64(norm(v) * p["w_in"], p, blk.ffn.buf["topk_idx"].long(), k, mode)
        y = norm(y) * p["w_out"]
        v = alpha * v + (y * p["gate"] if gated else y)
    # forward: per block xn, h, y_perm, y, out rounded; sqrt(10) 2^-9
    assert off(out, v) <= 10 ** 0.5 * 2 ** -9
    names = ["w_router", "w_gateup", "w_down", "bias", "w_in", "w_out"] + (["gate"] if gated else [])
    grads = torch.autograd.grad((v * dout.double()).sum(), [r64] + [p[n] for p in leaf for n in names])
    # backward: those, and dy, dy_perm, dh, g|u, dgu, dx_perm, dx, dr in each block; sqrt(26) 2^-9, and the router's gradient is a
    # difference of terms up to 4 times its size
    bar = 26 ** 0.5 * 2 ** -9
    assert off(ga["dr"], grads[0]) <= bar
    got = {"w_router": "dw_router", "w_gateup": "dw_gateup", "w_down": "dw_down", "bias": "dbias", "w_out": "dw_out", "gate": "dgate"}
    for i, gr in enumerate((ga, gb)):
        for j, name in enumerate(names):
            ref = grads[1 + i * len(names) + j]
            mine = (ga["dw_in"] if i == 0 else ga["dw_next"]) if name == "w_in" else gr[got[name]]
            assert off(mine.reshape(ref.shape), ref) <= (4 * bar if name in ("w_router", "bias") else bar), (i, name)
    assert gb["dw_in"] is None and ga["dw_next"] is not None


def test_block_with_few_tokens_and_a_gate_per_sequence():
    E, d, f, k = 8, 256, 128, 2
    w = weights(E, d, f, seed=3)
    gate = torch.randn(3, d, device="cuda").bfloat16()
    gains = 1 + 0.1 * torch.randn(2, d, device="cuda")
    r = torch.randn(7, d, device="cuda")
    outs = []
    for few in (False, True):
        ffn = MoEFFN(w["w_router"], w["w_gateup"], w["w_down"], k, bias=w["bias"], few=few)
        outs.append(MoEBlock(ffn, gains[0], gains[1], alpha=0.5)(r, gate=gate, gate_rows=3))
    assert off(outs[1], outs[0]) <= 4 ** 0.5 * 2 ** -9  # h and y_perm, or the few-token kernel's h; y of either
    with pytest.raises(ValueError):
        MoEBlock(ffn, gains[0], gains[1])(r, gate=gate, gate_rows=2)
    with pytest.raises(ValueError):
        MoEBlock(ffn, gains[0][:8], gains[1])


def test_block_refuses_a_training_forward_on_its_own_outputs():
    E, d, f, k = 4, 128, 64, 2
    w = weights(E, d, f, seed=5)
    gains = 1 + 0.1 * torch.randn(2, d, device="cuda")
    block = MoEBlock(MoEFFN(w["w_router"], w["w_gateup"], w["w_down"], k, bias=w["bias"]), gains[0], gains[1])
    r = torch.randn(9, d, device="cuda").bfloat16()
    out, xn = block(r, next_norm=gains[1])
    with pytest.raises(RuntimeError):
        block.backward(r)  # nothing was kept
    with pytest.raises(ValueError):
        block(out, train=True)
    with pytest.raises(ValueError):
        block(r, xn=xn, next_norm=gains[1], train=True)
    block(r, xn=xn, train=True)  # not overwritten without a next norm
    block.backward(torch.ones_like(r))
    first = block(r).clone()
    again = block(block(r))  # without training the stream may be updated in place
    assert torch.equal(again, block(first))
