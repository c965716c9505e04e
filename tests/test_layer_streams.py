"""MoEBlock and MoEFFN keep their buffers for the stream that works on them, also where they were allocated on another: what the caching
allocator is told (on the CPU), and what comes of it (on a B200)."""
import pytest
import torch


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


def test_block_buffers_are_recorded_on_every_stream_once(monkeypatch):
    from mixture_experts_ffn_11_b200 import MoEBlock
    from mixture_experts_ffn_11_b200 import layer

    told = []
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: told.append((t.data_ptr(), s.cuda_stream)))
    for name in ("block_norm_in", "block_norm_out", "block_norm_in_backward", "block_norm_out_backward"):
        monkeypatch.setattr(layer.N, name, lambda *a: None)

    class FFN:
        d, device = 16, torch.device("cpu")

        def forward(self, xn, stream=None, train=False):
            self._x = xn
            return torch.zeros(xn.shape, dtype=torch.bfloat16)

        def output_there(self, T):
            return None

        def backward(self, dy, weight_grads=True, stream=None):
            return {"dx": torch.zeros_like(dy)}

    block = MoEBlock(FFN(), torch.ones(16), torch.ones(16))
    r = torch.zeros(4, 16)
    block.forward(r, train=True, stream=Stream(1))
    kept = {t.data_ptr() for t in block._buf.values()}
    assert kept <= {p for p, s in told if s == 1}
    n = len(told)
    block.forward(r, train=True, stream=Stream(1))
    assert len(told) == n  # told once
    block.forward(r, train=True, stream=Stream(2))
    assert kept <= {p for p, s in told if s == 2}
    block.backward(r, stream=Stream(3))
    grads = {t.data_ptr() for t in block._gbuf.values() if t is not None}
    assert kept | grads <= {p for p, s in told if s == 3}
    block.forward(torch.zeros(5, 16), stream=Stream(1))  # other buffers
    assert {t.data_ptr() for t in block._buf.values()} <= {p for p, s in told[n:] if s == 1}


@pytest.mark.gpu
@pytest.mark.parametrize("few,weights", [(False, "bf16"), (True, "bf16"), (False, "fp8")])
def test_buffers_outlive_the_work_of_another_stream(few, weights):
    """A forward on a busy side stream, then another number of tokens and new tensors on the current one: the memory of the first call's
    intermediates is not given out before the side stream is done with it."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mixture_experts_ffn_11_b200 import MoEBlock, MoEFFN
    from mixture_experts_ffn_11_b200 import _native as N

    torch.cuda.set_device(0)
    E, d, f, k, T = 8, 512, 256, 2, 12
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g) * 0.05  # noqa: E731
    ffn = MoEFFN(n(E, d), n(E, 2 * f, d).bfloat16(), n(E, d, f).bfloat16(), k, few=few, weights=weights)
    block = MoEBlock(ffn, 1 + n(d), 1 + n(d))
    r, other = torch.randn(T, d, device="cuda", generator=g), torch.randn(3 * T, d, device="cuda", generator=g)
    want = block(r).clone()
    wanted = block(other).clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)  # some 50 ms
        got = block(r, stream=side)
        got_other = block(other)  # drops the buffers of T tokens
        filled = [torch.full((m, c), float("nan"), dtype=t, device="cuda") for _ in range(4) for m in (T, T * k)
                  for c in (1, d, f) for t in (torch.bfloat16, torch.float32)]
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(got_other, wanted)
        del filled
    assert N.get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("weights,fs", [("bf16", 0), ("bf16", 128), ("mxfp4", 256), ("fp8", 128)])
def test_first_call_on_a_side_stream_beside_a_busy_current_one(weights, fs):
    """What a first call lays out (offsets of the shared expert, unit weights and transposed copies of the backward pass) is ready on the
    stream of the call, whatever the current one has still to do."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mixture_experts_ffn_11_b200 import MoEFFN
    from mixture_experts_ffn_11_b200 import _native as N

    torch.cuda.set_device(0)
    E, d, f, k, T = 16, 256, 256, 2, 24
    g = torch.Generator(device="cuda").manual_seed(2)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g) * 0.05  # noqa: E731
    args = (n(E, d), n(E, 2 * f, d).bfloat16(), n(E, d, f).bfloat16(), k, "topk_softmax", None,
            n(2 * fs, d).bfloat16() if fs else None, n(d, fs).bfloat16() if fs else None)
    first, again = (MoEFFN(*args, weights=weights) for _ in range(2))
    train = weights == "bf16"
    x, dy = torch.randn(T, d, device="cuda", generator=g).bfloat16(), torch.randn(T, d, device="cuda", generator=g).bfloat16()
    y = first.forward(x, train=train)
    grads = first.backward(dy) if train else {}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(100_000_000)  # some 50 ms of the current stream
    y2 = again.forward(x, side, train=train)
    grads2 = again.backward(dy, side) if train else {}
    side.synchronize()
    assert torch.equal(y2, y)
    for name, v in grads.items():
        assert v is None or torch.equal(grads2[name], v), name
    assert N.get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("few,weights,fs", [(False, "bf16", 128), (True, "bf16", 0), (False, "mxfp4", 256), (False, "fp8", 128)])
def test_graphs_of_several_numbers_of_tokens(few, weights, fs):
    """One graph per number of tokens of a block, forward (with bf16 weights and the backward pass), the usual way: a call to warm up, then the
    capture. The graphs are replayed in any order between calls for other numbers of tokens, and nothing of them is written elsewhere."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from mixture_experts_ffn_11_b200 import MoEBlock, MoEFFN
    from mixture_experts_ffn_11_b200 import _native as N

    torch.cuda.set_device(0)
    E, d, f, k = 16, 256, 256, 2
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g) * 0.05  # noqa: E731
    args = (n(E, d), n(E, 2 * f, d).bfloat16(), n(E, d, f).bfloat16(), k, "topk_softmax", None,
            n(2 * fs, d).bfloat16() if fs else None, n(d, fs).bfloat16() if fs else None)
    train = weights == "bf16" and not few
    gains = 1 + n(d), 1 + n(d)
    block = MoEBlock(MoEFFN(*args, weights=weights, few=few), *gains)
    plain = MoEBlock(MoEFFN(*args, weights=weights, few=few), *gains)

    def step(b, r):
        out = b(r, train=train)
        got = {"out": out}
        if train:
            got.update({m: v for m, v in b.backward(torch.ones_like(r)).items() if v is not None})
        return got

    graphs = []
    for T in (4, 12, 40):
        r = torch.randn(T, d, device="cuda", generator=g)
        step(block, r)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step(block, r)
        graphs.append((graph, r, got))
    torch.cuda.empty_cache()
    block(torch.randn(7, d, device="cuda"))
    others = [torch.full((m, c), 7.0, dtype=t, device="cuda") for _ in range(6) for m in (4, 8, 12, 24, 40, 80) for c in (1, d, f, 2 * f)
              for t in (torch.bfloat16, torch.float32)]
    for graph, r, got in graphs + graphs[::-1]:
        r.copy_(torch.randn(r.shape, device="cuda", generator=g))
        block(torch.randn(9, d, device="cuda"))
        graph.replay()
        want = step(plain, r)
        for name, v in want.items():
            assert torch.equal(got[name], v), name
        twice = step(block, r)  # the same number of tokens without the graph
        assert torch.equal(twice["out"], want["out"])
    assert all(bool((o == 7).all()) for o in others)
    assert N.get_device_error() == 0
