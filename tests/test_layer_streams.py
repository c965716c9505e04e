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
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: told.append((t.data_ptr(), s.cuda_stream)))
    for name in ("block_norm_in", "block_norm_out", "block_norm_in_backward", "block_norm_out_backward"):
        monkeypatch.setattr(layer.N, name, lambda *a: None)

    class FFN:
        d, device = 16, torch.device("cpu")

        def forward(self, xn, stream=None, train=False):
            self._x = xn
            return torch.zeros(xn.shape, dtype=torch.bfloat16)

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
