"""MoEBlock's checks on the host, on the CPU with a stand-in for the layer and the norms: calls whose inputs it would overwrite before it, or
its backward pass, has read them, and backward passes whose kept values are gone."""
import gc
import weakref

import pytest
import torch


class Stream:
    cuda_stream = 1


@pytest.fixture
def block(monkeypatch):
    from mixture_experts_ffn_11_b200 import MoEBlock, layer

    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    refuse = []

    def norm_out(*args):
        if refuse:
            raise ValueError("refused")

    monkeypatch.setattr(layer.N, "block_norm_out", norm_out)
    for name in ("block_norm_in", "block_norm_in_backward", "block_norm_out_backward"):
        monkeypatch.setattr(layer.N, name, lambda *a: None)

    class FFN:
        d, device, buf, _x = 16, torch.device("cpu"), {}, None

        def forward(self, x, stream=None, train=False):
            self._x = x
            if self.buf.get("y") is None or self.buf["y"].shape != x.shape:
                self.buf = {"y": torch.zeros(x.shape, dtype=torch.bfloat16)}
            return self.buf["y"]

        def output_there(self, T):
            return self.buf["y"] if self.buf and self.buf["y"].shape[0] == T else None

        def backward(self, dy, weight_grads=True, stream=None):
            return {"dx": torch.zeros_like(dy)}

    made = MoEBlock(FFN(), torch.ones(16), torch.ones(16))
    made.refuse = refuse
    return made


GAIN = torch.ones(16)


def test_own_outputs_are_refused_where_the_backward_pass_reads_them(block):
    r = torch.zeros(4, 16, dtype=torch.bfloat16)
    out, nxt = block.forward(r, next_norm=GAIN, stream=Stream)
    for change in ({"r": out}, {"r": out[:, :]}, {"xn": out}, {"r": nxt}, {"xn": nxt}):
        with pytest.raises(ValueError):
            block.forward(**{"r": r, "next_norm": GAIN, "train": True, "stream": Stream, **change})
    for change in ({"r": out}, {"xn": out}, {"r": nxt}, {"xn": nxt}):  # without a backward pass all of them may be updated
        block.forward(**{"r": r, "next_norm": GAIN, "stream": Stream, **change})
    block.forward(nxt, train=True, stream=Stream)  # not written without a next norm
    block.forward(r, xn=nxt, train=True, stream=Stream)


def test_the_layers_output_is_refused_as_the_stream(block):
    y = block.ffn.forward(torch.zeros(4, 16, dtype=torch.bfloat16))
    for train in (False, True):
        with pytest.raises(ValueError):
            block.forward(y, train=train, stream=Stream)
    r = torch.zeros(4, 16)
    with pytest.raises(ValueError):
        block.forward(r, xn=y, train=True, stream=Stream)
    block.forward(r, xn=y, stream=Stream)
    block.forward(y.clone(), train=True, stream=Stream)
    block.forward(y[:2], stream=Stream)  # another number of tokens: the layer writes another buffer


def test_the_output_that_the_layer_will_write():
    from mixture_experts_ffn_11_b200 import MoEFFN

    lay = object.__new__(MoEFFN)
    y4, y8 = torch.zeros(4, 16), torch.zeros(8, 16)
    lay._T, lay.buf, lay._captured = 8, {"y": y8}, {4: ({"y": y4}, set())}
    assert lay.output_there(8) is y8 and lay.output_there(4) is y4 and lay.output_there(5) is None


def test_backward_after_another_forward_of_the_layer(block):
    r, dout = torch.zeros(4, 16), torch.zeros(4, 16)
    block.forward(r, train=True, stream=Stream)
    block.backward(dout, stream=Stream)
    block.backward(dout, stream=Stream)
    block.ffn.forward(torch.zeros(4, 16, dtype=torch.bfloat16))
    with pytest.raises(RuntimeError):
        block.backward(dout, stream=Stream)
    from mixture_experts_ffn_11_b200 import MoEBlock

    twin = MoEBlock(block.ffn, GAIN, GAIN)  # two blocks over one layer
    block.forward(r, train=True, stream=Stream)
    twin.forward(r, train=True, stream=Stream)
    twin.backward(dout, stream=Stream)
    with pytest.raises(RuntimeError):
        block.backward(dout, stream=Stream)


def test_a_refused_forward_leaves_nothing_to_go_back_to(block):
    r, dout = torch.zeros(4, 16), torch.zeros(4, 16)
    block.forward(r, train=True, stream=Stream)
    block.refuse.append(True)  # the norms have overwritten what was kept by the time a later argument is refused
    with pytest.raises(ValueError):
        block.forward(r, train=True, stream=Stream)
    with pytest.raises(RuntimeError):
        block.backward(dout, stream=Stream)


def test_buffers_of_a_captured_call_are_kept(block, monkeypatch):
    r = torch.zeros(4, 16)
    capturing = [True]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    block.forward(r, train=True, stream=Stream)
    block.backward(r, stream=Stream)
    held = [weakref.ref(t) for b in (block._buf, block._gbuf) for t in b.values() if t is not None]
    at = block._buf["out"].data_ptr(), block._gbuf["dr"].data_ptr()
    capturing[0] = False
    block.forward(torch.zeros(5, 16), train=True, stream=Stream)
    block.backward(torch.zeros(5, 16), stream=Stream)
    dropped = [weakref.ref(t) for b in (block._buf, block._gbuf) for t in b.values() if t is not None]
    block.forward(torch.zeros(6, 16), train=True, stream=Stream)
    block.backward(torch.zeros(6, 16), stream=Stream)
    gc.collect()
    assert all(h() is not None for h in held) and all(h() is None for h in dropped)
    block.forward(r, train=True, stream=Stream)  # the same tokens again: the same buffers
    block.backward(r, stream=Stream)
    assert at == (block._buf["out"].data_ptr(), block._gbuf["dr"].data_ptr())
