"""Norms around a block on a B200 for many rows of more than 8192 columns (rings with four vectors of 8 columns to a thread), against the
formulas in 64 bits, and a block that updates its stream in place with rows arriving ahead through the ring."""
import pytest
import torch

import test_gpu_block_norm as base
from test_gpu_block import weights
from test_gpu_block_norm import _device  # noqa: F401 - the fixture

pytestmark = pytest.mark.gpu

SHAPES = [(297, 8200), (700, 10248), (300, 12288), (601, 16376), (299, 16384)]


@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", SHAPES)
def test_norm_in(T, d, res):
    base.test_norm_in(T, d, res)


@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("rows,next_norm", [(0, True), (100, True), (7, False)])
def test_norm_out(T, d, rows, res, next_norm):
    base.test_norm_out(T, d, rows, res, next_norm)


@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("with_res", [True, False])
def test_norm_in_backward(T, d, res, with_res):
    base.test_norm_in_backward(T, d, res, with_res)


@pytest.mark.parametrize("T", [9, 700])
@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
def test_a_block_updates_its_stream_in_place(T, res):
    from mixture_experts_ffn_11_b200 import MoEBlock, MoEFFN

    d = 528
    w = weights(4, d, 64, seed=6)
    gains = 1 + 0.1 * torch.randn(2, d, device="cuda")
    r = torch.randn(T, d, device="cuda").to(res)
    new = lambda: MoEBlock(MoEFFN(w["w_router"], w["w_gateup"], w["w_down"], 2, bias=w["bias"]), *gains)  # noqa: E731
    one, other, third = new(), new(), new()
    want = third(other(one(r))).clone()  # three blocks, each with an output of its own
    assert not torch.equal(want, one(r))
    got = one(one(one(r)))
    assert got.data_ptr() == one(r).data_ptr()
    got = one(one(one(r)))
    assert torch.equal(got, want)
