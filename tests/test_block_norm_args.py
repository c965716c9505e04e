"""The block norms' argument checks, before any launch (no GPU)."""
import torch
import pytest


@pytest.fixture(scope="module")
def native():
    from mixture_experts_ffn_11_b200 import _native

    return _native


def test_sizes_types_and_pointers_are_refused(native):
    lib, bad = native.lib(), native.MOE_ERR_INVALID_ARG
    p = 64  # an aligned address that is never read: every call below is refused
    assert lib.moe_block_norm_in(p, 0, p, 4, 12, 1e-6, p, p, None) == bad  # d not a multiple of 8
    assert lib.moe_block_norm_in(p, 0, p, 4, 0, 1e-6, p, p, None) == bad
    assert lib.moe_block_norm_in(p, 0, p, 4, 16392, 1e-6, p, p, None) == bad  # d above the limit
    assert lib.moe_block_norm_in(p, 0, p, -1, 64, 1e-6, p, p, None) == bad
    assert lib.moe_block_norm_in(p, 2, p, 4, 64, 1e-6, p, p, None) == bad  # unknown type
    assert lib.moe_block_norm_in(p, 0, p, 4, 64, -1e-6, p, p, None) == bad
    assert lib.moe_block_norm_in(p, 0, p, 4, 64, float("nan"), p, p, None) == bad
    assert lib.moe_block_norm_in(p + 8, 0, p, 4, 64, 1e-6, p, p, None) == bad  # misaligned
    assert lib.moe_block_norm_in(None, 0, p, 4, 64, 1e-6, p, p, None) == bad
    out = [p, p, 0, p, p, 2, 1.0, p, 4, 64, 1e-6, p, p, p, p, None]
    for at, v in ((4, None), (5, 0), (5, -3), (7, p + 4), (11, None), (12, None), (13, None), (14, None)):
        args = list(out)
        args[at] = v
        assert lib.moe_block_norm_out(*args) == bad, (at, v)
    back = [p, p, p, p, 0, p, p, 2, 1.0, p, p, p, 4, 64, p, p, p, p, p, p, 1 << 20, None]
    for at, v in ((0, None), (1, None), (3, None), (9, None), (11, None), (17, None), (18, None), (14, p + 8)):
        args = list(back)
        args[at] = v
        assert lib.moe_block_norm_out_backward(*args) == bad, (at, v)
    args = list(back)
    args[20] = 100
    assert lib.moe_block_norm_out_backward(*args) == native.MOE_ERR_WORKSPACE
    args = [p, p, p, 0, p, p, 4, 64, p, p, None, 0, None]
    assert lib.moe_block_norm_in_backward(*args) == native.MOE_ERR_WORKSPACE


def test_workspace_size(native):
    size = native.block_norm_backward_workspace_size
    assert size(0, 64) == 0
    assert size(1, 64) == 2 * 64 * 4  # two sums, one range of rows
    assert size(5000, 2880, 1000) == 296 * 2880 * 4 * 4
    assert size(5000, 2880) == 296 * 2880 * 4 * 2


def test_cpu_tensors_are_refused(native):
    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        native.block_norm_in(x, torch.ones(8), 1e-6, x, torch.ones(2))
