"""Argument checks of the e4m3 products and of the few-token layer, before any launch (no GPU)."""
import pytest
import torch


@pytest.fixture(scope="module")
def native():
    from mixture_experts_ffn_11_b200 import _native

    return _native


def refused(fn, good, changes, status):
    for at, v in changes:
        args = list(good)
        args[at] = v
        assert fn(*args) == status, (at, v)


P = 256  # an aligned address that is never read: every call below is refused


def test_fp8_products(native):
    lib, bad = native.lib(), native.MOE_ERR_INVALID_ARG
    for fn in (lib.moe_grouped_gemm_gateup_fp8, lib.moe_grouped_gemm_down_fp8):
        good = [P, P, P, P, P, 4, 8, 64, 64, P, None]  # a, as, w, ws, offsets, G, M, d, f, out, stream
        refused(fn, good, [(0, None), (1, None), (2, None), (3, None), (4, None), (9, None), (0, P + 8), (1, P + 2), (2, P + 4),
                           (4, P + 1), (9, P + 8), (5, 0), (5, 1025), (6, -1), (7, 24), (7, 0), (8, 40), (8, -16)], bad)


def test_fp8_encoders(native):
    lib, bad = native.lib(), native.MOE_ERR_INVALID_ARG
    refused(lib.moe_fp8_block_quantize, [P, 1, 8, 32, P, P, None],
            [(0, None), (4, None), (5, None), (0, P + 8), (4, P + 8), (5, P + 2), (1, -1), (2, -1), (3, 24), (3, 0)], bad)
    refused(lib.moe_fp8_row_quantize, [P, P, 4, 32, 8, P, P, None],
            [(0, None), (1, None), (5, None), (6, None), (0, P + 8), (1, P + 2), (5, P + 4), (6, P + 2), (2, 0), (2, -1), (3, 8),
             (4, -1)], bad)  # (1, None): 8 rows of 4 without row_src


def test_few_tokens(native):
    lib, bad = native.lib(), native.MOE_ERR_INVALID_ARG
    size = native.few_tokens_workspace_size
    # x, w_router, bias, w_gateup, w_down, shared x 2, T, d, f, fs, E, k, mode, logits, idx, w, y, ws, bytes, stream
    good = [P, P, None, P, P, P, P, 4, 64, 64, 32, 8, 2, 0, P, P, P, P, P, 1 << 30, None]
    refused(lib.moe_few_tokens, good,
            [(0, None), (1, None), (3, None), (4, None), (5, None), (6, None), (14, None), (15, None), (16, None), (17, None),
             (0, P + 8), (3, P + 8), (4, P + 2), (17, P + 8), (7, 33), (7, -1), (8, 12), (8, 0), (9, 20), (10, 12), (10, -8),
             (11, 0), (11, 1025), (12, 9), (12, 0), (13, 3), (13, -1), (9, 1 << 26)], bad)
    refused(lib.moe_few_tokens, good, [(18, None), (18, P + 16), (19, size(4, 64, 64, 32, 8, 2) - 4096)],
            native.MOE_ERR_WORKSPACE)


def test_few_tokens_workspace_size(native):
    size = native.few_tokens_workspace_size
    assert size(0, 64, 64, 0, 8, 2) == 0 and size(33, 64, 64, 0, 8, 2) == 0
    # counters (1 + 2) * 4 -> 256, h 4 * 2 rows of 64 bf16 = 1024, 148 * 2 partial blocks of 32 x 8 fp32
    assert size(4, 64, 64, 0, 8, 2) == 256 + 1024 + 148 * 2 * 32 * 8 * 4
    assert native.FEW_TOKENS_MAX == 32


def test_python_checks_before_the_library(native):
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        native.fp8_row_quantize(x, None, x, x)  # CPU tensors
    with pytest.raises(ValueError):
        native.few_tokens(x, x, None, x, x.view(1, 2, 64), None, None, 1, "topk_softmax", x, x, x, x, None)
