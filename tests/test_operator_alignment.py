"""fp32 and int32 arrays that are not 4-byte aligned are refused by the norms around a block and the few-token layer before any launch
(no GPU): the kernels' accesses would fault."""
import pytest

P = 256  # an aligned address that is never read: every call below is refused


@pytest.mark.parametrize("name,good,at", [
    ("moe_block_norm_in", [P, 0, P, 4, 64, 1e-6, P, P, None], (7,)),
    ("moe_block_norm_out", [P, P, 0, P, P, 2, 1.0, P, 4, 64, 1e-6, P, P, P, P, None], (12, 14)),
    ("moe_block_norm_in_backward", [P, P, P, 0, P, P, 4, 64, P, P, P, 1 << 20, None], (5, 9)),
    ("moe_block_norm_out_backward", [P, P, P, P, 0, P, P, 2, 1.0, P, P, P, 4, 64, P, P, P, P, P, P, 1 << 20, None], (10, 11, 16, 18)),
    ("moe_few_tokens", [P, P, P, P, P, P, P, 4, 64, 64, 32, 8, 2, 0, P, P, P, P, P, 1 << 30, None], (2, 14, 15, 16)),
])
def test_misaligned_arrays(name, good, at):
    from mixture_experts_ffn_11_b200 import _native as N

    for i in at:
        for off in (1, 2):
            args = list(good)
            args[i] += off
            assert getattr(N.lib(), name)(*args) == N.MOE_ERR_INVALID_ARG, (name, i)
