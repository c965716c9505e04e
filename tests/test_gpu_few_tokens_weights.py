"""few_tokens on a B200 with infinities and NaN in one expert's weights: what the formulas say of a token that did not choose that expert
does not have them, so its row stays within the bounds that hold without them (test_gpu_few_tokens.py derives those), and everything
that the weight does not enter keeps its bits."""
import pytest
import torch

from test_gpu_few_tokens import N, _device, check, inputs, run  # noqa: F401 - the fixture

pytestmark = pytest.mark.gpu

def someones(idx, E):
    """An expert that some tokens chose and others did not: (expert, which tokens have it)."""
    tokens = torch.stack([(idx == e).any(1) for e in range(E)]).sum(1)
    e = int(torch.where((tokens > 0) & (tokens < idx.shape[0]), tokens, -1).argmax())
    has = (idx == e).any(1)
    assert has.any() and not has.all()
    return e, has


SHAPES = [(2, 256, 512, 8, 2, 0), (7, 264, 136, 16, 4, 64), (8, 4096, 1024, 8, 2, 0), (16, 1000, 768, 32, 4, 40), (20, 520, 264, 8, 2, 0),
          (32, 200, 104, 64, 8, 72), (29, 2880, 360, 6, 1, 0)]


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("T,d,f,E,k,fs", SHAPES)
def test_down_weight_of_one_expert(T, d, f, E, k, fs, bad):
    mode = "topk_softmax"
    st = inputs(T, d, f, E, k, fs, seed=T + d)
    clean = run(st, mode)
    e, has = someones(clean["topk_idx"], E)
    rest = (~has).nonzero()[:, 0].tolist()
    rows = sorted({0, 37, d // 2, d - 1})
    for i, r in enumerate(rows):
        st["w_down"][e, r, (f - 1) * i // (len(rows) - 1)] = bad
    got = run(st, mode)
    for name in ("logits", "topk_idx", "topk_w"):
        assert torch.equal(got[name], clean[name]), name
    check(st, mode, got, rest)
    others = torch.ones(d, dtype=torch.bool, device="cuda")
    others[rows] = False
    assert torch.equal(got["y"][:, others], clean["y"][:, others])
    assert not got["y"][has][:, rows].isfinite().any()
    again = run(st, mode)
    assert torch.equal(again["y"].view(torch.int16), got["y"].view(torch.int16))


@pytest.mark.parametrize("T,d,f,E,k,fs", SHAPES)
def test_gate_and_up_weights_of_one_expert(T, d, f, E, k, fs):
    mode = "sigmoid_topk_norm"
    st = inputs(T, d, f, E, k, fs, seed=T + f)
    clean = run(st, mode)
    e, has = someones(clean["topk_idx"], E)
    st["w_gateup"][e, f // 2, d // 3] = float("nan")
    st["w_gateup"][e, f + f // 3, d // 2] = float("inf")
    got = run(st, mode)
    assert torch.equal(got["y"][~has], clean["y"][~has])
    assert got["y"][has].isnan().all()


def test_a_whole_expert_of_nan():
    T, d, f, E, k = 8, 1024, 512, 16, 2
    st = inputs(T, d, f, E, k, seed=11)
    clean = run(st, "topk_softmax")
    e, has = someones(clean["topk_idx"], E)
    rest = (~has).nonzero()[:, 0].tolist()
    st["w_down"][e] = float("nan")
    got = run(st, "topk_softmax")
    check(st, "topk_softmax", got, rest)
    assert got["y"][has].isnan().all()
