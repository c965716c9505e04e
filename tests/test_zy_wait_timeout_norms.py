"""The failure path of the block norms on a B200: rings of rows whose first wait nothing ends, and the sums that the CTAs of a cluster send one
another with one CTA's missing (the test hook moe_test_set_wait, 1 ms). The kernel must end with MOE_DEVERR_WAIT_TIMEOUT, and the next call
must be right."""
import pytest
import torch

from test_zy_wait_timeout_fp8_few import N, _device  # noqa: F401 - the fixture

pytestmark = pytest.mark.gpu


def stalled_then_right(call, outs):
    call()
    want = [o.clone() for o in outs]
    assert N.get_device_error() == 0
    N.test_set_wait(1_000_000, stall=True)
    try:
        call()  # returns: its waits give up after 1 ms
        err = N.get_device_error()  # synchronises
    finally:
        N.test_set_wait(0, stall=False)
    assert err & 0x1 and N.get_device_error() == 0  # reported, then cleared
    for o in outs:
        o.zero_()
    call()
    torch.cuda.synchronize()
    assert N.get_device_error() == 0
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def tensors(T, d, rows, res):
    g = torch.Generator(device="cuda").manual_seed(T)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    z = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    return {"r": n(T, d).to(res), "y": n(T, d).to(bf), "w": 1 + 0.1 * n(d), "gate": n(-(-T // rows), d).to(bf) if rows else None,
            "out": z(T, d, t=res), "rstd": z(T), "xn": z(T, d, t=bf), "rstd_next": z(T), "dxn": n(T, d).to(bf), "dx": z(T, d, t=res),
            "dy": z(T, d, t=bf), "dw": z(d), "dw_next": z(d), "dgate": z(-(-T // rows), d) if rows else None,
            "ws": torch.empty(N.block_norm_backward_workspace_size(T, d, rows), dtype=torch.uint8, device="cuda")}


@pytest.mark.parametrize("T,d,res", [(600, 2880, torch.bfloat16), (2000, 512, torch.float32), (700, 16384, torch.float32)])
def test_rings_of_the_norms_and_of_the_gradient_in_front(T, d, res):
    t = tensors(T, d, 100, res)
    stalled_then_right(lambda: N.block_norm_in(t["r"], t["w"], 1e-6, t["xn"], t["rstd"]), [t["xn"], t["rstd"]])
    stalled_then_right(lambda: N.block_norm_out(t["y"], t["r"], t["w"], t["gate"], 100, 0.5, t["w"], 1e-6, t["out"], t["rstd"], t["xn"],
                                                t["rstd_next"]), [t["out"], t["rstd"], t["xn"], t["rstd_next"]])
    N.block_norm_in(t["r"], t["w"], 1e-6, t["xn"], t["rstd"])
    stalled_then_right(lambda: N.block_norm_in_backward(t["dxn"], t["out"], t["r"], t["w"], t["rstd"], t["dx"], t["dw"], t["ws"]),
                       [t["dx"], t["dw"]])


# one CTA to a row; three and eight CTAs with rings; five CTAs by plain loads, where only the sums can be waited for
@pytest.mark.parametrize("T,d,rows,res", [(3000, 2880, 7, torch.bfloat16), (2500, 4104, 0, torch.bfloat16), (900, 5000, 11, torch.float32),
                                          (500, 16384, 100, torch.float32), (20, 8200, 3, torch.bfloat16)])
@pytest.mark.parametrize("next_norm", [True, False])
def test_gradient_behind(T, d, rows, res, next_norm):
    t = tensors(T, d, rows, res)
    N.block_norm_out(t["y"], t["r"], t["w"], t["gate"], rows, 0.5, t["w"], 1e-6, t["out"], t["rstd"], t["xn"], t["rstd_next"])
    nxt = (t["dxn"], t["out"], t["w"], t["rstd_next"], t["dw_next"]) if next_norm else (None,) * 5
    outs = [t["dx"], t["dy"], t["dw"]] + ([t["dgate"]] if rows else []) + ([t["dw_next"]] if next_norm else [])
    stalled_then_right(lambda: N.block_norm_out_backward(t["r"], nxt[0], t["y"], nxt[1], t["w"], t["gate"], rows, 0.5, nxt[2], t["rstd"],
                                                         nxt[3], t["dx"], t["dy"], t["dw"], t["dgate"], nxt[4], t["ws"]), outs)
