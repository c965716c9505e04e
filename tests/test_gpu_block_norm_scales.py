"""The gradient behind a block on a B200 for rows of the stream whose scale is far from 1: the formulas are finite there (rstd_next is up to
1e17, and its cube is no fp32 number), and a row of zeros has a finite rstd_next with a positive eps. Tolerances as in
test_gpu_block_norm.py."""
import pytest
import torch

from test_gpu_block_norm import N, _device, gate64, inputs, near, run_out, run_out_backward  # noqa: F401 - the fixture

pytestmark = pytest.mark.gpu

SCALES = [(1e-14, 0.0), (1e15, 0.0), (1.0, 1e-6), (0.0, 1e-30), (1e-17, 0.0), (2e16, 0.0), (3e-13, 1e-30)]  # (rms of the row, eps)


@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d,rows", [(7, 264, 0), (7, 264, 2), (700, 264, 100), (700, 2880, 0), (14, 4104, 3), (350, 4104, 0),
                                      (420, 8200, 60)])
def test_gradient_of_tiny_and_huge_rows(T, d, rows, res):
    alpha = 0.5
    st = inputs(T, d, res, rows, seed=21)
    at = torch.arange(T, device="cuda") % len(SCALES)
    scale = torch.tensor([s for s, _ in SCALES], device="cuda", dtype=torch.float64)[at][:, None]
    eps = torch.tensor([e for _, e in SCALES], device="cuda", dtype=torch.float64)[at][:, None]
    g = torch.Generator(device="cuda").manual_seed(22)
    out = (torch.randn(T, d, device="cuda", generator=g, dtype=torch.float64) * scale).to(res)
    # along the stream: nothing for the largest rows, whose gradient through the norm is far below 1
    st["dout"] = torch.where(scale > 1e14, 0, st["dout"].double()).to(res)
    o = out.double()
    fwd = {"out": out, "rstd": run_out(st, alpha, False)["rstd"], "rstd_next": (o.square().mean(1, keepdim=True) + eps).rsqrt()[:, 0].float()}
    got = run_out_backward(st, fwd, alpha)
    y, w, gate = st["y"].double(), st["w"].double(), gate64(st, T)
    rstd, rn = fwd["rstd"].double()[:, None], fwd["rstd_next"].double()[:, None]
    hat, ohat, dxn = y * rstd, o * rn, st["dxn"].double()
    dn = dxn * st["w_next"].double()
    dR = st["dout"].double() + rn * (dn - ohat * (dn * ohat).mean(1, keepdim=True))
    size = st["dout"].double().abs() + rn * (dn.abs() + ohat.abs() * (dn * ohat).abs().mean(1, keepdim=True))
    near(got["dr"], alpha * dR, alpha * size, "dr")
    gabs = gate.abs() if rows else 1.0
    dn = dR * gate * w
    near(got["dy"], rstd * (dn - hat * (dn * hat).mean(1, keepdim=True)),
         rstd * (size * gabs * w.abs() + hat.abs() * (size * gabs * (w * hat).abs()).mean(1, keepdim=True)), "dy")
    near(got["dw"], (dR * gate * hat).sum(0), (size * gabs * hat.abs()).sum(0), "dw")
    near(got["dw_next"], (dxn * ohat).sum(0), (dxn * ohat).abs().sum(0), "dw_next")
    if rows:
        group = torch.arange(T, device="cuda") // rows
        add = lambda v: torch.zeros(st["gate"].shape, dtype=torch.float64, device="cuda").index_add_(0, group, v)  # noqa: E731
        near(got["dgate"], add(dR * w * hat), add(size * (w * hat).abs()), "dgate")
