"""Norms around a block (block_norm_in, block_norm_out) and their gradients on a B200, against the formulas in 64 bits.

Tolerances, from the arithmetic (u = 2^-24 the fp32 rounding, h = eps(type) / 2 the half step of the stored type):
  * A row sum of d <= 16384 products is a chain of at most 32 additions in a thread and a tree of 10: its error is at most
    (32 + 10 + 1) u of the sum of magnitudes, under 3e-6. rsqrtf adds 2 ulp, each further product or sum 1 u. E = 1e-5 covers
    a value computed from such sums, relative to the sum of the magnitudes that enter it.
  * Sums over tokens run over at most ceil(T / 296) rows in a CTA, then over at most 37 + 8 partial sums; for the T used here
    (<= 3000) that is under (11 + 45) u, inside the same E.
  * What is stored in `type` is off by h of its size besides.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

N = pytest.importorskip("mixture_experts_ffn_11_b200._native")

E = 1e-5
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)
    N.get_device_error()
    yield
    torch.cuda.synchronize()
    assert N.get_device_error() == 0


def half(dtype):
    return torch.finfo(dtype).eps / 2


def near(got, ref, size, what):
    """|got - ref| <= E * size + h * |ref|, element by element; size: the magnitudes that went into ref."""
    h = half(got.dtype) if got.dtype != torch.float32 else 0.0
    err = (got.double() - ref).abs()
    bound = E * size + h * ref.abs() * (1 + 2 * E) + 1e-37
    assert torch.isfinite(got.double()).all(), what
    assert (err <= bound).all(), f"{what}: off by {float((err / bound).max()):.3g} of the bound"


def inputs(T, d, res, gate_rows, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s, std=1.0: torch.randn(*s, device="cuda", generator=g) * std  # noqa: E731
    r = n(T, d, std=2.0)
    r[:, ::37] *= 20
    return {"r": r.to(res), "y": n(T, d, std=0.7).bfloat16(), "w": 1 + n(d, std=0.3), "w_next": 1 + n(d, std=0.3),
            "gate": n(-(-T // gate_rows), d).bfloat16() if gate_rows else None, "gate_rows": gate_rows,
            "dout": n(T, d).to(res), "dxn": n(T, d).bfloat16()}


def f64_norm(v):
    return (v.square().mean(1, keepdim=True) + EPS).rsqrt()


def gate64(st, T):
    if st["gate"] is None:
        return 1.0
    return st["gate"].double()[torch.arange(T, device="cuda") // st["gate_rows"]]


def run_out(st, alpha, next_norm=True, out=None, stream=None):
    T, d = st["y"].shape
    nan = float("nan")
    got = {"out": torch.full_like(st["r"], nan) if out is None else out,
           "rstd": torch.full((T,), nan, device="cuda"), "xn": torch.full((T, d), nan, dtype=torch.bfloat16, device="cuda"),
           "rstd_next": torch.full((T,), nan, device="cuda")}
    N.block_norm_out(st["y"], st["r"], st["w"], st["gate"], st["gate_rows"], alpha, st["w_next"] if next_norm else None, EPS,
                     got["out"], got["rstd"], got["xn"], got["rstd_next"], stream)
    return got


def run_out_backward(st, fwd, alpha, next_norm=True, dr=None):
    T, d = st["y"].shape
    nan = float("nan")
    new = lambda *s, t=torch.float32: torch.full(s, nan, dtype=t, device="cuda")  # noqa: E731
    ws = torch.full((max(16, N.block_norm_backward_workspace_size(T, d, st["gate_rows"])),), 255, dtype=torch.uint8,
                    device="cuda")
    got = {"dr": torch.full_like(st["dout"], nan) if dr is None else dr, "dy": new(T, d, t=torch.bfloat16), "dw": new(d),
           "dgate": new(*st["gate"].shape) if st["gate"] is not None else None, "dw_next": new(d) if next_norm else None}
    N.block_norm_out_backward(st["dout"], st["dxn"] if next_norm else None, st["y"], fwd["out"] if next_norm else None, st["w"],
                              st["gate"], st["gate_rows"], alpha, st["w_next"] if next_norm else None, fwd["rstd"],
                              fwd["rstd_next"] if next_norm else None, got["dr"], got["dy"], got["dw"], got["dgate"],
                              got["dw_next"], ws)
    return got


SHAPES = [(1, 8), (1, 2880), (2, 1000), (5, 1032), (64, 7168), (149, 4096), (333, 2880), (297, 4104), (3, 8200), (7, 16384),
          (3000, 520)]


@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", SHAPES)
def test_norm_in(T, d, res):
    st = inputs(T, d, res, 0)
    xn = torch.full((T + 1, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    rstd = torch.full((T,), float("nan"), device="cuda")
    N.block_norm_in(st["r"], st["w"], EPS, xn[:T], rstd)
    x = st["r"].double()
    ref = x * f64_norm(x) * st["w"].double()
    near(rstd, f64_norm(x)[:, 0], f64_norm(x)[:, 0], "rstd")
    near(xn[:T], ref, ref.abs(), "xn")
    assert xn[T].isnan().all()  # the row behind the last one is left as it was


@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d,rows", [(1, 8, 1), (1, 2880, 0), (5, 1032, 2), (64, 7168, 64), (333, 2880, 100), (297, 4104, 1),
                                      (7, 16384, 3), (3000, 520, 1000), (149, 4096, 500)])
@pytest.mark.parametrize("next_norm", [True, False])
def test_norm_out(T, d, rows, res, next_norm):
    st = inputs(T, d, res, rows, seed=1)
    got = run_out(st, 0.5, next_norm)
    y, r = st["y"].double(), st["r"].double()
    n = gate64(st, T) * (y * f64_norm(y) * st["w"].double())
    near(got["rstd"], f64_norm(y)[:, 0], f64_norm(y)[:, 0], "rstd")
    near(got["out"], 0.5 * r + n, 0.5 * r.abs() + n.abs(), "out")
    if next_norm:  # of the stream as it was stored
        o = got["out"].double()
        ref = o * f64_norm(o) * st["w_next"].double()
        near(got["rstd_next"], f64_norm(o)[:, 0], f64_norm(o)[:, 0], "rstd_next")
        near(got["xn"], ref, ref.abs(), "xn")
    else:
        assert got["xn"].isnan().all() and got["rstd_next"].isnan().all()
    again = run_out(st, 0.5, next_norm, out=st["r"])  # the residual updated in place: the same bits
    assert torch.equal(again["out"], got["out"])


@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", SHAPES)
@pytest.mark.parametrize("with_res", [True, False])
def test_norm_in_backward(T, d, res, with_res):
    st = inputs(T, d, res, 0, seed=2)
    x, w, dxn = st["r"].double(), st["w"].double(), st["dxn"].double()
    rstd = f64_norm(x)
    dres = st["dout"] if with_res else None
    ws = torch.full((N.block_norm_backward_workspace_size(T, d),), 255, dtype=torch.uint8, device="cuda")
    dx, dw = torch.full_like(st["r"], float("nan")), torch.full((d,), float("nan"), device="cuda")
    kept = rstd[:, 0].float()
    N.block_norm_in_backward(st["dxn"], dres, st["r"], st["w"], kept, dx, dw, ws)
    rstd = kept.double()[:, None]
    hat, dn = x * rstd, dxn * w
    ref = rstd * (dn - hat * (dn * hat).mean(1, keepdim=True))
    size = rstd * (dn.abs() + hat.abs() * (dn * hat).abs().mean(1, keepdim=True))
    if with_res:
        ref, size = ref + dres.double(), size + dres.double().abs()
    near(dx, ref, size, "dx")
    near(dw, (dxn * hat).sum(0), (dxn * hat).abs().sum(0), "dw")
    if with_res:  # in place of dres: the same bits
        before, dw2 = dx.clone(), torch.empty_like(dw)
        N.block_norm_in_backward(st["dxn"], st["dout"], st["r"], st["w"], kept, st["dout"], dw2, ws)
        assert torch.equal(before, st["dout"]) and torch.equal(dw, dw2)


@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d,rows", [(1, 8, 1), (1, 2880, 0), (5, 1032, 2), (64, 7168, 64), (333, 2880, 100), (333, 1000, 7),
                                      (297, 4104, 1), (299, 264, 2), (7, 16384, 3), (3000, 520, 1000), (3000, 264, 0),
                                      (149, 4096, 500), (2999, 128, 13), (600, 64, 5)])
@pytest.mark.parametrize("next_norm", [True, False])
def test_norm_out_backward(T, d, rows, res, next_norm):
    alpha = 0.22
    st = inputs(T, d, res, rows, seed=3)
    fwd = run_out(st, alpha)
    got = run_out_backward(st, fwd, alpha, next_norm)
    y, w, dout, g = st["y"].double(), st["w"].double(), st["dout"].double(), gate64(st, T)
    rstd = fwd["rstd"].double()[:, None]
    hat = y * rstd
    dR, size = dout, dout.abs()
    if next_norm:
        rn = fwd["rstd_next"].double()[:, None]
        o, dxn, wn = fwd["out"].double(), st["dxn"].double(), st["w_next"].double()
        ohat, dn = o * rn, dxn * wn
        dR = dout + rn * (dn - ohat * (dn * ohat).mean(1, keepdim=True))
        size = size + rn * (dn.abs() + ohat.abs() * (dn * ohat).abs().mean(1, keepdim=True))
        near(got["dw_next"], (dxn * ohat).sum(0), (dxn * ohat).abs().sum(0), "dw_next")
    near(got["dr"], alpha * dR, alpha * size, "dr")
    gabs = g.abs() if torch.is_tensor(g) else g
    dn = dR * g * w
    near(got["dy"], rstd * (dn - hat * (dn * hat).mean(1, keepdim=True)),
         rstd * (size * gabs * w.abs() + hat.abs() * (size * gabs * (w * hat).abs()).mean(1, keepdim=True)), "dy")
    near(got["dw"], (dR * g * hat).sum(0), (size * gabs * hat.abs()).sum(0), "dw")
    if rows:
        at = torch.arange(T, device="cuda") // rows
        add = lambda v: torch.zeros(st["gate"].shape, dtype=torch.float64, device="cuda").index_add_(0, at, v)  # noqa: E731
        near(got["dgate"], add(dR * w * hat), add(size * (w * hat).abs()), "dgate")
    again = run_out_backward(st, fwd, alpha, next_norm)  # no atomics: the same bits
    for name, v in got.items():
        assert v is None or torch.equal(v, again[name]), name
    st["dout"] = st["dout"].clone()
    inplace = run_out_backward(st, fwd, alpha, next_norm, dr=st["dout"])
    for name, v in got.items():
        assert v is None or torch.equal(v, inplace[name]), name


@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d,rows", [(149, 4104, 0), (700, 5000, 11), (311, 8192, 1), (601, 8200, 601), (160, 12288, 7), (450, 16384, 200)])
@pytest.mark.parametrize("next_norm", [True, False])
def test_norm_out_backward_of_wide_rows(T, d, rows, res, next_norm):
    """Rows over several CTAs, many of them to each: slices of unequal length, every count of CTAs from 3 to 8; in place and run again."""
    test_norm_out_backward(T, d, rows, res, next_norm)
    st = inputs(T, d, res, rows, seed=7)
    fwd = run_out(st, 1.0)
    first = run_out_backward(st, fwd, 1.0, next_norm)
    dout = st["dout"].clone()
    st["dout"].copy_(dout)
    again = run_out_backward(st, fwd, 1.0, next_norm, dr=st["dout"])  # in place of dout
    for name in first:
        if first[name] is not None:
            assert torch.equal(first[name], again[name]), name


def test_gradients_are_the_formulas_own():
    """The 64-bit formulas above against autograd and central differences of the forward in 64 bits."""
    T, d, rows, alpha = 6, 16, 4, 0.7
    st = inputs(T, d, torch.float32, rows, seed=4)
    leaf = {k: st[k].double().requires_grad_() for k in ("r", "y", "w", "w_next", "gate")}
    dout, dxn = st["dout"].double(), st["dxn"].double()
    at = torch.arange(T, device="cuda") // rows

    def loss(v):
        out = alpha * v["r"] + v["gate"][at] * (v["y"] * f64_norm(v["y"]) * v["w"])
        return (out * dout).sum() + (out * f64_norm(out) * v["w_next"] * dxn).sum()

    grads = dict(zip(leaf, torch.autograd.grad(loss(leaf), list(leaf.values()))))
    plain = {k: v.detach() for k, v in leaf.items()}
    for k, v in plain.items():
        flat = v.reshape(-1)
        for i in (0, 3, flat.numel() - 1):
            hi, lo = dict(plain), dict(plain)
            hi[k], lo[k] = flat.clone(), flat.clone()
            hi[k][i] += 1e-5
            lo[k][i] -= 1e-5
            hi[k], lo[k] = hi[k].view(v.shape), lo[k].view(v.shape)
            diff = (loss(hi) - loss(lo)) / 2e-5
            assert abs(float(diff - grads[k].reshape(-1)[i])) <= 1e-7 * (1 + abs(float(diff))), (k, i)
    fwd = run_out(st, alpha)
    got = run_out_backward(st, fwd, alpha)
    # fp32 throughout but for dy (bf16): E of magnitudes that are here within 100 of 1
    for name, key in (("dr", "r"), ("dw", "w"), ("dw_next", "w_next"), ("dgate", "gate"), ("dy", "y")):
        h = half(torch.bfloat16) if name == "dy" else 0.0
        assert ((got[name].double() - grads[key]).abs() <= 100 * E + h * grads[key].abs()).all(), name


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_bad_row_stays_in_its_row(bad):
    T, d = 9, 1000
    st = inputs(T, d, torch.bfloat16, 1, seed=5)
    clean = run_out(st, 1.0)
    st["y"] = st["y"].clone()
    st["y"][4, 17] = bad
    got = run_out(st, 1.0)
    rest = [t for t in range(T) if t != 4]
    for name in ("out", "xn", "rstd", "rstd_next"):
        assert torch.equal(got[name][rest], clean[name][rest]), name
    assert got["out"][4].isnan().any() and got["xn"][4].isnan().all()


def test_zero_rows_and_no_tokens():
    d = 264
    st = inputs(3, d, torch.bfloat16, 0, seed=6)
    st["y"].zero_()
    got = run_out(st, 1.0)
    assert torch.equal(got["out"], st["r"])  # a zero row normed is zero
    st = inputs(0, d, torch.float32, 4, seed=6)
    fwd = run_out(st, 1.0)
    grads = run_out_backward(st, fwd, 1.0)
    assert (grads["dw"] == 0).all() and (grads["dw_next"] == 0).all() and grads["dgate"].shape == (0, d)
    dw = torch.full((d,), float("nan"), device="cuda")
    N.block_norm_in_backward(st["dxn"], st["dout"], st["r"], st["w"], fwd["rstd"], torch.empty_like(st["r"]), dw, None)
    assert (dw == 0).all()


def test_side_stream_and_graph():
    st = inputs(200, 2880, torch.bfloat16, 50, seed=7)
    want = run_out(st, 1.0)
    gwant = run_out_backward(st, want, 1.0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run_out(st, 1.0)
    side.synchronize()
    for name in want:
        assert torch.equal(want[name], got[name])
    out = run_out(st, 1.0)
    gout = run_out_backward(st, out, 1.0)
    ws = torch.empty(N.block_norm_backward_workspace_size(200, 2880, 50), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        N.block_norm_out(st["y"], st["r"], st["w"], st["gate"], 50, 1.0, st["w_next"], EPS, out["out"], out["rstd"], out["xn"],
                         out["rstd_next"])
        N.block_norm_out_backward(st["dout"], st["dxn"], st["y"], out["out"], st["w"], st["gate"], 50, 1.0, st["w_next"],
                                  out["rstd"], out["rstd_next"], gout["dr"], gout["dy"], gout["dw"], gout["dgate"],
                                  gout["dw_next"], ws)
    for _ in range(3):
        for v in list(out.values()) + list(gout.values()):
            v.fill_(float("nan"))
        graph.replay()
    torch.cuda.synchronize()
    for name in want:
        assert torch.equal(want[name], out[name]), name
    for name in gwant:
        assert torch.equal(gwant[name], gout[name]), name


def test_refusals():
    st = inputs(4, 64, torch.bfloat16, 2, seed=8)
    fwd = run_out(st, 1.0)
    ok = dict(y=st["y"], r=st["r"], w=st["w"], gate=st["gate"], gate_rows=2, alpha=1.0, w_next=st["w_next"], eps=EPS,
              out=fwd["out"], rstd=fwd["rstd"], xn=fwd["xn"], rstd_next=fwd["rstd_next"])
    for change in ({"gate_rows": 0}, {"gate_rows": 3, "gate": st["gate"][:1]}, {"gate": None}, {"r": st["r"].half()},
                   {"out": fwd["out"].float()}, {"y": st["y"][:, ::2]}, {"w": st["w"].bfloat16()}, {"w": st["w"].cpu()},
                   {"xn": None}, {"rstd": fwd["rstd"][:3]}, {"y": st["y"].t()}):
        with pytest.raises(ValueError):
            N.block_norm_out(**{**ok, **change})
    for change in ({"eps": -1.0}, {"eps": float("nan")}, {"eps": float("inf")}):
        with pytest.raises(N.MoEError):
            N.block_norm_out(**{**ok, **change})
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(N.MoEError) as e:
        N.block_norm_in_backward(st["dxn"], None, st["r"], st["w"], fwd["rstd"], torch.empty_like(st["r"]),
                                 torch.empty_like(st["w"]), ws)
    assert e.value.status == N.MOE_ERR_WORKSPACE


def test_rows_past_two_to_the_31_elements():
    """The last rows of a stream of more than 2^31 elements, against the formulas."""
    d = 8192
    T = 2 ** 31 // d + 5
    g = torch.Generator(device="cuda").manual_seed(11)
    y, dout = (torch.empty(T, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    w = 1 + 0.3 * torch.randn(d, device="cuda", generator=g)
    xn, dr, dy = torch.empty_like(y), torch.empty_like(y), torch.empty_like(y)
    rstd, dw = torch.empty(T, device="cuda"), torch.empty(d, device="cuda")
    N.block_norm_in(y, w, EPS, xn, rstd)
    ws = torch.empty(N.block_norm_backward_workspace_size(T, d), dtype=torch.uint8, device="cuda")
    N.block_norm_out_backward(dout, None, y, None, w, None, 0, 0.5, None, rstd, None, dr, dy, dw, None, None, ws)
    a = slice(T - 4, T)
    y, dout, w, rs = y[a].double(), dout[a].double(), w.double(), f64_norm(y[a].double())
    near(rstd[a], rs[:, 0], rs[:, 0], "rstd")
    near(xn[a], y * rs * w, (y * rs * w).abs(), "xn")
    near(dr[a], 0.5 * dout, 0.5 * dout.abs(), "dr")
    rs = rstd[a].double()[:, None]
    hat, dn = y * rs, dout * w
    near(dy[a], rs * (dn - hat * (dn * hat).mean(1, keepdim=True)),
         rs * (dn.abs() + hat.abs() * (dn * hat).abs().mean(1, keepdim=True)), "dy")
