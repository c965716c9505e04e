"""Measured calls of the operators around the expert layer: fp8 expert products, the whole layer for few tokens, block norms.

``listed()`` gives the cases, ``draw(rng)`` one more case of the same ranges, ``prepare(case, seed)`` what a program has in
hand before the call, ``run(state)`` one pass and its outputs, ``work(case)`` the bytes and operations the pass cannot do
without, ``exact(case, seed)`` the outputs from the definitions in 64 bits. With ``own`` the pass calls the package's
operators; without it, elementary torch operations in 32 bits.

Operators (``case["op"]``):
  experts_fp8   rows of x gathered and quantized to e4m3 with a scale per 128 values, gate|up + SwiGLU and down products
                with e4m3 expert weights that have a scale per 128 x 128 block
  few_tokens    router, top-k, gate|up, SwiGLU, down and weighted sum of a whole layer for 1 to 32 tokens, bf16 weights
  norm_in       RMS norm in front of a block
  norm_out      RMS norm behind a block, times the gate, plus the scaled residual, then the next block's norm in front
  norm_in_grad, norm_out_grad   their gradients
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
EPS = 1e-6


def listed():
    return [
        # an 8-bit layer of 32 experts answering four streams: one or two rows per expert, weights streamed once
        {"name": "experts_fp8 decode 32e", "op": "experts_fp8", "T": 4, "d": 2880, "f": 2880, "E": 32, "k": 4},
        # wide experts, 16 streams on 64 of them
        {"name": "experts_fp8 decode wide", "op": "experts_fp8", "T": 16, "d": 7168, "f": 2048, "E": 64, "k": 8},
        # many small experts, ragged groups
        {"name": "experts_fp8 many experts", "op": "experts_fp8", "T": 1111, "d": 2048, "f": 768, "E": 128, "k": 8},
        # a prompt of 4096 tokens
        {"name": "experts_fp8 prompt", "op": "experts_fp8", "T": 4096, "d": 2880, "f": 2880, "E": 32, "k": 4},
        # the smallest layer: only latency counts
        {"name": "few_tokens small", "op": "few_tokens", "T": 2, "d": 256, "f": 512, "E": 8, "k": 2, "route": "topk_softmax",
         "fs": 0, "bias": False},
        # one stream on 4 of 32 experts
        {"name": "few_tokens one", "op": "few_tokens", "T": 1, "d": 2880, "f": 2880, "E": 32, "k": 4, "route": "topk_softmax",
         "fs": 0, "bias": True},
        # eight streams on large experts
        {"name": "few_tokens eight", "op": "few_tokens", "T": 8, "d": 4096, "f": 14336, "E": 8, "k": 2,
         "route": "softmax_topk_renorm", "fs": 0, "bias": False},
        # one stream on 8 of 256 experts and a shared one
        {"name": "few_tokens shared", "op": "few_tokens", "T": 1, "d": 7168, "f": 2048, "E": 256, "k": 8,
         "route": "sigmoid_topk_norm", "fs": 2048, "bias": False},
        # the norm in front of a block, one decoding step of 64 streams
        {"name": "norm_in decode", "op": "norm_in", "T": 64, "d": 7168, "res": "bf16"},
        # behind a block of a prompt: a learned gate per channel, bf16 residual, the next norm in the same pass
        {"name": "norm_out prompt", "op": "norm_out", "T": 4096, "d": 2880, "res": "bf16", "gate_rows": 4096, "alpha": 1.0},
        # its gradient, with the residual in 32 bits and one gate row for each sequence of 1000 tokens
        {"name": "norm_out_grad sequences", "op": "norm_out_grad", "T": 8192, "d": 4096, "res": "fp32", "gate_rows": 1000,
         "alpha": 0.5},
        # the gradient of the norm in front of a block
        {"name": "norm_in_grad prompt", "op": "norm_in_grad", "T": 4096, "d": 2880, "res": "bf16"},
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["experts_fp8", "experts_fp8", "few_tokens", "few_tokens", "norm_in", "norm_out", "norm_in_grad",
                     "norm_out_grad", "norm_out_grad"])
    if op == "experts_fp8":
        E = rng.randint(1, 96)
        case = {"op": op, "T": _log_between(rng, 1, 4096), "d": 16 * _log_between(rng, 8, 448),
                "f": 16 * _log_between(rng, 8, 256), "E": E, "k": rng.randint(1, min(E, 8))}
        while case["T"] * case["k"] * case["d"] * case["f"] > 1.2e11 or E * case["d"] * case["f"] > 8e8:
            case["T"], case["f"] = max(1, case["T"] // 2), max(128, case["f"] // 32 * 16)
            if case["T"] == 1 and case["f"] == 128:
                case["E"] = E = max(case["k"], E // 2)
        return case
    if op == "few_tokens":
        E = _log_between(rng, 2, 256)
        case = {"op": op, "T": rng.randint(1, 32), "d": 8 * _log_between(rng, 8, 896), "f": 8 * _log_between(rng, 8, 1024),
                "E": E, "k": rng.randint(1, min(E, 8)),
                "route": rng.choice(["topk_softmax", "softmax_topk_renorm", "sigmoid_topk_norm"]),
                "fs": rng.choice([0, 0, 8 * _log_between(rng, 8, 256)]), "bias": rng.random() < 0.5}
        while E * case["d"] * case["f"] > 1e9:
            case["f"] = max(64, case["f"] // 16 * 8)
            if case["f"] == 64:
                case["d"] = max(64, case["d"] // 16 * 8)
        while case["T"] * case["k"] * case["d"] * case["f"] > 9e8:
            case["T"] = max(1, case["T"] // 2)
            if case["T"] == 1:
                break
        return case
    case = {"op": op, "T": _log_between(rng, 1, 8192), "d": 8 * _log_between(rng, 8, 1024), "res": rng.choice(["bf16", "fp32"])}
    while case["T"] * case["d"] > 8192 * 4096:
        case["T"] //= 2
    if op in ("norm_out", "norm_out_grad"):
        T = case["T"]
        case["gate_rows"] = rng.choice([0, 1, T, _log_between(rng, 1, T)])  # 0: no gate
        case["alpha"] = rng.choice([1.0, 0.22, 0.5])
    return case


# ---- inputs -------------------------------------------------------------------------------------------------------


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    t.normal_(0.0, std, generator=g)
    return t


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _spread(s, n, dim):
    """Each scale along `dim` repeated for its 128 places, cut to n."""
    return s.repeat_interleave(BLOCK, dim).narrow(dim, 0, n)


def _to_e4m3(x, top):
    """448 x / top (top: the largest magnitude of x's block), rounded to e4m3, and the scales top / 448; zero blocks get 1.

    x holds bf16 values, so 448 x has 11 bits and the quotient is an exact tie between two e4m3 values or at least 2^-17
    of its size away from one: a correctly rounded 32-bit quotient of two tensors decides it. (A tensor divided by a Python
    number would be multiplied by the number's rounded reciprocal.)"""
    some = torch.where(top > 0, top, torch.full_like(top, E4M3_MAX))
    return lambda spread: (x * E4M3_MAX / spread(some)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), \
        some / torch.full_like(some, E4M3_MAX)


def _weights_fp8(w):
    """e4m3 values and 128 x 128 block scales of w [N, K] (bf16 values held in 32 bits)."""
    n, k = w.shape
    padded = torch.nn.functional.pad(w, (0, _blocks(k) * BLOCK - k, 0, _blocks(n) * BLOCK - n))
    q, s = _to_e4m3(w, padded.view(_blocks(n), BLOCK, _blocks(k), BLOCK).abs().amax((1, 3)))
    return q(lambda v: _spread(_spread(v, n, 0), k, 1)), s


def _prepare_experts(case, g):
    T, d, f, E, k = (case[n] for n in ("T", "d", "f", "E", "k"))
    x = _normal(g, (T, d))
    x[:, ::61] *= 12  # a few channels of a residual stream are much larger than the others
    # routing: some experts are chosen more often than others
    score = _normal(g, (T, E), dtype=torch.float32) + 0.5 * _normal(g, (1, E), dtype=torch.float32)
    chosen = score.topk(k, dim=1).indices.reshape(-1)
    order = torch.sort(chosen, stable=True).indices
    counts = torch.bincount(chosen, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    wq = {"gateup": torch.empty(E, 2 * f, d, dtype=torch.float8_e4m3fn, device="cuda"),
          "down": torch.empty(E, d, f, dtype=torch.float8_e4m3fn, device="cuda")}
    ws = {"gateup": torch.empty(E, 2, _blocks(f), _blocks(d), device="cuda"),
          "down": torch.empty(E, _blocks(d), _blocks(f), device="cuda")}
    for e in range(E):
        for half in range(2):
            wq["gateup"][e, half * f:(half + 1) * f], ws["gateup"][e, half] = _weights_fp8(_normal(g, (f, d), 0.02).float())
        wq["down"][e], ws["down"][e] = _weights_fp8(_normal(g, (d, f), 0.02).float())
    M = T * k
    u8 = dict(dtype=torch.float8_e4m3fn, device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    return {"x": x, "row_src": (order // k).to(torch.int32), "offsets": offsets, "most": int(counts.max()),
            "wq_gateup": wq["gateup"], "ws_gateup": ws["gateup"], "wq_down": wq["down"], "ws_down": ws["down"],
            "xq": torch.empty(M, d, **u8), "xs": torch.empty(_blocks(d), M, device="cuda"), "h": torch.empty(M, f, **bf),
            "hq": torch.empty(M, f, **u8), "hs": torch.empty(_blocks(f), M, device="cuda"), "y": torch.empty(M, d, **bf)}


def _prepare_few(case, g):
    T, d, f, E, k, fs = (case[n] for n in ("T", "d", "f", "E", "k", "fs"))
    return {"x": _normal(g, (T, d)), "w_router": _normal(g, (E, d), 0.02, torch.float32),
            "bias": _normal(g, (E,), 0.5, torch.float32) if case["bias"] else None,
            "w_gateup": _normal(g, (E, 2 * f, d), 0.02), "w_down": _normal(g, (E, d, f), 0.02),
            "w_gateup_shared": _normal(g, (2 * fs, d), 0.02) if fs else None,
            "w_down_shared": _normal(g, (d, fs), 0.02) if fs else None, "k": k, "route": case["route"],
            "logits": torch.empty(T, E, device="cuda"), "topk_idx": torch.empty(T, k, dtype=torch.int32, device="cuda"),
            "topk_w": torch.empty(T, k, device="cuda"), "y": torch.empty(T, d, dtype=torch.bfloat16, device="cuda")}


def _prepare_norm(case, g):
    T, d = case["T"], case["d"]
    res = torch.float32 if case["res"] == "fp32" else torch.bfloat16
    f32 = dict(dtype=torch.float32, device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")
    r = _normal(g, (T, d), 2.0, torch.float32)
    r[:, ::61] *= 10
    st = {"r": r.to(res), "w": 1 + _normal(g, (d,), 0.2, torch.float32)}
    if case["op"] == "norm_in":
        return st | {"xn": torch.empty(T, d, **bf), "rstd": torch.empty(T, **f32)}
    if case["op"] == "norm_in_grad":
        x = st["r"].double()
        return st | {"dxn": _normal(g, (T, d)), "dres": _normal(g, (T, d), 1.0, res),
                     "rstd": torch.rsqrt(x.square().mean(1) + EPS).float(), "dx": torch.empty(T, d, dtype=res, device="cuda"),
                     "dw": torch.empty(d, **f32)}
    rows = case["gate_rows"]
    st |= {"y": _normal(g, (T, d), 0.7), "w_next": 1 + _normal(g, (d,), 0.2, torch.float32), "gate_rows": rows,
           "alpha": case["alpha"], "gate": _normal(g, (-(-T // rows), d)) if rows else None}
    if case["op"] == "norm_out":
        return st | {"out": torch.empty(T, d, dtype=res, device="cuda"), "rstd": torch.empty(T, **f32),
                     "xn": torch.empty(T, d, **bf), "rstd_next": torch.empty(T, **f32)}
    # what a forward pass kept: its output and both rows of reciprocal norms
    y = st["y"].double()
    rstd = torch.rsqrt(y.square().mean(1) + EPS)
    n = y * rstd[:, None] * st["w"].double()
    if rows:
        n = n * st["gate"].double().repeat_interleave(rows, 0)[:T]
    out = (st["alpha"] * st["r"].double() + n).to(res)
    return st | {"out": out, "rstd": rstd.float(), "rstd_next": torch.rsqrt(out.double().square().mean(1) + EPS).float(),
                 "dout": _normal(g, (T, d), 1.0, res), "dxn": _normal(g, (T, d)),
                 "dr": torch.empty(T, d, dtype=res, device="cuda"), "dy": torch.empty(T, d, **bf),
                 "dw": torch.empty(d, **f32), "dw_next": torch.empty(d, **f32),
                 "dgate": torch.empty(-(-T // rows), d, **f32) if rows else None}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    how = {"experts_fp8": _prepare_experts, "few_tokens": _prepare_few}.get(case["op"], _prepare_norm)
    return {"op": case["op"], **how(case, g)}


# ---- one pass -----------------------------------------------------------------------------------------------------


def _rows_fp8(x):
    """Rows of x [R, K] (bf16 values in 32 bits) as the e4m3 values they become times their scales, 128 values to a scale."""
    R, K = x.shape
    q, s = _to_e4m3(x, torch.nn.functional.pad(x, (0, _blocks(K) * BLOCK - K)).view(R, _blocks(K), BLOCK).abs().amax(2))
    return q(lambda v: _spread(v, K, 1)).float() * _spread(s, K, 1)


def _plain_experts(st):
    E, d = st["wq_down"].shape[:2]
    f = st["wq_down"].shape[2]
    off = st["offsets"].long()
    M = st["row_src"].numel()
    # every group padded to the largest one's rows; rows past a group's end compute from its last row and are left out
    at = off[:-1, None] + torch.arange(st["most"], device="cuda")
    inside = at < off[1:, None]
    x = _rows_fp8(st["x"].float()[st["row_src"].long()])
    at = at.clamp(max=M - 1)
    ws = st["ws_gateup"]
    w = st["wq_gateup"].float().view(E, 2, f, d) * _spread(_spread(ws, f, 2), d, 3)
    gu = torch.bmm(x[at], w.view(E, 2 * f, d).transpose(1, 2))
    del w
    gate, up = gu[..., :f], gu[..., f:]
    h = (gate / (1 + torch.exp(-gate)) * up)[inside].to(torch.bfloat16)
    h = _rows_fp8(h.float())
    w = st["wq_down"].float() * _spread(_spread(st["ws_down"], d, 1), f, 2)
    return torch.bmm(h[at], w.transpose(1, 2))[inside].to(torch.bfloat16)


def _plain_few(st):
    x, k = st["x"].float(), st["k"]
    f = st["w_down"].shape[2]
    logits = x @ st["w_router"].T
    if st["bias"] is not None:
        logits = logits + st["bias"]
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    if st["route"] == "sigmoid_topk_norm":
        w = 1 / (1 + torch.exp(-top))
    else:  # both softmax forms come to the softmax over the chosen experts
        w = torch.exp(top - top[:, :1])
    w = w / w.sum(1, keepdim=True)
    gu = torch.einsum("td,tknd->tkn", x, st["w_gateup"][idx].float())
    h = gu[..., :f] / (1 + torch.exp(-gu[..., :f])) * gu[..., f:]
    y = torch.einsum("tk,tkf,tkdf->td", w, h, st["w_down"][idx].float()) if x.shape[0] * k <= 4 else \
        (w[..., None] * torch.einsum("tkf,tkdf->tkd", h, st["w_down"][idx].float())).sum(1)
    if st["w_gateup_shared"] is not None:
        fs = st["w_down_shared"].shape[1]
        gu = x @ st["w_gateup_shared"].float().T
        y = y + (gu[:, :fs] / (1 + torch.exp(-gu[:, :fs])) * gu[:, fs:]) @ st["w_down_shared"].float().T
    return {"y": y.to(torch.bfloat16), "idx": idx.to(torch.int32), "w": w}


def _gate_of(st, T):
    return st["gate"].float().repeat_interleave(st["gate_rows"], 0)[:T] if st["gate"] is not None else 1.0


def _plain_norm_in(st):
    x = st["r"].float()
    rstd = 1 / torch.sqrt((x * x).mean(1) + EPS)
    return {"xn": (x * rstd[:, None] * st["w"]).to(torch.bfloat16), "rstd": rstd}


def _plain_norm_out(st):
    y, r = st["y"].float(), st["r"].float()
    rstd = 1 / torch.sqrt((y * y).mean(1) + EPS)
    out = st["alpha"] * r + _gate_of(st, y.shape[0]) * (y * rstd[:, None] * st["w"])
    out = out.to(st["r"].dtype)
    o = out.float()
    rstd_next = 1 / torch.sqrt((o * o).mean(1) + EPS)
    return {"out": out, "rstd": rstd, "xn": (o * rstd_next[:, None] * st["w_next"]).to(torch.bfloat16), "rstd_next": rstd_next}


def _plain_norm_in_grad(st):
    x, d, rstd = st["r"].float(), st["dxn"].float(), st["rstd"][:, None]
    hat, dn = x * rstd, d * st["w"]
    dx = st["dres"].float() + rstd * (dn - hat * (dn * hat).mean(1, keepdim=True))
    return {"dx": dx.to(st["r"].dtype), "dw": (d * hat).sum(0)}


def _plain_norm_out_grad(st):
    T, d = st["y"].shape
    rstd, rstd_next, g = st["rstd"][:, None], st["rstd_next"][:, None], _gate_of(st, T)
    hat, d_next = st["out"].float() * rstd_next, st["dxn"].float()
    dn = d_next * st["w_next"]
    dR = st["dout"].float() + rstd_next * (dn - hat * (dn * hat).mean(1, keepdim=True))
    y_hat = st["y"].float() * rstd
    dn = dR * g * st["w"]
    dy = rstd * (dn - y_hat * (dn * y_hat).mean(1, keepdim=True))
    got = {"dr": (st["alpha"] * dR).to(st["r"].dtype), "dy": dy.to(torch.bfloat16), "dw": (dR * g * y_hat).sum(0),
           "dw_next": (d_next * hat).sum(0)}
    if st["gate"] is not None:
        rows, many = st["gate_rows"], st["gate"].shape[0]
        each = torch.nn.functional.pad(dR * st["w"] * y_hat, (0, 0, 0, many * rows - T))
        got["dgate"] = each.view(many, rows, d).sum(1)
    return got


def _own(st):
    import mixture_experts_ffn_11_b200 as moe

    op = st["op"]
    if op == "experts_fp8":
        moe.fp8_row_quantize(st["x"], st["row_src"], st["xq"], st["xs"])
        moe.grouped_gemm_gateup_fp8(st["xq"], st["xs"], st["wq_gateup"], st["ws_gateup"], st["offsets"], st["h"])
        moe.fp8_row_quantize(st["h"], None, st["hq"], st["hs"])
        moe.grouped_gemm_down_fp8(st["hq"], st["hs"], st["wq_down"], st["ws_down"], st["offsets"], st["y"])
        return st["y"]
    if op == "few_tokens":
        if "ws" not in st:  # a program keeps its workspace between calls
            (T, d), (E, _, f) = st["x"].shape, st["w_down"].shape
            fs = st["w_down_shared"].shape[1] if st["w_down_shared"] is not None else 0
            st["ws"] = torch.empty(moe.few_tokens_workspace_size(T, d, f, fs, E, st["k"]), dtype=torch.uint8, device="cuda")
        moe.few_tokens(st["x"], st["w_router"], st["bias"], st["w_gateup"], st["w_down"], st["w_gateup_shared"],
                       st["w_down_shared"], st["k"], st["route"], st["logits"], st["topk_idx"], st["topk_w"], st["y"], st["ws"])
        return {"y": st["y"], "idx": st["topk_idx"], "w": st["topk_w"]}
    if op == "norm_in":
        moe.block_norm_in(st["r"], st["w"], EPS, st["xn"], st["rstd"])
        return {"xn": st["xn"], "rstd": st["rstd"]}
    if op == "norm_out":
        moe.block_norm_out(st["y"], st["r"], st["w"], st["gate"], st["gate_rows"], st["alpha"], st["w_next"], EPS, st["out"],
                           st["rstd"], st["xn"], st["rstd_next"])
        return {n: st[n] for n in ("out", "rstd", "xn", "rstd_next")}
    if "ws" not in st:
        T, d = st["r"].shape
        st["ws"] = torch.empty(moe.block_norm_backward_workspace_size(T, d, st.get("gate_rows", 0)), dtype=torch.uint8,
                               device="cuda")
    if op == "norm_in_grad":
        moe.block_norm_in_backward(st["dxn"], st["dres"], st["r"], st["w"], st["rstd"], st["dx"], st["dw"], st["ws"])
        return {"dx": st["dx"], "dw": st["dw"]}
    moe.block_norm_out_backward(st["dout"], st["dxn"], st["y"], st["out"], st["w"], st["gate"], st["gate_rows"], st["alpha"],
                                st["w_next"], st["rstd"], st["rstd_next"], st["dr"], st["dy"], st["dw"], st["dgate"],
                                st["dw_next"], st["ws"])
    got = {n: st[n] for n in ("dr", "dy", "dw", "dw_next")}
    return got | ({"dgate": st["dgate"]} if st["gate"] is not None else {})


def run(state):
    if own:
        return _own(state)
    return {"experts_fp8": _plain_experts, "few_tokens": _plain_few, "norm_in": _plain_norm_in, "norm_out": _plain_norm_out,
            "norm_in_grad": _plain_norm_in_grad, "norm_out_grad": _plain_norm_out_grad}[state["op"]](state)


# ---- what a pass cannot do without --------------------------------------------------------------------------------


def work(case):
    op, T, d = case["op"], case["T"], case["d"]
    if op in ("experts_fp8", "few_tokens"):
        f, E, k = case["f"], case["E"], case["k"]
        active = E * (1 - (1 - k / E) ** T)  # experts that get a token, on average
        if op == "experts_fp8":
            scales = active * 4 * (2 * _blocks(f) * _blocks(d) + _blocks(d) * _blocks(f))
            return {"bytes": active * 3 * d * f + scales + 2 * T * d + 4 * T * k + 2 * T * k * d, "flops": 6 * T * k * d * f}
        fs = case["fs"]
        return {"bytes": 2 * 3 * d * (active * f + fs) + 4 * E * d + 2 * 2 * T * d + 8 * T * k,
                "flops": T * (6 * d * (k * f + fs) + 2 * E * d)}
    res = 4 if case["res"] == "fp32" else 2
    rows = case.get("gate_rows", 0)
    gate = -(-T // rows) * d if rows else 0
    if op == "norm_in":
        return {"bytes": T * d * (res + 2) + 4 * d + 4 * T, "flops": 4 * T * d}
    if op == "norm_out":
        return {"bytes": T * d * (2 + 2 * res + 2) + 2 * gate + 8 * d + 8 * T, "flops": 11 * T * d}
    if op == "norm_in_grad":
        return {"bytes": T * d * (2 + 3 * res) + 8 * d + 4 * T, "flops": 10 * T * d}
    return {"bytes": T * d * (3 * res + 2 + 2 + 2) + (2 + 4) * gate + 16 * d + 8 * T, "flops": 24 * T * d}


# ---- the definitions in 64 bits -----------------------------------------------------------------------------------


def _e4m3(v):
    """The nearest value with 3 bits after the leading one, exponents from -6, steps of 2^-9 below, at most 448; ties to even."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _exact_rows(x):
    got = torch.empty_like(x)
    for b in range(0, x.shape[1], 128):
        part = x[:, b:b + 128]
        top = part.abs().amax(1, keepdim=True)
        top[top == 0] = 448.0
        got[:, b:b + 128] = _e4m3(part * 448.0 / top) * (top / 448.0).float().double()
    return got


def _exact_weight(q, s):
    w = q.double()
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            w[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128] *= s[i, j].double()
    return w


def _exact_experts(st):
    offsets = st["offsets"].tolist()
    y = torch.zeros(st["row_src"].numel(), st["x"].shape[1], dtype=torch.float64, device="cuda")
    rows = _exact_rows(st["x"].double())
    f = st["wq_down"].shape[2]
    for e in range(len(offsets) - 1):
        lo, hi = offsets[e], offsets[e + 1]
        if lo == hi:
            continue
        a = rows[st["row_src"][lo:hi].long()]
        gate = a @ _exact_weight(st["wq_gateup"][e, :f], st["ws_gateup"][e, 0]).T
        up = a @ _exact_weight(st["wq_gateup"][e, f:], st["ws_gateup"][e, 1]).T
        h = (gate * torch.sigmoid(gate) * up).to(torch.bfloat16).double()  # h is held in bf16 by definition
        y[lo:hi] = _exact_rows(h) @ _exact_weight(st["wq_down"][e], st["ws_down"][e]).T
    return y


def _exact_few(st):
    x, k, f = st["x"].double(), st["k"], st["w_down"].shape[2]
    T, E = x.shape[0], st["w_router"].shape[0]
    y, idx, weights = torch.zeros_like(x), [], []
    silu = lambda v: v * torch.sigmoid(v)  # noqa: E731
    for t in range(T):
        logits = st["w_router"].double() @ x[t]
        if st["bias"] is not None:
            logits = logits + st["bias"].double()
        value = logits.tolist()
        best = sorted(range(E), key=lambda e: (-value[e], e))[:k]
        chosen = logits[best]
        if st["route"] == "softmax_topk_renorm":
            w = torch.softmax(logits, 0)[best]
        elif st["route"] == "sigmoid_topk_norm":
            w = torch.sigmoid(chosen)
        else:
            w = torch.softmax(chosen, 0)
        w = w / w.sum()
        for j, e in enumerate(best):
            gu = st["w_gateup"][e].double() @ x[t]
            y[t] += w[j] * (st["w_down"][e].double() @ (silu(gu[:f]) * gu[f:]))
        if st["w_gateup_shared"] is not None:
            fs = st["w_down_shared"].shape[1]
            gu = st["w_gateup_shared"].double() @ x[t]
            y[t] += st["w_down_shared"].double() @ (silu(gu[:fs]) * gu[fs:])
        idx.append(best)
        weights.append(w)
    return {"y": y, "idx": torch.tensor(idx, dtype=torch.int32), "w": torch.stack(weights)}


def _exact_norm(st):
    op, w, r = st["op"], st["w"].double(), st["r"].double()
    T, d = r.shape
    norm = lambda v: (v.square().sum(1, keepdim=True) / d + EPS) ** -0.5  # noqa: E731
    if op == "norm_in":
        return {"xn": w * (r * norm(r)), "rstd": norm(r)[:, 0]}
    if op == "norm_in_grad":
        c = st["rstd"].double()[:, None]
        dxn = st["dxn"].double()
        s1 = (dxn * w * r).sum(1, keepdim=True)
        return {"dx": st["dres"].double() + c * dxn * w - c ** 3 / d * s1 * r, "dw": (dxn * r * c).sum(0)}
    rows = st["gate_rows"]
    group = torch.arange(T, device="cuda") // max(rows, 1)
    gate = st["gate"].double()[group] if rows else torch.ones_like(r)
    y, w2 = st["y"].double(), st["w_next"].double()
    if op == "norm_out":
        out = st["alpha"] * r + gate * w * (y * norm(y))
        held = out.to(st["r"].dtype).double()  # the next norm reads the residual as it is held
        return {"out": out, "rstd": norm(y)[:, 0], "xn": w2 * (held * norm(held)), "rstd_next": norm(held)[:, 0]}
    a, c = st["rstd"].double()[:, None], st["rstd_next"].double()[:, None]
    out, dxn = st["out"].double(), st["dxn"].double()
    dR = st["dout"].double() + c * dxn * w2 - c ** 3 / d * (dxn * w2 * out).sum(1, keepdim=True) * out
    dn = dR * gate * w
    got = {"dr": st["alpha"] * dR, "dy": a * dn - a ** 3 / d * (dn * y).sum(1, keepdim=True) * y,
           "dw": (dR * gate * y * a).sum(0), "dw_next": (dxn * out * c).sum(0)}
    if rows:
        got["dgate"] = torch.zeros(st["gate"].shape, dtype=torch.float64, device="cuda").index_add_(0, group, dR * w * y * a)
    return got


def exact(case, seed):
    st = prepare(case, seed)
    how = {"experts_fp8": _exact_experts, "few_tokens": _exact_few}.get(case["op"], _exact_norm)
    return how(st)
