"""The sparse MoE feed-forward layer as a sequence of C-ABI calls.

Blog post "Mixture of Experts (MoEs) in Transformers": the layer keeps the transformer backbone and
replaces the dense feed-forward block with experts and a router (section "From Dense to Sparse"); at
run time it dispatches tokens to their selected experts, runs the projections, applies the routing
weights and collects the results in token order (section "Expert Backend"), here the grouped_mm way:
sort by expert id, group, one grouped GEMM over all experts.

This module owns device buffers (allocated with torch; the library never allocates) and calls the five
library entry points in order on one stream. It does no arithmetic of its own.
"""
from __future__ import annotations

import copy

import torch

from . import _native as N


def _encode_mxfp4(*ws):
    """bf16 weights [G_i, N, K] (one or more tensors, stacked on dim 0 in the order given) -> (codes
    [sum G_i, N, K/2], scales [sum G_i, K/32, N]) on the weights' device."""
    G = sum(w.shape[0] for w in ws)
    _, Nr, K = ws[0].shape
    q = torch.empty(G, Nr, K // 2, dtype=torch.uint8, device=ws[0].device)
    s = torch.empty(G, K // 32, Nr, dtype=torch.uint8, device=ws[0].device)
    g = 0
    for w in ws:
        N.mxfp4_quantize(w, q[g:g + w.shape[0]], s[g:g + w.shape[0]])
        g += w.shape[0]
    return q, s


def _encode_fp8(w, halves: int):
    """bf16 weights [G, N, K] -> (e4m3 [G, N, K], scales per 128 x 128 block [G, halves, ceil(N/halves/128), ceil(K/128)]);
    halves = 2 for gate|up, which are blocked apart. A pair (e4m3, scales) is taken as it is."""
    G, n, K = (w[0] if isinstance(w, tuple) else w).shape
    shape = (G, halves, N.fp8_blocks(n // halves), N.fp8_blocks(K))
    shape = shape if halves > 1 else (shape[0],) + shape[2:]
    if isinstance(w, tuple):
        q, s = w
        if q.dtype != N.E4M3 or s.dtype != torch.float32 or tuple(s.shape) != shape:
            raise ValueError(f"want (float8_e4m3fn {(G, n, K)}, float32 {shape}), got ({q.dtype}, {s.dtype} {tuple(s.shape)})")
        return q, s
    q = torch.empty(G, n, K, dtype=N.E4M3, device=w.device)
    s = torch.empty(shape, dtype=torch.float32, device=w.device)
    N.fp8_block_quantize(w.view(G * halves, n // halves, K), q.view(G * halves, n // halves, K),
                         s.view(G * halves, *shape[-2:]))
    return q, s


def _in_use(buffers: dict, stream, device, seen: set, captured: dict, key):
    """Tell the caching allocator that `stream` (None: the device's current one) uses these buffers, which were allocated on whichever stream was current: when they are
    dropped (for another number of tokens), their memory is not given out while that stream's work is still to come. `seen`: streams
    it has been told of. While a CUDA graph is captured they are entered in `captured` under their key and never dropped: the graph's
    replays write them."""
    raw = stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(device.index)
    if raw != 0 and torch.cuda.is_current_stream_capturing():  # (the default stream cannot be captured)
        captured[key] = (buffers, seen)
    if raw in seen:
        return
    seen.add(raw)
    stream = stream if stream is not None else torch.cuda.current_stream(device)
    for v in buffers.values():
        for t in v if isinstance(v, tuple) else (v,):  # (encoded rows: values and scales)
            if t is not None:
                t.record_stream(stream)


def _overlap(a, b) -> bool:
    """Whether two contiguous tensors share memory."""
    a0, b0 = a.data_ptr(), b.data_ptr()
    return a0 < b0 + b.nbytes and b0 < a0 + a.nbytes


class MoEFFN:
    """One MoE feed-forward layer with packed expert weights.

    w_router [E, d] fp32; w_gateup [E, 2f, d] bf16 (gate rows, then up rows); w_down [E, d, f] bf16;
    bias [E] fp32 or None; optional shared expert w_gateup_shared [2fs, d], w_down_shared [d, fs].
    weights: "bf16" keeps the expert weights as given; "mxfp4" encodes them once (moe_mxfp4_quantize, 4.25 bits
    per weight) and the layer then computes with the weights the encoding represents, through the MXFP4 grouped
    GEMMs; the bf16 tensors are not kept. "fp8" encodes them once as e4m3 with a scale per 128 x 128 block
    (moe_fp8_block_quantize), or takes them so encoded, each weight given as a pair (e4m3 values, scales); the rows
    that enter each product are encoded on the way, with a scale per 128 columns (moe_fp8_row_quantize). d and f are
    multiples of 16 then. Half the memory of bf16 weights, and faster where their bytes bound a call (decoding); a prompt's
    products take as long as in bf16.
    fused: with bf16 weights and groups of 128 rows or more on average (prefill), let the dispatch and the
    collect steps ride in the grouped GEMMs: the gate|up GEMM reads its rows straight from x through perm_src
    (moe_grouped_gemm_gateup_gather) instead of a grouped copy x_perm made by moe_permute, and the down GEMM's
    epilogue does the weighted combine (moe_grouped_gemm_down_combine). Same results, bit for bit; the backward
    pass then gathers x_perm itself. Off by default: on B200 the separate gather and combine kernels are faster
    (the per-row gather loads and the combine's arrival counting slow the GEMMs by more than the two kernels
    take).
    few: with bf16 weights and 1 to 16 tokens, run the whole layer in two kernels (moe_few_tokens) instead of eight. Measured on six
    shapes: faster on all of them up to 12 tokens (one token on 4 of 32 experts of 2880 x 2880 47 against 123 us, 12 tokens 221
    against 239), at 16 from 1.45 times as fast (2 of 8 experts of 4096 x 14336, 458 against 664 us) to 8 % slower; at 20 to 32
    tokens, which the kernels also take, the grouped GEMMs are up to 1.8 times as fast. Results agree to rounding, not bit for bit
    (the routing weight is applied before h is rounded, and the experts' outputs are summed without rounding). Not used by a
    training forward, whose backward pass reads the separate calls' buffers.
    """

    few = False

    def __init__(self, w_router, w_gateup, w_down, k: int, route: str = "topk_softmax", bias=None,
                 w_gateup_shared=None, w_down_shared=None, weights: str = "bf16", fused: bool = False,
                 few: bool = False):
        self.E, self.d = w_router.shape
        first = w_gateup[0] if isinstance(w_gateup, tuple) else w_gateup
        self.f = first.shape[1] // 2
        self.k = k
        self.route = route
        if route not in N.ROUTE_MODES:
            raise ValueError(f"unknown routing mode {route!r}")
        if weights not in ("bf16", "mxfp4", "fp8"):
            raise ValueError(f"unknown weight format {weights!r}")
        if isinstance(w_gateup, tuple) and weights != "fp8":
            raise ValueError('encoded weights are for weights="fp8"')
        self.weights = weights
        self.fused = fused
        self.few = few
        self._x_perm_valid = False
        self.w_router, self.w_gateup, self.w_down, self.bias = w_router, w_gateup, w_down, bias
        self.w_gateup_shared, self.w_down_shared = w_gateup_shared, w_down_shared
        shared = w_gateup_shared[0] if isinstance(w_gateup_shared, tuple) else w_gateup_shared
        self.shared_f = shared.shape[-2] // 2 if shared is not None else 0
        self.device = first.device
        # MXFP4 with a shared expert as wide as a routed one: its weights are encoded as group E of the routed
        # tensors; for decode-sized T (_fold) its T rows (x itself) follow the R routed rows, and the routed GEMM
        # launches compute it as one more group, spread over every SM like the rest (on its own it is one group of
        # T rows, which the MXFP4 kernels run on a few SMs: 139 us on the decode layer's side stream, half of it
        # after the routing and grouping beside it; folded in, it adds 3.6% to the routed GEMMs' work, and on one
        # box the decode layer took 1.206-1.212 ms against 1.210-1.216 ms, at a power-capped clock 2-3% lower)
        self.fold_shared = weights == "mxfp4" and self.shared_f == self.f and self.shared_f > 0
        if weights == "mxfp4":
            E = self.E
            if self.fold_shared:  # the routed and shared names are views of the stacked tensors
                qg, sg = self.mx_gateup_all = _encode_mxfp4(w_gateup, w_gateup_shared.unsqueeze(0))
                qd, sd = self.mx_down_all = _encode_mxfp4(w_down, w_down_shared.unsqueeze(0))
                self.mx_gateup, self.mx_down = (qg[:E], sg[:E]), (qd[:E], sd[:E])
                self.mx_gateup_shared, self.mx_down_shared = (qg[E:], sg[E:]), (qd[E:], sd[E:])
            else:
                self.mx_gateup = _encode_mxfp4(w_gateup)
                self.mx_down = _encode_mxfp4(w_down)
                if self.shared_f:
                    self.mx_gateup_shared = _encode_mxfp4(w_gateup_shared.unsqueeze(0))
                    self.mx_down_shared = _encode_mxfp4(w_down_shared.unsqueeze(0))
            self.w_gateup = self.w_down = self.w_gateup_shared = self.w_down_shared = None
        elif weights == "fp8":
            self.f8 = {"gateup": _encode_fp8(w_gateup, 2), "down": _encode_fp8(w_down, 1)}
            if self.shared_f:  # one group; given encoded, a pair has that group's dimension
                one = lambda w: w if isinstance(w, tuple) else w.unsqueeze(0)  # noqa: E731
                self.f8["gateup_shared"] = _encode_fp8(one(w_gateup_shared), 2)
                self.f8["down_shared"] = _encode_fp8(one(w_down_shared), 1)
            self.w_gateup = self.w_down = self.w_gateup_shared = self.w_down_shared = None
        self._T = None
        self.buf = {}
        self._captured, self._gcaptured = {}, {}  # buffers that CUDA graphs were captured with, by T
        # the tensor-core router (E <= 128) reads W_r as three bf16 pieces: split once here, not in every call
        self.w_pieces = None
        if self.E <= 128:
            self.w_pieces = torch.empty(3, self.E, self.d, dtype=torch.bfloat16, device=self.device)
            self.refresh_router()
        # the shared expert depends only on x: it runs on a side stream, beside routing and grouping (which
        # leave most SMs free), and the routed GEMMs wait for it
        self._side = torch.cuda.Stream(self.device) if self.shared_f else None

    def sibling(self) -> "MoEFFN":
        """Another layer over the same weights (nothing is copied or re-encoded) with its own intermediate buffers
        and side stream, so that two calls can be in flight at once."""
        twin = copy.copy(self)
        twin.buf, twin._T = {}, None
        twin._captured, twin._gcaptured = {}, {}
        twin._gbuf, twin._gT, twin._gu_saved = None, None, False  # its own backward buffers too
        twin._side = torch.cuda.Stream(self.device) if self.shared_f else None
        return twin

    def refresh_router(self):
        """Re-split the router weights; call after changing w_router in place."""
        if self.w_pieces is not None:
            N.router_split_weights(self.w_router, self.w_pieces)

    def buffers(self, T: int) -> dict:
        """Every intermediate the layer writes, for T tokens: those of the last call, or of a CUDA graph captured with T tokens, else
        new ones."""
        if self._T == T:
            return self.buf
        if T in self._captured:
            (self.buf, self._seen), self._T = self._captured[T], T
            return self.buf
        dev, E, d, f, k = self.device, self.E, self.d, self.f, self.k
        R = T * k
        i32, f32, bf = torch.int32, torch.float32, torch.bfloat16
        b = {
            "logits": torch.empty(T, E, dtype=f32, device=dev),
            "topk_idx": torch.empty(T, k, dtype=i32, device=dev),
            "topk_w": torch.empty(T, k, dtype=f32, device=dev),
            "counts": torch.empty(E, dtype=i32, device=dev),
            "offsets": torch.empty(E + 1, dtype=i32, device=dev),
            "perm_src": torch.empty(R, dtype=i32, device=dev),
            "inv_perm": torch.empty(R, dtype=i32, device=dev),
            "x_perm": torch.empty(R if self.weights != "fp8" else 0, d, dtype=bf, device=dev),
            "h": torch.empty(R, f, dtype=bf, device=dev),
            "y_perm": torch.empty(R, d, dtype=bf, device=dev),
            "ws": torch.empty(max(N.permute_workspace_size(T, E, k), 256), dtype=torch.uint8, device=dev),
            "combine_ws": torch.empty(max(N.grouped_gemm_down_combine_workspace_size(T, d), 256), dtype=torch.uint8,
                                      device=dev),
            "y": torch.empty(T, d, dtype=bf, device=dev),
        }
        if self._fold(T):
            # the R routed rows, then the shared expert's T rows (group E, offsets[E + 1] = R + T); the routed-only
            # names are views of the first R rows and E + 1 offsets
            b["offsets_all"] = torch.full((E + 2,), R + T, dtype=i32, device=dev)
            b["x_perm_all"] = torch.empty(R + T, d, dtype=bf, device=dev)
            b["h_all"] = torch.empty(R + T, f, dtype=bf, device=dev)
            b["y_perm_all"] = torch.empty(R + T, d, dtype=bf, device=dev)
            b["offsets"] = b["offsets_all"][:E + 1]
            b["x_perm"], b["h"], b["y_perm"] = b["x_perm_all"][:R], b["h_all"][:R], b["y_perm_all"][:R]
            b["shared_rows"] = torch.arange(T, dtype=i32, device=dev)
            b["shared"] = b["y_perm_all"][R:]
        elif self.shared_f:
            b["shared_offsets"] = torch.tensor([0, T], dtype=i32, device=dev)
            b["h_shared"] = torch.empty(T, self.shared_f, dtype=bf, device=dev)
            b["shared"] = torch.empty(T, d, dtype=bf, device=dev)
        if self.weights == "fp8":  # the rows entering each product: e4m3 values and scales
            def rows(n, K):
                return (torch.empty(n, K, dtype=N.E4M3, device=dev), torch.empty(N.fp8_blocks(K), n, dtype=f32, device=dev))
            b["xq"], b["hq"] = rows(R, d), rows(R, f)
            if self.shared_f:
                b["xq_shared"], b["hq_shared"] = rows(T, d), rows(T, self.shared_f)
        self.buf, self._T, self._seen = b, T, set()
        return b

    @staticmethod
    def _made_on(stream, there: bool, make, *args):
        """make(*args), on `stream` unless it is there already: some buffers have first values, and the transposed weights are copies."""
        if there:
            return make(*args)
        with torch.cuda.stream(stream):
            return make(*args)

    def output_there(self, T: int):
        """The output buffer that forward() will write for T tokens, if it is there already, else None."""
        if self._T == T:
            return self.buf["y"]
        return self._captured[T][0]["y"] if T in self._captured else None

    def forward(self, x, stream=None, timing=None, train: bool = False):
        """y = MoE(x) for x [T, d] bf16 on the GPU. Returns the layer's output buffer [T, d] (bf16).

        train: keep the routed experts' gate|up pre-activations (moe_grouped_gemm_gateup_save, bf16 weights) so
        that the following backward() does not recompute them; the output is the same.

        timing: optional dict; if given, a (start, end) pair of CUDA events is recorded around each stage
        ("route", "permute", "gateup", "down", "combine" on the layer's stream; "shared", the always-on
        expert, on the side stream where it overlaps routing and grouping: its GEMMs, or, folded into the routed
        GEMMs (MXFP4), the copy of its rows; "few" alone, the whole layer, where the few-token kernels run).
        """
        T = x.shape[0]
        s = stream if stream is not None else torch.cuda.current_stream(x.device)
        b = self._made_on(s, self._T == T, self.buffers, T)
        few = self._few(T) and not train
        if few and "few_ws" not in b:
            n = N.few_tokens_workspace_size(T, self.d, self.f, self.shared_f, self.E, self.k)
            b["few_ws"] = torch.empty(n, dtype=torch.uint8, device=self.device)
            self._seen.clear()
        _in_use(b, s, self.device, self._seen, self._captured, T)
        self._x = x  # the backward pass reads the forward's input and intermediates

        def mark(name, first):
            if timing is None:
                return
            if first:
                timing[name] = (torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True))
            timing[name][0 if first else 1].record(s)

        if few:
            mark("few", True)
            N.few_tokens(x, self.w_router, self.bias, self.w_gateup, self.w_down, self.w_gateup_shared, self.w_down_shared,
                         self.k, self.route, b["logits"], b["topk_idx"], b["topk_w"], b["y"], b["few_ws"], s)
            mark("few", False)
            self._x = None  # nothing is kept for a backward pass
            return b["y"]
        shared = None
        if self.shared_f:
            side = self._side
            x_ready = torch.cuda.Event()
            x_ready.record(s)
            side.wait_event(x_ready)  # also orders after the previous call's combine, which read `shared`
            if timing is not None:
                timing["shared"] = (torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True))
                timing["shared"][0].record(side)
            if self._fold(T):  # its rows after the routed ones; the routed GEMMs compute it
                N.gather_rows(x, b["shared_rows"], b["x_perm_all"][T * self.k:], side)
            else:
                if self.weights == "fp8":
                    N.fp8_row_quantize(x, None, *b["xq_shared"], side)
                self._gateup(x, "shared", b["shared_offsets"], b["h_shared"], side)
                self._down(b["h_shared"], "shared", b["shared_offsets"], b["shared"], side)
            shared_done = torch.cuda.Event()
            shared_done.record(side)
            if timing is not None:
                timing["shared"][1].record(side)
            shared = b["shared"]
        mark("route", True)
        if self.w_pieces is not None:
            N.route_topk_split(x, self.w_router, self.w_pieces, self.bias, self.k, self.route, b["logits"],
                               b["topk_idx"], b["topk_w"], s)
        else:
            N.route_topk(x, self.w_router, self.bias, self.k, self.route, b["logits"], b["topk_idx"], b["topk_w"], s)
        mark("route", False)
        fused = self._fused(T) and not train  # the saving gate|up GEMM reads x_perm
        save = train and self.weights == "bf16"
        self._gu_saved = False
        mark("permute", True)
        if fused or self.weights == "fp8":  # grouping only; the gate|up GEMM, or the encoder, gathers its rows from x
            N.permute(None, b["topk_idx"], self.E, b["counts"], b["offsets"], b["perm_src"], b["inv_perm"], None,
                      b["ws"], s)
            if not fused:
                N.fp8_row_quantize(x, b["perm_src"], *b["xq"], s)
        else:
            N.permute(x, b["topk_idx"], self.E, b["counts"], b["offsets"], b["perm_src"], b["inv_perm"], b["x_perm"],
                      b["ws"], s)
        self._x_perm_valid = not fused and self.weights != "fp8"
        mark("permute", False)
        if shared is not None:
            # the routed GEMMs are persistent kernels sized to every SM: they start once the shared expert is done
            # (or, folded, its rows are in place)
            s.wait_event(shared_done)
        mark("gateup", True)
        if fused:
            N.grouped_gemm_gateup_gather(x, b["perm_src"], self.w_gateup, b["offsets"], b["h"], None, s)
        elif save:
            g = self._made_on(s, getattr(self, "_gT", None) == T, self._grad_buffers, T)
            _in_use(g, s, self.device, self._gseen, self._gcaptured, T)
            N.grouped_gemm_gateup_save(b["x_perm"], self.w_gateup, b["offsets"], b["h"], g["gu"], s)
            self._gu_saved = True
        else:
            self.routed_gateup(b, s)
        mark("gateup", False)
        mark("down", True)
        if fused:  # y_perm and, in the same kernel, y
            N.grouped_gemm_down_combine(b["h"], self.w_down, b["offsets"], b["perm_src"], b["inv_perm"],
                                        b["topk_w"], shared, b["y_perm"], b["y"], b["combine_ws"], s)
            mark("down", False)
            return b["y"]
        self.routed_down(b, s)
        mark("down", False)
        mark("combine", True)
        N.unpermute_combine(b["y_perm"], b["inv_perm"], b["topk_w"], shared, b["y"], s)
        mark("combine", False)
        return b["y"]

    __call__ = forward

    def _fused(self, T: int) -> bool:
        """Whether forward() folds the row gather into the gate|up GEMM and the combine into the down GEMM for
        T tokens."""
        return (self.fused and self.weights == "bf16" and T > 0
                and N.grouped_gemm_gateup_gather_workspace_size(self.E, T * self.k, self.d) == 0)

    def _few(self, T: int) -> bool:
        """Whether forward() runs the whole layer in the few-token kernels for T tokens."""
        return self.few and self.weights == "bf16" and 0 < T <= 16

    def _fold(self, T: int) -> bool:
        """Whether forward() computes the shared expert inside the routed MXFP4 GEMMs for T tokens: when the
        R + T rows stay within the decode kernel's range (at most 8 rows per group on average, as the library's
        dispatch decides), so that the routed experts keep that kernel, and E + 1 groups are within the grouped
        GEMMs' limit of 1024."""
        return (self.fold_shared and T > 0 and T * self.k + T <= 8 * (self.E + 1)
                and self.E + 1 <= N.MAX_GEMM_GROUPS)

    def routed_gateup(self, b, stream):
        """The routed gate|up GEMM of forward() on buffers b (with the folded shared expert as group E)."""
        if "x_perm_all" in b:
            q, sc = self.mx_gateup_all
            N.grouped_gemm_gateup_mxfp4(b["x_perm_all"], q, sc, b["offsets_all"], b["h_all"], stream)
        else:
            self._gateup(b["x_perm"], "routed", b["offsets"], b["h"], stream)

    def routed_down(self, b, stream):
        """The routed down GEMM of forward() on buffers b (with the folded shared expert as group E)."""
        if "x_perm_all" in b:
            q, sc = self.mx_down_all
            N.grouped_gemm_down_mxfp4(b["h_all"], q, sc, b["offsets_all"], b["y_perm_all"], stream)
        else:
            self._down(b["h"], "routed", b["offsets"], b["y_perm"], stream)

    def _gateup(self, a, which, offsets, h, stream):
        if self.weights == "mxfp4":
            q, sc = self.mx_gateup if which == "routed" else self.mx_gateup_shared
            N.grouped_gemm_gateup_mxfp4(a, q, sc, offsets, h, stream)
        elif self.weights == "fp8":  # of the rows encoded before
            shared = which == "shared"
            N.grouped_gemm_gateup_fp8(*self.buf["xq_shared" if shared else "xq"],
                                      *self.f8["gateup_shared" if shared else "gateup"], offsets, h, stream)
        else:
            w = self.w_gateup if which == "routed" else self.w_gateup_shared.unsqueeze(0)
            N.grouped_gemm_gateup(a, w, offsets, h, stream)

    def _down(self, h, which, offsets, y, stream):
        if self.weights == "mxfp4":
            q, sc = self.mx_down if which == "routed" else self.mx_down_shared
            N.grouped_gemm_down_mxfp4(h, q, sc, offsets, y, stream)
        elif self.weights == "fp8":
            shared = which == "shared"
            hq = self.buf["hq_shared" if shared else "hq"]
            N.fp8_row_quantize(h, None, *hq, stream)
            N.grouped_gemm_down_fp8(*hq, *self.f8["down_shared" if shared else "down"], offsets, y, stream)
        else:
            w = self.w_down if which == "routed" else self.w_down_shared.unsqueeze(0)
            N.grouped_gemm_down(h, w, offsets, y, stream)

    # ---- training: gradients of the last forward() call ----------------------------------------------------

    def _transposed(self):
        """Per-expert transposed weight copies for the backward GEMMs, made once (call refresh_backward after
        changing the weights in place)."""
        if getattr(self, "_wt", None) is None:
            if self.weights != "bf16":
                raise NotImplementedError("the backward pass needs the bf16 expert weights")
            E, d, f = self.E, self.d, self.f
            wt = {"down": torch.empty(E, f, d, dtype=torch.bfloat16, device=self.device),
                  "gateup": torch.empty(E, d, 2 * f, dtype=torch.bfloat16, device=self.device)}
            N.transpose_weights(self.w_down, wt["down"])
            N.transpose_weights(self.w_gateup, wt["gateup"])
            if self.shared_f:
                fs = self.shared_f
                wt["down_shared"] = torch.empty(1, fs, d, dtype=torch.bfloat16, device=self.device)
                wt["gateup_shared"] = torch.empty(1, d, 2 * fs, dtype=torch.bfloat16, device=self.device)
                N.transpose_weights(self.w_down_shared.unsqueeze(0), wt["down_shared"])
                N.transpose_weights(self.w_gateup_shared.unsqueeze(0), wt["gateup_shared"])
            self._wt = wt
        return self._wt

    def refresh_backward(self):
        """Drop the transposed weight copies (rebuilt by the next backward)."""
        self._wt = None

    def _grad_buffers(self, T: int) -> dict:
        if getattr(self, "_gT", None) == T:
            return self._gbuf
        if T in self._gcaptured:
            (self._gbuf, self._gseen), self._gT = self._gcaptured[T], T
            return self._gbuf
        dev, E, d, f, k = self.device, self.E, self.d, self.f, self.k
        R = T * k
        bf, f32 = torch.bfloat16, torch.float32
        g = {"dy_perm": torch.empty(R, d, dtype=bf, device=dev), "dtopk_w": torch.empty(T, k, dtype=f32, device=dev),
             "dh": torch.empty(R, f, dtype=bf, device=dev), "gu": torch.empty(R, 2 * f, dtype=bf, device=dev),
             "dgu": torch.empty(R, 2 * f, dtype=bf, device=dev), "dx_perm": torch.empty(R, d, dtype=bf, device=dev),
             "dx_router": torch.empty(T, d, dtype=bf, device=dev), "dx": torch.empty(T, d, dtype=bf, device=dev),
             "ones": torch.ones(T, k, dtype=f32, device=dev),
             "router_ws": torch.empty(max(N.router_backward_workspace_size(T, d, E, k), 256), dtype=torch.uint8,
                                      device=dev),
             "dw_router": torch.empty(E, d, dtype=f32, device=dev),
             "dbias": torch.empty(E, dtype=f32, device=dev) if self.bias is not None else None,
             "dw_down": torch.empty(E, d, f, dtype=f32, device=dev),
             "dw_gateup": torch.empty(E, 2 * f, d, dtype=f32, device=dev)}
        wsz = max(N.grouped_weight_grad_workspace_size(max(R, 1), E, d, f),
                  N.grouped_weight_grad_workspace_size(max(R, 1), E, 2 * f, d))
        if self.shared_f:
            fs = self.shared_f
            g.update({"dh_s": torch.empty(T, fs, dtype=bf, device=dev), "gu_s": torch.empty(T, 2 * fs, dtype=bf, device=dev),
                      "dgu_s": torch.empty(T, 2 * fs, dtype=bf, device=dev), "dx_s": torch.empty(T, d, dtype=bf, device=dev),
                      "dw_down_shared": torch.empty(1, d, fs, dtype=f32, device=dev),
                      "dw_gateup_shared": torch.empty(1, 2 * fs, d, dtype=f32, device=dev)})
            wsz = max(wsz, N.grouped_weight_grad_workspace_size(max(T, 1), 1, d, fs),
                      N.grouped_weight_grad_workspace_size(max(T, 1), 1, 2 * fs, d))
        g["wgrad_ws"] = torch.empty(max(wsz, 256), dtype=torch.uint8, device=dev)
        self._gbuf, self._gT, self._gseen = g, T, set()
        return g

    def backward(self, dy, stream=None, weight_grads: bool = True, timing=None) -> dict:
        """Gradients of the last forward() call for the upstream gradient dy [T, d] (bf16), the top-k selection
        held fixed. Returns a dict of device tensors owned by the layer (overwritten by the next backward):
        dx [T, d] bf16 (experts and router), dtopk_w [T, k] (routing weights), dw_router [E, d], dbias [E] (with
        a router bias), and with weight_grads dw_gateup [E, 2f, d], dw_down [E, d, f] (fp32), plus the shared
        expert's dw_gateup_shared [1, 2fs, d] and dw_down_shared [1, d, fs].
        timing: optional dict; if given, (start, end) CUDA events are recorded around each stage ("bwd_permute",
        "bwd_dh", "bwd_preact", "bwd_swiglu", "bwd_dx_perm", "bwd_shared", "bwd_router", "bwd_combine", "bwd_dw_down",
        "bwd_dw_gateup", "bwd_dw_shared")."""
        T = dy.shape[0]
        if self._T != T or getattr(self, "_x", None) is None or self._x.shape[0] != T:
            raise RuntimeError("backward() follows a forward() over the same tokens")
        s = stream if stream is not None else torch.cuda.current_stream(dy.device)
        b = self.buf
        wt = self._made_on(s, getattr(self, "_wt", None) is not None, self._transposed)
        g = self._made_on(s, getattr(self, "_gT", None) == T, self._grad_buffers, T)
        _in_use(b, s, self.device, self._seen, self._captured, T)
        _in_use(g, s, self.device, self._gseen, self._gcaptured, T)
        x = self._x

        def mark(name, first):
            if timing is None:
                return
            if first:
                timing[name] = (torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True))
            timing[name][0 if first else 1].record(s)

        mark("bwd_permute", True)
        N.permute_backward(dy, b["inv_perm"], b["topk_w"], b["y_perm"], g["dy_perm"], g["dtopk_w"], s)
        mark("bwd_permute", False)
        mark("bwd_dh", True)
        N.grouped_gemm_down(g["dy_perm"], wt["down"], b["offsets"], g["dh"], s)
        mark("bwd_dh", False)
        mark("bwd_preact", True)
        if not self._x_perm_valid:  # the forward gathered its rows inside the GEMM: x_perm is made here
            N.gather_rows(x, b["perm_src"], b["x_perm"], s)
            self._x_perm_valid = True
        if not getattr(self, "_gu_saved", False):  # a training forward kept them
            N.grouped_gemm_gateup_preact(b["x_perm"], self.w_gateup, b["offsets"], g["gu"], s)
        mark("bwd_preact", False)
        mark("bwd_swiglu", True)
        N.swiglu_backward(g["dh"], g["gu"], g["dgu"], s)
        mark("bwd_swiglu", False)
        mark("bwd_dx_perm", True)
        N.grouped_gemm_down(g["dgu"], wt["gateup"], b["offsets"], g["dx_perm"], s)
        mark("bwd_dx_perm", False)
        addend = None
        if self.shared_f:
            mark("bwd_shared", True)
            so = b["shared_offsets"]
            N.grouped_gemm_down(dy, wt["down_shared"], so, g["dh_s"], s)
            N.grouped_gemm_gateup_preact(x, self.w_gateup_shared.unsqueeze(0), so, g["gu_s"], s)
            N.swiglu_backward(g["dh_s"], g["gu_s"], g["dgu_s"], s)
            N.grouped_gemm_down(g["dgu_s"], wt["gateup_shared"], so, g["dx_s"], s)
            addend = g["dx_s"]
            mark("bwd_shared", False)
        mark("bwd_router", True)
        N.router_backward(x, self.w_router, b["logits"], b["topk_idx"], b["topk_w"], g["dtopk_w"], b["perm_src"],
                          b["inv_perm"], b["offsets"], self.route, g["dx_router"], g["dw_router"], g["dbias"], addend,
                          g["router_ws"], s)
        mark("bwd_router", False)
        mark("bwd_combine", True)
        N.unpermute_combine(g["dx_perm"], b["inv_perm"], g["ones"], g["dx_router"], g["dx"], s)
        mark("bwd_combine", False)
        out = {"dx": g["dx"], "dtopk_w": g["dtopk_w"], "dw_router": g["dw_router"], "dbias": g["dbias"]}
        if weight_grads:
            mark("bwd_dw_down", True)
            N.grouped_weight_grad(g["dy_perm"], b["h"], b["offsets"], g["dw_down"], g["wgrad_ws"], s)
            mark("bwd_dw_down", False)
            mark("bwd_dw_gateup", True)
            N.grouped_weight_grad(g["dgu"], b["x_perm"], b["offsets"], g["dw_gateup"], g["wgrad_ws"], s)
            mark("bwd_dw_gateup", False)
            out["dw_down"], out["dw_gateup"] = g["dw_down"], g["dw_gateup"]
            if self.shared_f:
                mark("bwd_dw_shared", True)
                so = b["shared_offsets"]
                N.grouped_weight_grad(dy, b["h_shared"], so, g["dw_down_shared"], g["wgrad_ws"], s)
                N.grouped_weight_grad(g["dgu_s"], x, so, g["dw_gateup_shared"], g["wgrad_ws"], s)
                mark("bwd_dw_shared", False)
                out["dw_down_shared"], out["dw_gateup_shared"] = g["dw_down_shared"], g["dw_gateup_shared"]
        return out

    def backward_kernel_launches(self, T: int, weight_grads: bool = True, train_forward: bool = False) -> int:
        """Kernels one backward() launches: permute-backward 1, dh 1, pre-activations 1 (none after a training
        forward, which kept them; + 1 gather of x_perm after a forward that folded it into the gate|up GEMM),
        SwiGLU-backward 1, dx_perm 1, router 5, combine 1, and per weight gradient 4 (padded offsets, two
        transposes, the GEMM); the shared expert 4 more (+ 8 with weight gradients)."""
        if T <= 0:
            return 0
        n = 11 + (8 if weight_grads else 0)
        if train_forward:
            n -= 1
        elif self._fused(T):
            n += 1
        if self.shared_f:
            n += 4 + (8 if weight_grads else 0)
        return n

    def kernel_launches(self, T: int, train: bool = False) -> int:
        """Kernels one forward() launches (mirrors the library's dispatch): the router is one kernel when the
        tensor-core path with fused top-k is taken (E <= 128, T >= 2048), else logits + top-k;
        permute 4, gate|up, down, combine 1 each (fused: permute 3, gate|up 1, down with combine 1; train: the
        gate|up that keeps its pre-activations is 1 kernel with 128 rows or more per expert, else 2); the shared
        expert 2 more (1 folded: the copy of its rows). fp8: one more, which encodes h (the gather encodes x), and 2
        more for the shared expert. few: 2 in all where it is taken."""
        if T <= 0:
            return 0
        if self._few(T) and not train:
            return 2
        route = 1 if (self.E <= 128 and T >= 2048) else 2
        if train and self.weights == "bf16":
            body = 4 + 3 + (0 if T * self.k >= 128 * self.E else 1)
        else:
            body = 3 + 2 if self._fused(T) else 4 + 3
        if self.weights == "fp8":
            return route + body + 1 + (4 if self.shared_f else 0)
        return route + body + ((1 if self._fold(T) else 2) if self.shared_f else 0)


class MoEBlock:
    """A residual block around a MoEFFN: the "dense feed-forward block" of a transformer backbone with its norms and residual
    (blog post "Mixture of Experts (MoEs) in Transformers", section "From Dense to Sparse").

        out = alpha * r + gate * (w_out * norm(ffn(w_in * norm(r)))),  norm(v) = v / sqrt(mean(v^2) + eps)

    ffn: the MoEFFN (one to a block while training: backward() reads its intermediates; MoEFFN.sibling() gives another over the same
    weights); w_in, w_out [d] fp32 gains; gate: None, or a learned gate [d] bf16 (forward() also takes one per call); alpha
    the residual scale. The residual stream r is bf16 or fp32 [T, d]. Blocks in a row pass the next one's normed input on, made in
    the same pass as the residual: out, xn = a(r, next_norm=b.w_in); out = b(out, xn=xn).
    """

    def __init__(self, ffn: MoEFFN, w_in, w_out, gate=None, alpha: float = 1.0, eps: float = 1e-6):
        if w_in.shape != (ffn.d,) or w_out.shape != (ffn.d,) or (gate is not None and gate.shape != (ffn.d,)):
            raise ValueError(f"w_in, w_out and gate are vectors of d = {ffn.d}")
        self.ffn, self.w_in, self.w_out, self.gate, self.alpha, self.eps = ffn, w_in, w_out, gate, alpha, eps
        self._key, self._buf, self._call = None, {}, None
        self._gkey, self._gbuf = None, {}
        self._captured, self._gcaptured = {}, {}  # buffers that CUDA graphs were captured with

    def _buffers(self, T: int, dtype) -> dict:
        """Outputs and kept values for T tokens and this type of the stream, kept as MoEFFN.buffers() keeps its own."""
        if self._key == (T, dtype):
            return self._buf
        if (T, dtype) in self._captured:
            self._buf, self._seen = self._captured[T, dtype]
        else:
            d, dev = self.ffn.d, self.ffn.device
            new = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device=dev)  # noqa: E731
            self._buf = {"xn": new(T, d, t=torch.bfloat16), "rstd_in": new(T), "out": new(T, d, t=dtype), "rstd": new(T),
                         "xn_next": new(T, d, t=torch.bfloat16), "rstd_next": new(T)}
            self._seen = set()
        self._key = (T, dtype)
        return self._buf

    def forward(self, r, xn=None, next_norm=None, gate=None, gate_rows: int = 0, train: bool = False, stream=None):
        """The block's output stream [T, d] (a buffer of the block), or with next_norm (the next block's w_in) the pair (output
        stream, its normed input for the next block). xn: this block's normed input, if the block before made it. gate [ceil(T /
        gate_rows), d] bf16: a gate for this call, one row per gate_rows tokens. train: keep what backward() reads; r and xn then may
        not be this block's own outputs, which the call overwrites. r may never be the MoEFFN's own output, nor xn with train."""
        T = r.shape[0]
        self._call = None  # whatever becomes of this call, the kept values of the one before are gone
        b = self._buffers(T, r.dtype)
        _in_use(b, stream, self.ffn.device, self._seen, self._captured, self._key)
        if T > 0:
            reads = (r,) if xn is None or not train else (r, xn)
            y = self.ffn.output_there(T)
            if y is not None and any(_overlap(t, y) for t in reads):
                raise ValueError("r (and xn, with train) may not be the MoEFFN's own output: its forward() overwrites that before it is read")
            if train and any(_overlap(t, b["out"]) or (next_norm is not None and _overlap(t, b["xn_next"])) for t in reads):
                raise ValueError("backward() reads r and xn, and this forward would overwrite them: they are the block's own outputs")
        if gate is None and self.gate is not None:
            gate, gate_rows = self.gate.view(1, -1)[:min(T, 1)], max(T, 1)
        made = xn is None
        if made:
            xn = b["xn"]
            N.block_norm_in(r, self.w_in, self.eps, xn, b["rstd_in"], stream)
        y = self.ffn.forward(xn, stream, train=train)
        N.block_norm_out(y, r, self.w_out, gate, gate_rows, self.alpha, next_norm, self.eps, b["out"], b["rstd"],
                         b["xn_next"] if next_norm is not None else None, b["rstd_next"] if next_norm is not None else None, stream)
        if train:
            self._call = (r, xn, y, gate, gate_rows, next_norm, made)
        return b["out"] if next_norm is None else (b["out"], b["xn_next"])

    __call__ = forward

    def backward(self, dout, dxn=None, weight_grads: bool = True, stream=None) -> dict:
        """Gradients of the last forward(train=True) for the output stream's gradient dout [T, d] (type of the stream) and, where
        the next block's norm was part of it, dxn [T, d] bf16, the gradient of the normed input made for that block.

        Returns MoEFFN.backward's gradients (of the expert and router weights) and "dr" (of r), "dw_out", "dgate" (rows of the gate,
        fp32, or None), "dw_next" (of next_norm, or None), and "dw_in"; where xn was given to forward(), "dw_in" is None and "dxn"
        is xn's gradient, both of which the block before takes: a.backward(g["dr"], g["dxn"])."""
        if self._call is None:
            raise RuntimeError("backward() follows a forward(train=True)")
        r, xn, y, gate, gate_rows, next_norm, made = self._call
        b, f = self._buf, self.ffn
        if f._x is not xn:
            raise RuntimeError("the MoEFFN has run another forward() since: its intermediates are gone (blocks in flight at once, or calls "
                               "beside them, need a MoEFFN of their own: sibling() gives one over the same weights)")
        T, d = r.shape
        key = (T, r.dtype, gate_rows)
        if self._gkey != key and key in self._gcaptured:
            (self._gbuf, self._gseen), self._gkey = self._gcaptured[key], key
        if self._gkey != key:
            new = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device=f.device)  # noqa: E731
            ws = N.block_norm_backward_workspace_size(T, d, gate_rows)
            self._gbuf = {"dr": new(T, d, t=r.dtype), "dy": new(T, d, t=torch.bfloat16), "dw_out": new(d), "dw_in": new(d),
                          "dw_next": new(d), "dgate": new(-(-T // gate_rows), d) if gate_rows else None,
                          "ws": new(max(ws, 16), t=torch.uint8)}
            self._gkey, self._gseen = key, set()
        g = self._gbuf
        _in_use(b, stream, f.device, self._seen, self._captured, self._key)
        _in_use(g, stream, f.device, self._gseen, self._gcaptured, key)
        nxt = next_norm is not None
        N.block_norm_out_backward(dout, dxn, y, b["out"] if nxt else None, self.w_out, gate, gate_rows, self.alpha, next_norm,
                                  b["rstd"], b["rstd_next"] if nxt else None, g["dr"], g["dy"], g["dw_out"], g["dgate"],
                                  g["dw_next"] if nxt else None, g["ws"], stream)
        out = dict(f.backward(g["dy"], weight_grads=weight_grads, stream=stream))
        dx = out.pop("dx")
        if made:
            N.block_norm_in_backward(dx, g["dr"], r, self.w_in, b["rstd_in"], g["dr"], g["dw_in"], g["ws"], stream)
        else:
            out["dxn"] = dx
        out.update(dr=g["dr"], dw_out=g["dw_out"], dgate=g["dgate"], dw_in=g["dw_in"] if made else None,
                   dw_next=g["dw_next"] if nxt else None)
        return out
