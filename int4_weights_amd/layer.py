"""MoE expert layer built on the libmoe entry points.

One forward pass is the data flow of rainlin, "GEMM 执行方式", sec. 4.6:
quantise tokens -> route and pack -> grouped GEMM -> weighted combine, on one
stream with no host synchronisation (the first two steps can run as one call
that quantises while it packs).  Buffers are allocated
once, for a maximum token count, so a forward allocates nothing.
"""

from __future__ import annotations

import torch

from . import _lib as L


class MoeFP8Layer:
    """FP8 block-scaled expert GEMM (1x128 activation scales, 128x128 weight scales)."""

    def __init__(self, w_codes: torch.Tensor, sfw: torch.Tensor, topk: int, max_tokens: int,
                 layout: int = L.LAYOUT_CONTIGUOUS, align_or_max_m: int = 128, expected_m: int = 0,
                 weights_packed: bool = False):
        """weights_packed: w_codes (and any weights passed to gemm()) are in moe_pack_weight_fp8 order."""
        E, N, K = w_codes.shape
        self.wflag = L.WEIGHTS_PACKED if weights_packed else 0
        self.E, self.N, self.K, self.topk = E, N, K, topk
        self.w, self.sfw = w_codes, sfw
        self.layout, self.am = layout, align_or_max_m
        self.expected_m = expected_m
        dev = w_codes.device
        self.max_tokens = max_tokens
        if layout == L.LAYOUT_CONTIGUOUS:
            self.rows_cap = L.moe_packed_rows_cap(max_tokens, topk, E, align_or_max_m)
        else:
            self.rows_cap = E * align_or_max_m
        self.q = torch.empty(max_tokens, K, dtype=torch.uint8, device=dev)
        self.sf = torch.empty(max_tokens, K // 128, dtype=torch.float32, device=dev)
        self.packed = torch.empty(self.rows_cap, K, dtype=torch.uint8, device=dev)
        self.packed_sf = torch.empty(self.rows_cap, K // 128, dtype=torch.float32, device=dev)
        self.counts = torch.zeros(E, dtype=torch.int32, device=dev)
        self.seg_offsets = torch.zeros(E + 1, dtype=torch.int32, device=dev)
        self.m_indices = torch.empty(self.rows_cap, dtype=torch.int32, device=dev)
        self.output_index = torch.empty(max_tokens, topk, dtype=torch.int32, device=dev)
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=dev)
        wsb = L.moe_route_pack_workspace_bytes(max_tokens, topk, E)
        self.workspace = torch.empty(max(wsb, 16), dtype=torch.uint8, device=dev)
        self.D = torch.empty(self.rows_cap, N, dtype=torch.bfloat16, device=dev)
        self.Z = torch.empty(max_tokens, N, dtype=torch.bfloat16, device=dev)

    def _views(self, T):
        return self.q[:T], self.sf[:T], self.output_index[:T], self.Z[:T]

    def quant(self, x):
        q, sf, _, _ = self._views(x.shape[0])
        L.moe_quant_act(x, q, sf)

    def route(self, topk_ids):
        T = topk_ids.shape[0]
        q, sf, oi, _ = self._views(T)
        rows = L.moe_packed_rows_cap(T, self.topk, self.E, self.am) if self.layout == L.LAYOUT_CONTIGUOUS \
            else self.rows_cap
        L.moe_route_pack(topk_ids, self.E, self.layout, self.am, q, self.packed[:rows], self.counts,
                         self.seg_offsets, self.m_indices[:rows], oi, self.dev_status, payload2=sf,
                         packed2=self.packed_sf[:rows], workspace=self.workspace)

    def quant_route(self, x, topk_ids):
        """quant() and route() in one launch sequence (moe_route_pack_quant): the packed codes and scales are the
        same bits, each token row is quantised once, and the token-order codes (self.q, self.sf) are not written."""
        T = topk_ids.shape[0]
        _, _, oi, _ = self._views(T)
        rows = L.moe_packed_rows_cap(T, self.topk, self.E, self.am) if self.layout == L.LAYOUT_CONTIGUOUS \
            else self.rows_cap
        L.moe_route_pack_quant(topk_ids, self.E, self.layout, self.am, x, self.packed[:rows],
                               self.packed_sf[:rows], self.counts, self.seg_offsets, self.m_indices[:rows], oi,
                               self.dev_status, workspace=self.workspace)

    def gemm(self, A=None, SFA=None, D=None, w=None, sfw=None, N=None, K=None):
        """Grouped GEMM on the packed rows (defaults: this layer's buffers and weights)."""
        A = self.packed if A is None else A
        SFA = self.packed_sf if SFA is None else SFA
        D = self.D if D is None else D
        w = self.w if w is None else w
        sfw = self.sfw if sfw is None else sfw
        N = self.N if N is None else N
        K = self.K if K is None else K
        am = self.am if self.layout == L.LAYOUT_MASKED else self.rows_cap
        L.moe_grouped_gemm_fp8(self.layout | self.wflag, A, SFA, w, sfw, D, self.counts, self.seg_offsets, self.E,
                               am, N, K, self.expected_m)

    def swiglu_quant(self, q, sf, D=None):
        """silu(gate) * up of the up-projection output D (default: this layer's), requantised into the
        down-projection's FP8 codes q [rows, N/2] and 1x128 scales sf [rows, N/256]."""
        D = self.D if D is None else D
        am = self.am if self.layout == L.LAYOUT_MASKED else self.rows_cap
        L.moe_swiglu_quant(self.layout, D, am, self.counts, self.seg_offsets, self.E, q, sf)

    def gemm_swiglu(self, q, sf):
        """The up-projection on the packed rows with SwiGLU and the requantisation fused (this layer's weights
        are the up-projection's, N = 2I): codes q [rows, N/2] and 1x128 scales sf [rows, N/256], the same bits
        as gemm() followed by swiglu_quant(), without the bf16 output D."""
        am = self.am if self.layout == L.LAYOUT_MASKED else self.rows_cap
        L.moe_grouped_gemm_fp8_swiglu(self.layout | self.wflag, self.packed, self.packed_sf, self.w, self.sfw, q, sf,
                                      self.counts, self.seg_offsets, self.E, am, self.N // 2, self.K,
                                      self.expected_m)

    def combine(self, topk_weights, D=None, Z=None):
        """Weighted combine of packed rows D (default: this layer's GEMM output) into Z [T, D.shape[1]]."""
        T = topk_weights.shape[0]
        _, _, oi, Zl = self._views(T)
        D = self.D if D is None else D
        if Z is None:
            if D.shape[1] != self.N:
                raise ValueError("pass Z when D is not [rows, N]")
            Z = Zl
        L.moe_unpermute_combine(D, oi, topk_weights, Z)
        return Z

    def combine_backward(self, dZ, topk_weights, dD, dweights, D=None, workspace=None):
        """Gradient of combine() with the routing of the last route()/quant_route(): dZ [T, N] -> dD, the gradient of the
        packed rows D (default: this layer's GEMM output) that a token was routed to (the padding's are not written),
        and dweights [T, topk].  workspace: moe_unpermute_combine_bwd_workspace_bytes(T, topk, rows of D) bytes; without
        one, a call that needs it allocates it."""
        T = dZ.shape[0]
        D = self.D if D is None else D
        if workspace is None:
            need = L.moe_unpermute_combine_bwd_workspace_bytes(T, self.topk, D.shape[0])
            if need > 0:
                workspace = torch.empty(need, dtype=torch.uint8, device=dZ.device)
        L.moe_unpermute_combine_bwd(dZ, D, self.output_index[:T], topk_weights, dD, dweights, workspace=workspace)
        return dD, dweights

    def forward(self, x, topk_ids, topk_weights, fused_quant=False):
        """fused_quant: quantise while packing (quant_route) instead of quant() then route()."""
        if fused_quant:
            self.quant_route(x, topk_ids)
        else:
            self.quant(x)
            self.route(topk_ids)
        self.gemm()
        return self.combine(topk_weights)


class MoeInt4Layer:
    """4-bit weight-only expert GEMM (group 128, fp16 scales, zero point 8), bf16 activations."""

    def __init__(self, w_q4: torch.Tensor, s16: torch.Tensor, topk: int, max_tokens: int,
                 layout: int = L.LAYOUT_MASKED, align_or_max_m: int = 16, expected_m: int = 0,
                 weights_packed: bool = False):
        """weights_packed: w_q4 is in the order written by moe_pack_weight_int4."""
        E, N, K2 = w_q4.shape
        K = K2 * 2
        self.E, self.N, self.K, self.topk = E, N, K, topk
        self.w, self.s16 = w_q4, s16
        self.wflag = L.WEIGHTS_PACKED if weights_packed else 0
        self.layout, self.am, self.expected_m = layout, align_or_max_m, expected_m
        dev = w_q4.device
        if layout == L.LAYOUT_CONTIGUOUS:
            self.rows_cap = L.moe_packed_rows_cap(max_tokens, topk, E, align_or_max_m)
        else:
            self.rows_cap = E * align_or_max_m
        self.packed = torch.empty(self.rows_cap, K, dtype=torch.bfloat16, device=dev)
        self.counts = torch.zeros(E, dtype=torch.int32, device=dev)
        self.seg_offsets = torch.zeros(E + 1, dtype=torch.int32, device=dev)
        self.m_indices = torch.empty(self.rows_cap, dtype=torch.int32, device=dev)
        self.output_index = torch.empty(max_tokens, topk, dtype=torch.int32, device=dev)
        self.dev_status = torch.zeros(1, dtype=torch.int32, device=dev)
        wsb = L.moe_route_pack_workspace_bytes(max_tokens, topk, E)
        self.workspace = torch.empty(max(wsb, 16), dtype=torch.uint8, device=dev)
        self.D = torch.empty(self.rows_cap, N, dtype=torch.bfloat16, device=dev)
        self.Z = torch.empty(max_tokens, N, dtype=torch.bfloat16, device=dev)

    def route(self, x, topk_ids):
        T = topk_ids.shape[0]
        rows = L.moe_packed_rows_cap(T, self.topk, self.E, self.am) if self.layout == L.LAYOUT_CONTIGUOUS \
            else self.rows_cap
        L.moe_route_pack(topk_ids, self.E, self.layout, self.am, x, self.packed[:rows], self.counts,
                         self.seg_offsets, self.m_indices[:rows], self.output_index[:T], self.dev_status,
                         workspace=self.workspace)

    def gemm(self, w=None, s16=None):
        w = self.w if w is None else w
        s16 = self.s16 if s16 is None else s16
        am = self.am if self.layout == L.LAYOUT_MASKED else self.rows_cap
        L.moe_grouped_gemm_int4(self.layout | self.wflag, self.packed, w, s16, self.D, self.counts, self.seg_offsets,
                                self.E, am, self.N, self.K, self.expected_m)

    def combine(self, topk_weights):
        T = topk_weights.shape[0]
        L.moe_unpermute_combine(self.D, self.output_index[:T], topk_weights, self.Z[:T])
        return self.Z[:T]

    def forward(self, x, topk_ids, topk_weights):
        self.route(x, topk_ids)
        self.gemm()
        return self.combine(topk_weights)


class MoeRouter:
    """The router before a layer: gate logits -> (topk_ids, topk_weights), with the gradient back to the logits.

    Holds the balance bias and output buffers for up to max_tokens tokens; a call allocates nothing.  forward() without
    buffers of the caller's writes those: its result lasts until the next such forward, so the gradient comes before that,
    and such calls that overlap in time must not run on two streams.  Where several batches are under way (micro-batches, a
    graph beside eager work), give each topk_ids and topk_weights of its own."""

    def __init__(self, E: int, topk: int, max_tokens: int, score: str = "softmax", bias: torch.Tensor | None = None,
                 n_group: int = 1, topk_group: int = 1, group_top: int = 1, renormalize: bool = True,
                 scale: float = 1.0, device="cuda"):
        self.E, self.topk, self.bias = E, topk, bias
        self.score, self.renormalize, self.scale = score, renormalize, scale
        self.groups = dict(n_group=n_group, topk_group=topk_group, group_top=group_top)
        self.topk_ids = torch.empty(max_tokens, topk, dtype=torch.int32, device=device)
        self.topk_weights = torch.empty(max_tokens, topk, dtype=torch.float32, device=device)

    def forward(self, logits, topk_ids=None, topk_weights=None):
        """logits float32 or bf16 [T, E] -> topk_ids int32 and topk_weights float32, [T, topk] each: the caller's if given
        (both, of any T), else this router's."""
        if (topk_ids is None) != (topk_weights is None):
            raise ValueError("topk_ids and topk_weights come together")
        T = logits.shape[0]
        ids, w = (self.topk_ids[:T], self.topk_weights[:T]) if topk_ids is None else (topk_ids, topk_weights)
        if ids.shape != (T, self.topk):
            raise ValueError(f"topk_ids is {tuple(ids.shape)}, needs {(T, self.topk)}")
        L.moe_router_topk(logits, ids, w, score=self.score, bias=self.bias, renormalize=self.renormalize,
                          scale=self.scale, **self.groups)
        return ids, w

    def backward(self, logits, topk_ids, dweights, dlogits):
        """d logits of the weights that forward(logits) gave for topk_ids (which must still hold that choice)."""
        L.moe_router_topk_bwd(logits, topk_ids, dweights, dlogits, score=self.score, renormalize=self.renormalize,
                              scale=self.scale)
        return dlogits


class DenseFP8Linear:
    """y = x W^T for one weight matrix that every token uses (a shared expert, a projection), block-scaled FP8.

    w_codes uint8 [N, K] and sfw float32 [ceil(N/128), K/128], any fp32 scales; for grad_input wt_codes [K, N] and
    sfwt [ceil(K/128), N/128] hold the transposed weight (N % 128 == 0).  The activations' codes have buffers for
    max_tokens tokens, so calls of one object that overlap in time must not run on two streams.  A product that splits
    K (few output tiles) and grad_weight take their scratch from torch's allocator, which a graph's capture keeps."""

    def __init__(self, w_codes: torch.Tensor, sfw: torch.Tensor, max_tokens: int, wt_codes: torch.Tensor | None = None,
                 sfwt: torch.Tensor | None = None):
        self.N, self.K = w_codes.shape
        self.w, self.sfw, self.wt, self.sfwt = w_codes, sfw, wt_codes, sfwt
        dev = w_codes.device
        wide = self.K if wt_codes is None else max(self.K, self.N)
        self.max_tokens = max_tokens
        self.q = torch.empty(max_tokens * wide, dtype=torch.uint8, device=dev)
        self.sf = torch.empty(max_tokens * (wide // 128), dtype=torch.float32, device=dev)

    def _gemm(self, A, SFA, W, SFW, out, C=None):
        need = L.moe_gemm_fp8_workspace_bytes(A.shape[0], W.shape[0], A.shape[1])
        ws = torch.empty(need, dtype=torch.uint8, device=A.device) if need > 0 else None
        L.moe_gemm_fp8(A, SFA, W, SFW, out, C=C, workspace=ws)
        return out

    def _product(self, x, w, sfw, out):
        T, K = x.shape
        if T > self.max_tokens or K != w.shape[1]:
            raise ValueError(f"x is {tuple(x.shape)}, needs [at most {self.max_tokens}, {w.shape[1]}]")
        q, sf = self.q[:T * K].view(T, K), self.sf[:T * (K // 128)].view(T, K // 128)
        L.moe_quant_act(x, q, sf)
        return self._gemm(q, sf, w, sfw, out)

    def forward(self, x, out):
        """x bf16 [T, K] -> out bf16 or float32 [T, N] (float32: every product in full, at half the rate)."""
        return self._product(x, self.w, self.sfw, out)

    def grad_input(self, dy, dx):
        """dy bf16 [T, N] -> dx bf16 or float32 [T, K]."""
        if self.wt is None:
            raise ValueError("grad_input needs the transposed weight (wt_codes, sfwt)")
        return self._product(dy, self.wt, self.sfwt, dx)

    def grad_weight(self, dy, x, dw, accumulate=True):
        """dw float32 [N, K] (+)= dy^T x of dy bf16 [T, N] and x bf16 [T, K], both quantised along the tokens."""
        if dy.shape[0] != x.shape[0]:
            raise ValueError(f"dy has {dy.shape[0]} tokens, x {x.shape[0]}")
        mb = (x.shape[0] + 127) // 128
        if mb == 0:
            return dw if accumulate else dw.zero_()
        qs = []
        for t in (dy, x):
            q = torch.empty(t.shape[1], 128 * mb, dtype=torch.uint8, device=t.device)
            sf = torch.empty(t.shape[1], mb, dtype=torch.float32, device=t.device)
            L.moe_quant_act_t(t, q, sf)
            qs += [q, sf]
        return self._gemm(*qs, dw, C=dw if accumulate else None)
