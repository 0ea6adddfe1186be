"""A pre-norm residual MoE block of separate operators, with what it keeps for the backward in 8 bits.

    h = x (+ residual);  n = layernorm(h);  out = the experts' output on n, combined per token

and the block's output is h + out, which the next block's norm adds (its x = h, residual = out).
Buffers are allocated with torch and the C entry points called in order; no arithmetic happens
here.

Forward:  moe_layernorm_fwd -> moe_router_fwd -> moe_route -> moe_ep_pack (world 1: dense rows by
          expert) -> moe_grouped_linear_fwd -> moe_swiglu_fwd -> moe_grouped_linear_fwd ->
          moe_unpermute_combine
Backward: the same in reverse, from 8-bit checkpoints of the normalised input (T * H bytes) and
          of g and u (T * k * 2I bytes); n, the packed rows and the activation are computed
          again.  ``layer.ExpertFFN`` is the fused layer, in MXFP8, FP8 or bf16, for the same sizes;
          this block adds the norm and the 8-bit checkpoints, for bf16 training whose memory is bound
          by what each layer keeps: everything in Scratch is shared by all blocks of a model.
"""
from __future__ import annotations

import torch

from . import binding as B

U8, BF16, F32, I32 = torch.uint8, torch.bfloat16, torch.float32, torch.int32


class Scratch:
    """Buffers that hold nothing between two calls of a block: one set serves every block of these
    sizes on one stream."""

    def __init__(self, T, H, I, E, k, device="cuda"):
        R = T * k
        dev = torch.device(device)
        e = lambda *s, dt=BF16: torch.empty(*s, dtype=dt, device=dev)  # noqa: E731
        self.sizes = (T, H, I, E, k)
        self.d = B.dims(T, H, I, E, k)
        self.cap = B.moe_rows_capacity(self.d)
        if self.cap == 0:
            raise B.MoeError(2, f"unsupported sizes T={T} H={H} I={I} E={E} k={k}")
        self.up, self.down = B.grouped(R, H, 2 * I, E), B.grouped(R, I, H, E)
        self.norm = B.norm(T, H)
        self.ws = torch.zeros(B.moe_workspace_size(self.d, 1), dtype=U8, device=dev)
        self.ws_norm = torch.zeros(max(256, B.moe_layernorm_workspace_size(self.norm)), dtype=U8, device=dev)
        self.ws_linear = torch.zeros(B.moe_grouped_linear_workspace_size(self.up), dtype=U8, device=dev)
        self.n = e(T, H)
        self.rows, self.drows = e(R, H), e(R, H)
        self.gu, self.dgu = e(R, 2 * I), e(R, 2 * I)
        self.a = e(R, I)
        self.eid, self.counts = e(R, dt=I32), e(1, dt=I32)
        self.src_of, self.prob_perm = e(self.cap, dt=I32), e(self.cap, dt=F32)
        self.dprob_rows, self.dprob, self.dlogits = e(R, dt=F32), e(T, k, dt=F32), e(T, E, dt=F32)


class MoEBlock:
    """One block for fixed sizes (H and I multiples of 128, as the routing's entry points have them)."""

    def __init__(self, T, H, I, E, k, device="cuda", scratch=None, eps=1e-5):
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.s = scratch if scratch is not None else Scratch(T, H, I, E, k, device)
        if self.s.sizes != (T, H, I, E, k):
            # the calls take their sizes from the scratch and would run past this block's tensors
            raise ValueError(f"scratch made for T, H, I, E, k = {self.s.sizes}, block for {(T, H, I, E, k)}")
        self.norm = B.norm(T, H, eps=eps)
        R, dev = T * k, self.s.ws.device
        e = lambda *s, dt=BF16: torch.empty(*s, dtype=dt, device=dev)  # noqa: E731
        # kept from the forward pass to the backward
        self.rstd = e(T, dt=F32)
        self.n_codes, self.n_scales = e(T, H, dt=U8), e(T, (H + 31) // 32, dt=U8)
        self.gu_codes, self.gu_scales = e(R, 2 * I, dt=U8), e(R, 2 * ((I + 31) // 32), dt=U8)
        self.logits, self.idx, self.prob = e(T, E, dt=F32), e(T, k, dt=I32), e(T, k, dt=F32)
        self.split_sizes, self.row_of, self.pos_of = e(E, dt=I32), e(T, k, dt=I32), e(T, k, dt=I32)
        self.prob_rows = e(R, dt=F32)
        # results
        self.h, self.out, self.dx = e(T, H), e(T, H), e(T, H)
        self.dgamma, self.dbeta, self.dw_r = e(H), e(H), e(E, H, dt=F32)
        self.dw_gu, self.dw_d = e(E, 2 * I, H), e(E, H, I)
        self._kept = False                                   # nothing kept yet

    def kept_bytes(self) -> int:
        """Bytes that this block keeps between the passes."""
        kept = (self.rstd, self.n_codes, self.n_scales, self.gu_codes, self.gu_scales, self.logits, self.idx, self.prob,
                self.split_sizes, self.row_of, self.pos_of, self.prob_rows)
        return sum(t.numel() * t.element_size() for t in kept)

    def _pack(self, rows_in, rows_out, stream):
        """The (token, slot) rows of a [T][H] tensor in expert order, without padding."""
        s = self.s
        B.moe_ep_pack(s.d, 1, rows_in, self.idx, self.prob, self.row_of, self.split_sizes, rows_out, self.prob_rows, s.eid,
                      self.pos_of, s.counts, s.ws, stream)

    def forward(self, x, weights, residual=None, stream=None):
        """(h, out) of x bf16 [T][H] (and residual); weights: gamma, beta bf16 [H], w_r bf16 [E][H],
        w_gu bf16 [E][2I][H], w_d bf16 [E][H][I].  Without a residual h is x itself."""
        s, w = self.s, weights
        B._dense(w["w_r"], BF16, self.E * self.H)            # the router's call does not look at its tensors
        h = self.h if residual is not None else None
        B.moe_layernorm_fwd(self.norm, x, residual, w["gamma"], w["beta"], h, s.n, None, self.rstd, self.n_codes,
                            self.n_scales, stream)
        B._on(stream, w["w_r"])
        B.moe_router_fwd(s.d, s.n, w["w_r"], self.logits, s.ws, stream)
        B.moe_route(s.d, self.logits, self.idx, self.prob, self.split_sizes, self.row_of, s.src_of, s.prob_perm, s.ws, stream)
        self._pack(s.n, s.rows, stream)
        B.moe_grouped_linear_fwd(s.up, s.rows, self.split_sizes, w["w_gu"], s.gu, s.ws_linear, stream)
        B.moe_swiglu_fwd(s.gu, self.prob_rows, s.a, self.gu_codes, self.gu_scales, stream)
        B.moe_grouped_linear_fwd(s.down, s.a, self.split_sizes, w["w_d"], s.rows, s.ws_linear, stream)
        B.moe_unpermute_combine(s.d, s.rows, self.pos_of, None, self.out, stream)
        self._kept = True
        return (x if h is None else h), self.out

    def backward(self, dout, weights, stream=None):
        """From the gradient of h + out: dx (of x and of residual), and dgamma, dbeta, dw_r, dw_gu, dw_d."""
        s, w = self.s, weights
        # the packing's and the router's calls do not look at their tensors; a gradient may well be expanded
        B._pitched(dout, self.T, self.H, self.H, BF16)
        B._dense(w["w_r"], BF16, self.E * self.H)
        if not self._kept:
            raise RuntimeError("backward before forward: the rows' places are not set yet")
        B._on(stream, dout, w["w_r"])
        self._pack(dout, s.drows, stream)
        B.moe_grouped_linear_dgrad(s.down, s.drows, self.split_sizes, w["w_d"], s.a, s.ws_linear, stream)
        B.moe_swiglu_bwd(None, self.gu_codes, self.gu_scales, self.prob_rows, s.a, s.dgu, s.dprob_rows, s.a, stream)
        B.moe_grouped_linear_wgrad(s.down, s.a, s.drows, self.split_sizes, self.dw_d, s.ws_linear, stream)
        B.moe_act8_unpack(self.n_codes, self.n_scales, w["gamma"], w["beta"], s.n, stream)
        self._pack(s.n, s.rows, stream)
        B.moe_grouped_linear_wgrad(s.up, s.rows, s.dgu, self.split_sizes, self.dw_gu, s.ws_linear, stream)
        B.moe_grouped_linear_dgrad(s.up, s.dgu, self.split_sizes, w["w_gu"], s.drows, s.ws_linear, stream)
        B.moe_unpermute_combine(s.d, s.drows, self.pos_of, None, self.dx, stream)
        B.moe_gather_f32(s.dprob_rows, self.pos_of, self.T * self.k, s.dprob, s.ws, stream)
        B.moe_router_bwd(s.d, s.n, w["w_r"], self.logits, self.idx, self.prob, s.dprob, s.dlogits, self.dx, self.dw_r,
                         s.ws, stream)
        B.moe_layernorm_bwd(self.norm, self.dx, None, None, self.rstd, self.n_codes, self.n_scales, w["gamma"], dout,
                            self.dx, self.dgamma, self.dbeta, s.ws_norm, stream)
        return self.dx

    def device_error(self, stream=None):
        """(code, site) of the first device error recorded in a workspace of this block."""
        for ws in (self.s.ws, self.s.ws_linear):
            code, site = B.moe_get_device_error(ws, stream)
            if code != 0:
                return code, site
        return 0, 0
