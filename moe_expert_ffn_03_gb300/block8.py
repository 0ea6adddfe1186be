"""A pre-norm residual MoE block whose products read 8-bit operands with one f32 scale per block of 128.

    h = x (+ residual);  n = rmsnorm(h);  out = the experts' output on n, combined per token

and the block's output is h + out, which the next block's norm adds (its x = h, residual = out), as with
``block.MoEBlock``.  Next to ``MoEBlock`` (layer norm, bf16 products, 8-bit checkpoints) and
``layer.ExpertFFN`` (the fused layer with scales per 32 values) this one takes weights as they are
quantized in blocks of 128 x 128, by ``quantize_weights`` or elsewhere, and adds the router's balance loss.
Buffers are allocated with torch and the C entry points called in order; no arithmetic happens here.

Forward:  moe_rmsnorm_fwd (n for the router, and in 8 bits) -> moe_router_fwd -> moe_route
          -> moe_balance_loss_fwd -> moe_fp8_block_pack -> moe_grouped_linear_fp8_fwd -> moe_swiglu_fwd
          -> moe_fp8_block_quantize -> moe_grouped_linear_fp8_fwd -> moe_unpermute_combine
Backward: the same in reverse.  A weight gradient's operands are quantized along tokens; its x is what the
          product has read, the values of n in 8 bits, and the activation is computed again from its
          8-bit checkpoint.  The router's weight gradient takes n from the same codes, E4M3 (2^-4 of a value at most)
          where the forward pass gave the router bf16: n is not kept a second time.
"""
from __future__ import annotations

import torch

from . import binding as B

U8, BF16, F32, I32 = torch.uint8, torch.bfloat16, torch.float32, torch.int32


def _cuts(n):
    return (n + 127) // 128


class Weights8:
    """A layer's weights [E][N][K] in 8 bits: codes and the scales of their blocks of 128 x 128."""

    def __init__(self, E, N, K, device="cuda"):
        self.codes = torch.empty(E, N, K, dtype=U8, device=device)
        self.scales = torch.empty(E, _cuts(N), _cuts(K), dtype=F32, device=device)

    def quantize(self, w, stream=None):
        """From masters (bf16 or f32) of the same shape."""
        if w.shape != self.codes.shape:
            raise ValueError(f"weights of shape {tuple(w.shape)}, {tuple(self.codes.shape)} expected")
        B.moe_fp8_block_quantize_weights(w, self.codes, self.scales, stream)
        return self


class Scratch8:
    """Buffers that hold nothing between two calls of a block: one set serves every block of these sizes on one
    stream."""

    def __init__(self, T, H, I, E, k, device="cuda", training=True):
        R = T * k
        dev = torch.device(device)
        e = lambda *s, dt=BF16: torch.empty(*s, dtype=dt, device=dev)  # noqa: E731
        self.sizes, self.training = (T, H, I, E, k), training
        self.d = B.dims(T, H, I, E, k)
        self.cap = B.moe_rows_capacity(self.d)
        if self.cap == 0:
            raise B.MoeError(2, f"unsupported sizes T={T} H={H} I={I} E={E} k={k}")
        self.up, self.down = B.grouped(R, H, 2 * I, E), B.grouped(R, I, H, E)
        zeros = lambda n: torch.zeros(max(256, n), dtype=U8, device=dev)  # noqa: E731
        self.ws = zeros(B.moe_workspace_size(self.d, int(training)))
        self.ws_linear = zeros(B.moe_grouped_linear_fp8_workspace_size(self.up))
        self.ws_balance = zeros(B.moe_balance_loss_workspace_size(B.balance(T, E, k)))
        self.ws_pack = zeros(256)
        self.n = e(T, H)
        self.rows, self.a = e(R, H), e(R, I)
        self.rows8, self.rows8_s = e(R, H, dt=U8), e(_cuts(H), R, dt=F32)
        self.a8, self.a8_s = e(R, I, dt=U8), e(_cuts(I), R, dt=F32)
        self.gu = e(R, 2 * I)
        self.src_of, self.prob_perm = e(self.cap, dt=I32), e(self.cap, dt=F32)
        if training:
            blocks = B.fp8_blocks(R, E)
            self.ws_norm = zeros(B.moe_rmsnorm_workspace_size(B.norm(T, H)))
            self.dgu8, self.dgu8_s = e(R, 2 * I, dt=U8), e(_cuts(2 * I), R, dt=F32)
            # along tokens: gradients by columns, what they are multiplied with in tiles
            self.dyt, self.dyt_s = e(blocks * 128, max(H, 2 * I), dt=U8), e(blocks, max(H, 2 * I), dt=F32)
            self.xt, self.xt_s = e(blocks * 128, max(H, I), dt=U8), e(blocks, _cuts(max(H, I)), dt=F32)
            self.eid, self.counts, self.pos_of, self.prob_rows = e(R, dt=I32), e(1, dt=I32), e(T, k, dt=I32), e(R, dt=F32)
            self.dprob_rows, self.dprob = e(R, dt=F32), e(T, k, dt=F32)
            self.aux, self.dlogits = e(T, E, dt=F32), e(T, E, dt=F32)

    def tokens(self, which, cols):
        """The part of a buffer along tokens that rows of `cols` values take: codes and scales."""
        codes, scales = (self.dyt, self.dyt_s) if which == "dy" else (self.xt, self.xt_s)
        n = cols if which == "dy" else _cuts(cols)
        blocks = codes.shape[0] // 128
        return codes.view(-1)[: blocks * 128 * cols].view(blocks * 128, cols), scales.view(-1)[: blocks * n].view(blocks, n)


class Fp8MoEBlock:
    """One block for fixed sizes (H and I multiples of 128, as the routing's entry points have them).

    alpha and beta weigh the balance loss and the z loss; both 0 leaves them out, and counts, prob_mean and loss stay
    zeros (split_sizes has the experts' rows).  Without `training` nothing is kept for a backward pass."""

    def __init__(self, T, H, I, E, k, device="cuda", scratch=None, eps=1e-5, alpha=0.0, beta=0.0, training=True):
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.s = scratch if scratch is not None else Scratch8(T, H, I, E, k, device, training)
        if self.s.sizes != (T, H, I, E, k):
            # the calls take their sizes from the scratch and would run past this block's tensors
            raise ValueError(f"scratch made for T, H, I, E, k = {self.s.sizes}, block for {(T, H, I, E, k)}")
        if training and not self.s.training:
            raise ValueError("scratch made for inference, block for training")
        self.training = training
        self.norm, self.loss_of = B.norm(T, H, eps=eps), B.balance(T, E, k, alpha, beta)
        self.balanced = alpha != 0.0 or beta != 0.0
        R, dev = T * k, self.s.ws.device
        e = lambda *s, dt=BF16: torch.empty(*s, dtype=dt, device=dev)  # noqa: E731
        # kept from the forward pass to the backward
        self.rstd = e(T, dt=F32)
        self.n_codes, self.n_scales = e(T, H, dt=U8), e(_cuts(H), T, dt=F32)
        self.logits, self.idx, self.prob = e(T, E, dt=F32), e(T, k, dt=I32), e(T, k, dt=F32)
        self.split_sizes, self.row_of, self.pos_of = e(E, dt=I32), e(T, k, dt=I32), e(T, k, dt=I32)
        self.prob_rows = e(R, dt=F32)
        self.gu_codes = e(R, 2 * I, dt=U8) if training else None
        self.gu_scales = e(R, 2 * ((I + 31) // 32), dt=U8) if training else None
        # results
        self.counts, self.prob_mean = torch.zeros(E + 1, dtype=I32, device=dev), torch.zeros(E, device=dev)
        self.loss = torch.zeros(3, device=dev)
        self.h, self.out = e(T, H), e(T, H)
        if training:
            self.dx, self.dgamma, self.dw_r = e(T, H), e(H), e(E, H, dt=F32)
            self.dw_gu, self.dw_d = e(E, 2 * I, H), e(E, H, I)
        self._kept = None                                    # the forward pass's h and mask

    def _weights(self, w):
        B._dense(w["w_r"], BF16, self.E * self.H)            # the router's call does not look at its tensors
        B._on(None, w["w_r"])
        for name, N, K in (("w_gu", 2 * self.I, self.H), ("w_d", self.H, self.I)):
            if w[name].codes.shape != (self.E, N, K):
                raise ValueError(f"{name} of shape {tuple(w[name].codes.shape)}, {(self.E, N, K)} expected")

    def forward(self, x, weights, residual=None, mask=None, stream=None):
        """(h, out) of x bf16 [T][H] (and residual); weights: gamma bf16 [H], w_r bf16 [E][H], w_gu and w_d Weights8.
        mask uint8 [T]: tokens with 0 are padding, which the balance loss leaves out.  Without a residual h is x
        itself, which the backward pass reads again, as it does mask.  counts, prob_mean and loss are the balance loss's."""
        s, w = self.s, weights
        self._weights(w)
        h = self.h if residual is not None else None
        B.moe_rmsnorm_fwd(self.norm, x, residual, w["gamma"], h, s.n, self.rstd, self.n_codes, self.n_scales, stream)
        B.moe_router_fwd(s.d, s.n, w["w_r"], self.logits, s.ws, stream)
        B.moe_route(s.d, self.logits, self.idx, self.prob, self.split_sizes, self.row_of, s.src_of, s.prob_perm, s.ws, stream)
        if self.balanced:
            B.moe_balance_loss_fwd(self.loss_of, self.logits, self.idx, mask, self.counts, self.prob_mean, self.loss,
                                   s.ws_balance, stream)
        B.moe_fp8_block_pack(self.n_codes, self.n_scales, self.idx, self.prob, self.row_of, self.split_sizes, s.rows8,
                             s.rows8_s, self.prob_rows, self.pos_of, s.ws_pack, stream)
        B.moe_grouped_linear_fp8_fwd(s.up, s.rows8, s.rows8_s, self.split_sizes, w["w_gu"].codes, w["w_gu"].scales, s.gu,
                                     s.ws_linear, stream)
        B.moe_swiglu_fwd(s.gu, self.prob_rows, s.a, self.gu_codes, self.gu_scales, stream)
        B.moe_fp8_block_quantize(s.a, s.a8, s.a8_s, stream=stream)
        B.moe_grouped_linear_fp8_fwd(s.down, s.a8, s.a8_s, self.split_sizes, w["w_d"].codes, w["w_d"].scales, s.rows,
                                     s.ws_linear, stream)
        B.moe_unpermute_combine(s.d, s.rows, self.pos_of, None, self.out, stream)
        if self.training:
            self._kept = (x if h is None else h, mask)
        return (x if h is None else h), self.out

    def _pack(self, rows_in, stream):
        """The (token, slot) rows of a [T][H] tensor in expert order, without padding, in the scratch."""
        s = self.s
        B.moe_ep_pack(s.d, 1, rows_in, self.idx, self.prob, self.row_of, self.split_sizes, s.rows, s.prob_rows, s.eid, s.pos_of,
                      s.counts, s.ws, stream)

    def backward(self, dout, weights, dloss=None, stream=None):
        """From the gradient of h + out, and dloss (f32 [1] on the device; None: 1) of the loss: dx (of x and of
        residual), and dgamma, dw_r, dw_gu, dw_d."""
        s, w = self.s, weights
        if not self.training:
            raise RuntimeError("block made for inference")
        # the packing's call does not look at its tensors; a gradient may well be expanded
        B._pitched(dout, self.T, self.H, self.H, BF16)
        self._weights(w)
        if self._kept is None:
            raise RuntimeError("backward before forward: the rows' places are not set yet")
        B._on(stream, dout)
        h, mask = self._kept
        H, I, ss = self.H, self.I, self.split_sizes
        # down: the gradient of its rows along rows and along tokens, then the activation's
        dyt, dyt_s = s.tokens("dy", H)
        self._pack(dout, stream)
        B.moe_fp8_block_quantize(s.rows, s.rows8, s.rows8_s, ss, dyt, dyt_s, "tokens", stream)
        B.moe_grouped_linear_fp8_dgrad(s.down, s.rows8, s.rows8_s, ss, w["w_d"].codes, w["w_d"].scales, s.a, s.ws_linear, stream)
        B.moe_swiglu_bwd(None, self.gu_codes, self.gu_scales, self.prob_rows, s.a, s.gu, s.dprob_rows, s.a, stream)
        xt, xt_s = s.tokens("x", I)
        B.moe_fp8_block_quantize(s.a, None, None, ss, xt, xt_s, "tiles", stream)
        B.moe_grouped_linear_fp8_wgrad(s.down, xt, xt_s, dyt, dyt_s, ss, self.dw_d, s.ws_linear, stream)
        # up: the same, with the rows that its product has read
        B.moe_fp8_block_dequantize(self.n_codes, self.n_scales, "rows", s.n, stream)
        self._pack(s.n, stream)
        xt, xt_s = s.tokens("x", H)
        B.moe_fp8_block_quantize(s.rows, None, None, ss, xt, xt_s, "tiles", stream)
        dyt, dyt_s = s.tokens("dy", 2 * I)
        B.moe_fp8_block_quantize(s.gu, s.dgu8, s.dgu8_s, ss, dyt, dyt_s, "tokens", stream)
        B.moe_grouped_linear_fp8_wgrad(s.up, xt, xt_s, dyt, dyt_s, ss, self.dw_gu, s.ws_linear, stream)
        B.moe_grouped_linear_fp8_dgrad(s.up, s.dgu8, s.dgu8_s, ss, w["w_gu"].codes, w["w_gu"].scales, s.rows, s.ws_linear, stream)
        B.moe_unpermute_combine(s.d, s.rows, self.pos_of, None, self.dx, stream)
        # router, with the loss's gradient of its logits
        B.moe_gather_f32(s.dprob_rows, self.pos_of, self.T * self.k, s.dprob, s.ws, stream)
        if self.balanced:
            B.moe_balance_loss_bwd(self.loss_of, self.logits, mask, self.counts, dloss, s.aux, stream)
        B.moe_router_bwd_aux(s.d, s.n, w["w_r"], self.logits, self.idx, self.prob, s.dprob, s.aux if self.balanced else None,
                             s.dlogits, self.dx, self.dw_r, s.ws, stream)
        B.moe_rmsnorm_bwd(self.norm, self.dx, h, self.rstd, w["gamma"], dout, self.dx, self.dgamma, s.ws_norm, stream)
        return self.dx

    def device_error(self, stream=None):
        """(code, site) of the first device error recorded in a workspace of this block."""
        s = self.s
        for ws in (s.ws, s.ws_linear, s.ws_balance, s.ws_pack):
            code, site = B.moe_get_device_error(ws, stream)
            if code != 0:
                return code, site
        return 0, 0
