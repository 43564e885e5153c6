"""An expert layer out of this library's calls, with the experts' weights in int8.

    layer = ExpertLayer(R, T, w13, w13_scales, w2, w2_scales, gamma, topk=8)
    y = layer.norm(x, residual)                  # bf16 [R*T, H]: what the router reads
    topk_idx, topk_weights = router(y)
    out = layer.experts(topk_idx, topk_weights)  # bf16 [R*T, H]

``norm`` adds the residual (kept in ``layer.h``), normalises, and leaves the rows in int8 as well
(ep_rms_norm_quant).  ``experts`` takes one of two ways:

  - up to 64 tokens (``few_tokens``): ep_moe_few_tokens on y, which reads the chosen experts once and moves no rows;
  - more: layout, dispatch of the int8 rows as they are, gate and up products with SwiGLU, the
    inner rows to int8, the down product, combine.

The first way keeps activations in bf16 where the second has them in int8.  From about 32 tokens on,
the second is the faster one where the tokens choose many experts (few, more; us, 4096 x 1024, top-8:
16 tokens over 32 experts 99, 115; 64 over 32 experts 208, 118; 16 over 128 experts 208, 215; 64 over
128 experts 357, 299): ``few_tokens`` says up to how many take the first.
"""
from __future__ import annotations

import contextlib

import torch

from . import ep

FEW_TOKENS = 64   # the most that ep_moe_few_tokens takes
STATUS_WORDS = 1024


def _on(stream):
    """Inside, torch's own kernels and allocations are of a call's stream (None: the current one)."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


class ExpertLayer:
    """Buffers and weights of one layer on one GPU that holds all R ranks.

    w13 [E, 2I, H] int8 (gate rows, then up rows) with w13_scales [E, 2I] float32; w2 [E, H, I] int8
    with w2_scales [E, H]; gamma [H] bf16.  Every call runs on the current stream, or on ``stream``."""

    def __init__(self, R: int, T: int, w13, w13_scales, w2, w2_scales, gamma, topk: int, eps: float = 1e-6,
                 alpha: int = 1, few_tokens: int = FEW_TOKENS):
        self.w13, self.w13_scales, self.w2, self.w2_scales, self.gamma = w13, w13_scales, w2, w2_scales, gamma
        self.E, self.I, self.H = w13.shape[0], w13.shape[1] // 2, w13.shape[2]
        self.R, self.T, self.N, self.K, self.eps = R, T, R * T, topk, eps
        dev = w13.device
        self.y = torch.empty((self.N, self.H), dtype=torch.bfloat16, device=dev)
        self.h = torch.empty_like(self.y)
        self.out = torch.empty_like(self.y)
        self.rows = torch.empty((self.N, self.H), dtype=torch.int8, device=dev)
        self.row_scales = torch.empty((self.N, 1), dtype=torch.float32, device=dev)
        self.few = self.N <= min(few_tokens, FEW_TOKENS)
        if self.few:
            n = ep.ep_moe_few_tokens_workspace_size(self.N, self.H, self.E, topk, self.I)
            self.workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
            self._words, self._word = torch.zeros(STATUS_WORDS, dtype=torch.int32, device=dev), 0
            return
        self.layout = ep.EPLayout(R, T, self.H, self.E, topk, alpha, device=dev)
        cap = self.layout.worst_rows
        self.recv, self.recv_scales = self.layout.alloc_recv(ep.EP_QUANT_INT8_PER_TOKEN, cap, device=dev)
        self.inner = torch.empty((cap, self.I), dtype=torch.bfloat16, device=dev)
        self.inner_rows = torch.empty((cap, self.I), dtype=torch.int8, device=dev)
        self.inner_scales = torch.empty((cap, 1), dtype=torch.float32, device=dev)
        self.expert_out = torch.empty((cap, self.H), dtype=torch.bfloat16, device=dev)

    def norm(self, x: torch.Tensor, residual: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """y = RMSNorm(x + residual) * gamma, bf16; the sum is kept in self.h."""
        ep.ep_rms_norm_quant(x, residual, self.gamma, self.eps, ep.EP_QUANT_INT8_PER_TOKEN, self.h, self.rows,
                             self.row_scales, stream, self.y)
        return self.y

    def experts(self, topk_idx: torch.Tensor, topk_weights: torch.Tensor, shared: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
        """The weighted sum of the chosen experts' outputs of the rows that norm() left, plus shared rows:
        bf16 [R, S, T, H] (as EPLayout.combine) or [S, N, H], whichever way is taken.  topk_idx int64 and
        topk_weights float32, contiguous, hold K entries for each of the N tokens."""
        for t, dtype, what in ((topk_idx, torch.int64, "topk_idx: contiguous int64 [N, K]"),
                               (topk_weights, torch.float32, "topk_weights: contiguous float32 [N, K]")):
            if t.dtype is not dtype or not t.is_contiguous() or t.numel() != self.N * self.K:
                raise ep.EPError(ep.EP_ERR_INVALID_ARG, what)
        if shared is not None:
            shared = self._shared_rows(shared, stream)
        if self.few:
            status = self._next_status(stream)   # (the layout clears its own on the other way)
            ep.ep_moe_few_tokens(self.y, topk_idx.view(self.N, self.K), topk_weights.view(self.N, self.K), self.w13,
                                 self.w2, self.out, self.workspace, self.w13_scales, self.w2_scales, shared,
                                 status, stream)
            return self.out
        lay, q = self.layout, ep.EP_QUANT_INT8_PER_TOKEN
        lay.layout(topk_idx, stream)
        lay.dispatch_ex(self.rows, q, self.recv, self.recv_scales, stream, x_scales=self.row_scales, pre_encoded=True)
        lay.expert_matmul(self.recv, self.recv_scales, self.w13, self.w13_scales, self.inner, swiglu=True, stream=stream)
        ep.ep_quant_rows(self.inner, q, self.inner_rows, self.inner_scales, stream)
        lay.expert_matmul(self.inner_rows, self.inner_scales, self.w2, self.w2_scales, self.expert_out, stream=stream)
        return lay.combine(self.expert_out, topk_weights, self.out, shared, stream)

    def _shared_rows(self, shared: torch.Tensor, stream) -> torch.Tensor:
        """The shared rows as this layer's way reads them: [S, N, H], or [R, S, T, H].  Where that takes a copy
        (several ranks and several rows), it is made on the call's stream, in that stream's memory."""
        R, T, H = self.R, self.T, self.H
        if shared.dim() == 3 and shared.shape[1:] == (self.N, H):
            ranks = shared.unflatten(1, (R, T)).transpose(0, 1)
        elif shared.dim() == 4 and (shared.shape[0], *shared.shape[2:]) == (R, T, H):
            ranks = shared
        else:
            ranks = None
        if ranks is None or shared.dtype is not torch.bfloat16:
            raise ep.EPError(ep.EP_ERR_INVALID_ARG, "shared: bf16 [R, S, T, H] or [S, N, H]")
        with _on(stream):
            return ranks.transpose(0, 1).reshape(ranks.shape[1], self.N, H).contiguous() if self.few else ranks.contiguous()

    def _next_status(self, stream) -> int:
        """The address of the status word of one step of the few-token way.  To clear it in front of each step would
        cost 2 to 10 us (28 us for 18 on a small layer, where the host is the bound): steps take words in turn, which
        are cleared together, and captured ones share the first, which status() clears."""
        if torch.cuda.is_current_stream_capturing():
            self._word = 0
        else:
            self._word += 1
            if self._word == STATUS_WORDS:
                self._word = 1
                with _on(stream):
                    self._words[1:].zero_()
        return self._words.data_ptr() + 4 * self._word

    def status(self, stream=None) -> int:
        """The first device-side error of the last experts() call; waits for ``stream``, the one that it ran on.  Of
        captured calls: of the replays since the last status() (few tokens), or of the last replay."""
        if not self.few:
            return self.layout.status(stream)
        with _on(stream):
            error = int(self._words[self._word].item())
            if error and self._word == 0:
                self._words[:1].zero_()
            return error
