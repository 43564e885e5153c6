"""An expert layer out of this library's calls, with the experts' weights in int8, FP8 or bf16; and its experts in training.

    layer = ExpertLayer(R, T, w13, w13_scales, w2, w2_scales, gamma, topk=8)
    y = layer.norm(x, residual)                  # bf16 [R*T, H]: what the router reads
    topk_idx, topk_weights = router(y)
    out = layer.experts(topk_idx, topk_weights)  # bf16 [R*T, H]

``norm`` adds the residual (kept in ``layer.h``), normalises, and leaves the rows in int8 as well
(ep_rms_norm_quant).  ``experts`` takes one of two ways:

  - up to 64 tokens (``few_tokens``): ep_moe_few_tokens on y, which reads the chosen experts once and moves no rows;
  - more: layout, dispatch of the int8 rows as they are, gate and up products with SwiGLU, the
    inner rows to int8, the down product, combine.

FP8 weights (e4m3 with a scale for each block of 128) take the second way always, with FP8 rows that have a scale for each
128 columns; bf16 weights take either, with bf16 rows.

With int8 weights the first way keeps activations in bf16 where the second has them in int8.  From about 32 tokens on,
the second is the faster one where the tokens choose many experts (few, more; us, 4096 x 1024, top-8:
16 tokens over 32 experts 99, 115; 64 over 32 experts 208, 118; 16 over 128 experts 208, 215; 64 over
128 experts 357, 299): ``few_tokens`` says up to how many take the first.

    experts = TrainableExperts(R, T, w13, w2, topk=8)            # bf16 weights
    out = experts.forward(x, topk_idx, topk_weights)
    grad_x, grad_topk_weights = experts.backward(grad_out)       # adds to experts.grad_w13, experts.grad_w2

``TrainableExperts`` runs layout, dispatch, the products, SwiGLU with its gates and ups kept in 8 bits, and combine, and their
gradients.  The routing weight of a row is multiplied in with SwiGLU, so that combine is a plain sum: its gradient is a
dispatch of the output's gradient, and that of dispatch a combine.  The two calls stand outside of autograd: ``forward`` returns
a tensor without a graph, whatever x and the weights require.  A model whose other layers are autograd's puts them into a
function of its own:

    class Experts(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, topk_weights, topk_idx, experts):
            ctx.experts = experts
            return experts.forward(x, topk_idx, topk_weights)

        @staticmethod
        def backward(ctx, grad_out):
            grad_x, grad_topk_weights = ctx.experts.backward(grad_out.contiguous())
            return grad_x, grad_topk_weights, None, None

    out = Experts.apply(x, topk_weights, topk_idx, experts)      # topk_weights [N, K]; one backward pass before the next forward
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

    w13 [E, 2I, H] (gate rows, then up rows) and w2 [E, H, I], gamma [H] bf16.  int8 weights have a float32 scale for
    each row, w13_scales [E, 2I] and w2_scales [E, H]; float8_e4m3fn ones for each block of 128, w13_scales [E, 2 *
    ceil(I / 128), H / 128] (of the gates, then of the ups) and w2_scales [E, ceil(H / 128), I / 128], H and I multiples of
    128; bf16 ones none (None).  Every call runs on the current stream, or on ``stream``."""

    def __init__(self, R: int, T: int, w13, w13_scales, w2, w2_scales, gamma, topk: int, eps: float = 1e-6,
                 alpha: int = 1, few_tokens: int = FEW_TOKENS):
        self.w13, self.w13_scales, self.w2, self.w2_scales, self.gamma = w13, w13_scales, w2, w2_scales, gamma
        self.E, self.I, self.H = w13.shape[0], w13.shape[1] // 2, w13.shape[2]
        self.R, self.T, self.N, self.K, self.eps = R, T, R * T, topk, eps
        self.fp8, self.bf16 = w13.dtype is torch.float8_e4m3fn, w13.dtype is torch.bfloat16
        if w2.dtype is not w13.dtype or self.bf16 != (w13_scales is None) or self.bf16 != (w2_scales is None):
            raise ep.EPError(ep.EP_ERR_INVALID_ARG, "w13, w2: int8 or float8_e4m3fn with scales, or bf16 without")
        if self.fp8 and (self.H % 128 or self.I % 128):
            raise ep.EPError(ep.EP_ERR_INVALID_ARG, "FP8 weights: H and I multiples of 128")
        # of the rows that norm() leaves beside y (with bf16 weights nobody reads them)
        self.quant = ep.EP_QUANT_FP8_E4M3_PER_GROUP if self.fp8 else ep.EP_QUANT_INT8_PER_TOKEN
        row = torch.float8_e4m3fn if self.fp8 else torch.int8
        dev = w13.device
        self.y = torch.empty((self.N, self.H), dtype=torch.bfloat16, device=dev)
        self.h = torch.empty_like(self.y)
        self.out = torch.empty_like(self.y)
        self.rows = torch.empty((self.N, self.H), dtype=row, device=dev)
        self.row_scales = torch.empty((self.N, self.H // 128 if self.fp8 else 1), dtype=torch.float32, device=dev)
        self.few = self.N <= min(few_tokens, FEW_TOKENS) and not self.fp8
        if self.few:
            n = ep.ep_moe_few_tokens_workspace_size(self.N, self.H, self.E, topk, self.I)
            self.workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
            self._words, self._word = torch.zeros(STATUS_WORDS, dtype=torch.int32, device=dev), 0
            return
        self.layout = ep.EPLayout(R, T, self.H, self.E, topk, alpha, device=dev)
        cap = self.layout.worst_rows
        self.inner = torch.empty((cap, self.I), dtype=torch.bfloat16, device=dev)
        self.expert_out = torch.empty((cap, self.H), dtype=torch.bfloat16, device=dev)
        if self.bf16:
            self.recv = torch.empty((cap, self.H), dtype=torch.bfloat16, device=dev)
            return
        self.recv, self.recv_scales = self.layout.alloc_recv(self.quant, cap, device=dev)
        self.inner_rows = torch.empty((cap, self.I), dtype=row, device=dev)
        self.inner_scales = torch.empty((cap, self.I // 128 if self.fp8 else 1), dtype=torch.float32, device=dev)

    def norm(self, x: torch.Tensor, residual: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """y = RMSNorm(x + residual) * gamma, bf16; the sum is kept in self.h."""
        ep.ep_rms_norm_quant(x, residual, self.gamma, self.eps, self.quant, self.h, self.rows,
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
        lay, q = self.layout, self.quant
        lay.layout(topk_idx, stream)
        if self.bf16:
            lay.dispatch(self.y, ep.EP_QUANT_NONE, self.recv.view(torch.uint8), None, stream)
            lay.expert_matmul_bf16(self.recv, self.w13, self.inner, swiglu=True, stream=stream)
            lay.expert_matmul_bf16(self.inner, self.w2, self.expert_out, stream=stream)
            return lay.combine(self.expert_out, topk_weights, self.out, shared, stream)
        product = lay.expert_matmul_fp8 if self.fp8 else lay.expert_matmul
        lay.dispatch_ex(self.rows, q, self.recv, self.recv_scales, stream, x_scales=self.row_scales, pre_encoded=True)
        product(self.recv, self.recv_scales, self.w13, self.w13_scales, self.inner, swiglu=True, stream=stream)
        ep.ep_quant_rows(self.inner, q, self.inner_rows, self.inner_scales, stream)
        product(self.inner_rows, self.inner_scales, self.w2, self.w2_scales, self.expert_out, stream=stream)
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


class TrainableExperts:
    """The experts of a layer in training, on one GPU that holds all R ranks: bf16 weights w13 [E, 2I, H] (gate rows, then
    up rows) and w2 [E, H, I], gradients grad_w13 and grad_w2 of their shapes in float32, to which each backward() adds.
    H a multiple of 8, I of 128.  What backward() needs of the forward pass is kept in this object's buffers: rows in bf16,
    gates and ups in 8 bits.  Calls of one object, its making among them, are issued on one stream, or ordered across streams by the
    caller."""

    def __init__(self, R: int, T: int, w13: torch.Tensor, w2: torch.Tensor, topk: int, alpha: int = 1):
        # (the products check these again, but by then a forward() is on its way)
        if w13.dim() != 3 or w13.dtype is not torch.bfloat16 or not w13.is_contiguous() or w13.shape[1] % 256 or w13.shape[2] % 8:
            raise ep.EPError(ep.EP_ERR_INVALID_ARG, "w13: contiguous bf16 [E, 2I, H], I a multiple of 128, H of 8")
        self.E, self.I, self.H = w13.shape[0], w13.shape[1] // 2, w13.shape[2]
        if w2.dtype is not torch.bfloat16 or not w2.is_contiguous() or w2.shape != (self.E, self.H, self.I):
            raise ep.EPError(ep.EP_ERR_INVALID_ARG, "w2: contiguous bf16 [E, H, I]")
        if R * T < 1:
            raise ep.EPError(ep.EP_ERR_INVALID_ARG, "R * T: at least one token")
        self.R, self.T, self.N, self.K, self.w13, self.w2 = R, T, R * T, topk, w13, w2
        dev, bf = w13.device, torch.bfloat16
        self.layout = ep.EPLayout(R, T, self.H, self.E, topk, alpha, device=dev)
        cap = self.layout.worst_rows
        self._dst = self.layout.views()["dst_row"]
        # a layout without entries, until one has run (a captured forward() runs when its graph is replayed)
        self.layout.ws.zero_()
        self._dst.fill_(-1)
        self._ran = False   # whether the buffers are those of a whole forward()
        self.rows = torch.empty((cap, self.H), dtype=bf, device=dev)
        self.inner = torch.empty((cap, self.I), dtype=bf, device=dev)
        self.c = torch.empty((cap, 2 * self.I), dtype=bf, device=dev)       # and its gradient
        self.codes = torch.empty((cap, 2 * self.I), dtype=torch.float8_e4m3fn, device=dev)
        self.scales = torch.empty((cap, self.I // 64), dtype=torch.float32, device=dev)
        self.expert_out = torch.empty((cap, self.H), dtype=bf, device=dev)  # and its gradient
        self.row_weights = torch.zeros(cap + 1, dtype=torch.float32, device=dev)   # one more: of entries without an expert
        self.row_weights_grad = torch.zeros(cap + 1, dtype=torch.float32, device=dev)
        self.ones = torch.ones((self.N, topk), dtype=torch.float32, device=dev)
        self.grad_inner = torch.empty((cap, self.I), dtype=bf, device=dev)
        self.grad_rows = torch.empty((cap, self.H), dtype=bf, device=dev)
        self.grad_w13 = torch.zeros(w13.shape, dtype=torch.float32, device=dev)
        self.grad_w2 = torch.zeros(w2.shape, dtype=torch.float32, device=dev)

    def zero_grad(self, stream=None) -> None:
        with _on(stream):
            self.grad_w13.zero_()
            self.grad_w2.zero_()

    def _entries(self):
        """The row of each token's entry; the one behind the last for entries without an expert."""
        return torch.where(self._dst < 0, self.row_weights.numel() - 1, self._dst).view(-1).long()

    def forward(self, x: torch.Tensor, topk_idx: torch.Tensor, topk_weights: torch.Tensor, stream=None) -> torch.Tensor:
        """The weighted sum of the chosen experts' outputs of x [R*T, H] bf16: a new bf16 [R*T, H], without an autograd graph.
        topk_idx int64 and topk_weights float32, contiguous, hold K entries for each token (-1: no expert)."""
        for t, dtype, n, what in ((x, torch.bfloat16, self.N * self.H, "x: contiguous bf16 [N, H]"),
                                  (topk_idx, torch.int64, self.N * self.K, "topk_idx: contiguous int64 [N, K]"),
                                  (topk_weights, torch.float32, self.N * self.K, "topk_weights: contiguous float32 [N, K]")):
            if t.dtype is not dtype or not t.is_contiguous() or t.numel() != n:
                raise ep.EPError(ep.EP_ERR_INVALID_ARG, what)
        lay, self._ran = self.layout, False
        lay.layout(topk_idx, stream)
        lay.dispatch(x, ep.EP_QUANT_NONE, self.rows.view(torch.uint8), None, stream)
        lay.expert_matmul_bf16(self.rows, self.w13, self.c, stream=stream)
        with _on(stream), torch.no_grad():   # (the router's weights may belong to a graph of its own)
            # rows that no token fills have weight 0, whatever the step before had there
            self.row_weights.zero_().scatter_(0, self._entries(), topk_weights.view(-1))
            out = torch.empty((self.N, self.H), dtype=torch.bfloat16, device=x.device)
        ep.ep_swiglu_keep(self.c, self.inner, self.codes, self.scales, self.row_weights[:-1], lay.rows_used, stream)
        lay.expert_matmul_bf16(self.inner, self.w2, self.expert_out, stream=stream)
        lay.combine(self.expert_out, self.ones, out, None, stream)
        self._ran = True
        return out

    def backward(self, grad_out: torch.Tensor, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
        """(grad_x bf16 [R*T, H], grad_topk_weights float32 [R*T, K]) of the last forward(), of grad_out bf16 [R*T, H]; an
        entry without an expert has gradient 0.  The weights' gradients are added to grad_w13 and grad_w2.  Refused before the
        first forward(), and after one that raised on its way."""
        if not self._ran:
            raise ep.EPError(ep.EP_ERR_INVALID_ARG, "backward() needs a forward() before it")
        if grad_out.dtype is not torch.bfloat16 or not grad_out.is_contiguous() or grad_out.numel() != self.N * self.H:
            raise ep.EPError(ep.EP_ERR_INVALID_ARG, "grad_out: contiguous bf16 [N, H]")
        lay = self.layout
        lay.dispatch(grad_out, ep.EP_QUANT_NONE, self.expert_out.view(torch.uint8), None, stream)
        lay.expert_matmul_grad_rows(self.expert_out, self.w2, self.grad_inner, stream)
        ep.ep_swiglu_keep_grad(self.codes, self.scales, self.grad_inner, self.c, self.inner, self.row_weights[:-1],
                               self.row_weights_grad[:-1], lay.rows_used, stream)
        lay.expert_matmul_grad_weights(self.expert_out, self.inner, self.grad_w2, accumulate=True, stream=stream)
        lay.expert_matmul_grad_weights(self.c, self.rows, self.grad_w13, accumulate=True, stream=stream)
        lay.expert_matmul_grad_rows(self.c, self.w13, self.grad_rows, stream)
        with _on(stream), torch.no_grad():
            grad_x = torch.empty((self.N, self.H), dtype=torch.bfloat16, device=grad_out.device)
            grad_weights = self.row_weights_grad[self._entries()].view(self.N, self.K)
        return lay.combine(self.grad_rows, self.ones, grad_x, None, stream), grad_weights

    def status(self, stream=None) -> int:
        """The first device-side error since the last forward(); waits for ``stream``."""
        return self.layout.status(stream)
