"""An MoE layer put together from the library's calls.

``route`` is the router with its gradient (moe_route / moe_route_backward under
autograd), for training and serving.  ``Int8Experts``, for serving, is a gated
MLP whose experts' weights are int8 with a scale for each output channel.  It
has no gradient, and refuses inputs that ask for one:

    moe_layout           slots of the routing
    moe_dispatch_int8    rows to int8, packed by expert
    moe_expert_matmul_int8   gate and up projections      [rows, 2 I]
    silu(gate) * up      (PyTorch)                        [rows, I]
    moe_dispatch_int8    rows to int8 (K = 1, in place order)
    moe_expert_matmul_int8   down projection              [rows, H]
    moe_combine          the routing-weighted sum         [T, H]
"""
from __future__ import annotations

import torch

from . import _binding as moe


def quantize_channels(w: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """[E, N, H] weights to int8 codes and fp32 scales [E, N]: each channel's
    largest magnitude becomes 127.  Done once, when the weights are loaded."""
    w = w.float()
    scale = w.abs().amax(dim=2) / 127.0
    q = torch.round(w / torch.where(scale == 0, 1.0, scale)[..., None])
    return q.clamp_(-127, 127).to(torch.int8), scale


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, K, renormalize, loss_coef, token_mask):
        T, E = logits.shape
        logits = logits.contiguous()
        b = moe.RouteBuffers(T, K, E, device=logits.device)
        b.loss = torch.empty((), dtype=torch.float32, device=logits.device)   # a view could not be scaled in place
        b.run(logits, renormalize, loss_coef, token_mask)
        ctx.settings = renormalize, loss_coef
        # saved, not kept on ctx: an edit in place is then an error in backward,
        # and the outputs are in no cycle with their own node
        ctx.save_for_backward(logits, b.topk_ids, b.expert_counts, b.routed_tokens)
        ctx.mark_non_differentiable(b.topk_ids, b.expert_counts)
        return b.topk_ids, b.topk_weights, b.expert_counts, b.loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, _ids, grad_weights, _counts, grad_loss):
        logits, ids, counts, routed = ctx.saved_tensors
        grad = torch.empty_like(logits)
        moe.moe_route_backward(logits, ids, counts, routed, grad_weights.float().contiguous(),
                               grad_loss.float().reshape(1).contiguous(), grad, *ctx.settings)
        return grad, None, None, None, None


def route(logits: torch.Tensor, K: int, renormalize: bool = True, loss_coef: float = 1.0,
          token_mask: torch.Tensor | None = None):
    """Router logits [T, E] to (topk_ids, topk_weights, expert_counts, loss);
    topk_weights and loss carry gradients to the logits.  The gradient needs
    topk_ids and expert_counts as they are: to drop entries, edit a copy
    (``topk_ids.masked_fill(full, -1)``); after an edit in place backward
    raises."""
    return _Route.apply(logits, K, renormalize, loss_coef, token_mask)


class Int8Experts:
    """The experts of one layer: gate_up [E, 2 I, H] and down [E, H, I].

    ``dev_error``, [3] int32 on the device, holds the last call's error words:
    the layout's (MOE_DEV_ERR_EXPERT_RANGE where an id is -1) and the two
    products', whose MOE_DEV_ERR_TIMEOUT says that the output is unspecified."""

    def __init__(self, gate_up: torch.Tensor, down: torch.Tensor, ranks: int = 1):
        E, two_i, H = gate_up.shape
        if down.shape != (E, H, two_i // 2) or two_i % 2:
            raise ValueError("Int8Experts: gate_up must be [E, 2 I, H] and down [E, H, I]")
        self.E, self.H, self.I, self.R = E, H, two_i // 2, ranks
        self.gate_up, self.gate_up_scales = quantize_channels(gate_up)
        self.down, self.down_scales = quantize_channels(down)
        self.dev_error = None

    def __call__(self, x: torch.Tensor, topk_ids: torch.Tensor,
                 topk_weights: torch.Tensor) -> torch.Tensor:
        """x [T, H] bf16 and its routing to [T, H] bf16; under no_grad, or with
        inputs that do not require a gradient."""
        if torch.is_grad_enabled() and (x.requires_grad or topk_weights.requires_grad):
            raise RuntimeError("Int8Experts has no gradient: detach x and topk_weights, or call it under no_grad")
        (T, H), K, dev = x.shape, topk_ids.shape[1], x.device
        rows = T * K
        # every call has words of its own; products of no rows do not write theirs
        self.dev_error = err = (torch.empty if rows else torch.zeros)(3, dtype=torch.int32, device=dev)
        lay = moe.LayoutBuffers(T, K, self.E, self.R, device=dev)
        lay.dev_error = err[:1]
        lay.run(topk_ids)
        codes = torch.empty((rows, H), dtype=torch.int8, device=dev)
        scales = torch.empty(rows, dtype=torch.float32, device=dev)
        moe.moe_dispatch_int8(x, lay.dst_row, codes, scales)
        mid = torch.empty((rows, 2 * self.I), dtype=torch.bfloat16, device=dev)
        moe.moe_expert_matmul_int8(codes, scales, self.gate_up, self.gate_up_scales,
                                   lay.expert_offsets, mid, err[1:2])
        act = torch.nn.functional.silu(mid[:, :self.I]) * mid[:, self.I:]
        codes = torch.empty((rows, self.I), dtype=torch.int8, device=dev)
        same = torch.arange(rows, dtype=torch.int32, device=dev).view(rows, 1)
        moe.moe_dispatch_int8(act, same, codes, scales)
        out_rows = torch.empty((rows, H), dtype=torch.bfloat16, device=dev)
        moe.moe_expert_matmul_int8(codes, scales, self.down, self.down_scales,
                                   lay.expert_offsets, out_rows, err[2:])
        out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        moe.moe_combine(out_rows, topk_weights, lay.dst_row, out)
        return out
