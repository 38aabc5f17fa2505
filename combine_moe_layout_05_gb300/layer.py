"""MoE layers put together from the library's calls.

``route`` and ``route_grouped`` are the routers with their gradients
(moe_route / moe_route_grouped and their backward calls under autograd), for
training and serving.  ``expert_linear`` is the experts' bf16 product with bias,
activation and residual, under autograd, and ``Experts`` a gated MLP of them,
with a shared expert where the model has one:

    moe_layout           slots of the routing
    moe_dispatch         rows packed by expert
    moe_expert_matmul    gate and up projections, SwiGLU  [rows, I]
    moe_expert_matmul    down projection                  [rows, H]
    moe_combine          the routing-weighted sum         [T, H]
    moe_expert_matmul    (shared) gate and up, SwiGLU; down, the routed sum its residual

``Int8Experts``, for serving, is a gated MLP whose experts' weights are int8 with
a scale for each output channel.  It has no gradient, and refuses inputs that
ask for one:

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


class _RouteGrouped(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, bias, K, scoring, groups, top_groups, group_top, renormalize, scale, loss_coef, token_mask):
        T, E = logits.shape
        logits, dev = logits.contiguous(), logits.device
        i32 = dict(dtype=torch.int32, device=dev)
        ids, counts, routed = torch.empty((T, K), **i32), torch.empty(E, **i32), torch.empty(1, **i32)
        weights = torch.empty((T, K), dtype=torch.float32, device=dev)
        loss = torch.empty((), dtype=torch.float32, device=dev)
        workspace = torch.empty(moe.moe_route_grouped_workspace_bytes(T, E), dtype=torch.uint8, device=dev)
        moe.moe_route_grouped(logits, bias, ids, weights, counts, routed, loss, scoring, groups, top_groups, group_top,
                              renormalize, scale, loss_coef, token_mask, workspace)
        ctx.settings = scoring, renormalize, scale, loss_coef
        ctx.save_for_backward(logits, ids, counts, routed)
        ctx.mark_non_differentiable(ids, counts)
        return ids, weights, counts, loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, _ids, grad_weights, _counts, grad_loss):
        logits, ids, counts, routed = ctx.saved_tensors
        grad = torch.empty_like(logits)
        moe.moe_route_grouped_backward(logits, ids, counts, routed, grad_weights.float().contiguous(),
                                       grad_loss.float().reshape(1).contiguous(), grad, *ctx.settings)
        return (grad,) + (None,) * 10


def route_grouped(logits: torch.Tensor, K: int, bias: torch.Tensor | None = None, scoring: str = "sigmoid",
                  groups: int = 1, top_groups: int = 1, group_top: int = 2, renormalize: bool = True,
                  scale: float = 1.0, loss_coef: float = 1.0, token_mask: torch.Tensor | None = None):
    """Router logits [T, E] to (topk_ids, topk_weights, expert_counts, loss) as moe_route_grouped has
    them; topk_weights and loss carry gradients to the logits, the bias (fp32, for the choice alone)
    has none: ``move_balance_bias`` moves it.  As with ``route`` the outputs are not to be edited in place."""
    if bias is not None:
        bias = bias.detach()
    return _RouteGrouped.apply(logits, bias, K, scoring, groups, top_groups, group_top, renormalize, scale, loss_coef,
                               token_mask)


def move_balance_bias(bias: torch.Tensor, expert_counts: torch.Tensor, rate: float) -> torch.Tensor:
    """One step of the balance bias, in place: up by `rate` for experts below the mean of the counts,
    down for those above it."""
    counts = expert_counts.to(bias.dtype)
    with torch.no_grad():
        return bias.add_(torch.sign(counts.mean() - counts), alpha=rate)


def _whole(t: torch.Tensor) -> torch.Tensor:
    """Contiguous and on 16 bytes, as the calls need a matrix.  A view into a larger buffer may be neither,
    and gradients come as such views too (torch.cat's): it is copied."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class _ExpertLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weights, expert_offsets, bias, activation, residual, error, train):
        rows, (E, N, _) = x.shape[0], weights.shape
        x, weights = _whole(x), _whole(weights)
        bias = None if bias is None else bias.contiguous()
        residual = None if residual is None else _whole(residual)
        out = torch.empty((rows, N // 2 if activation == "swiglu" else N), dtype=torch.bfloat16, device=x.device)
        pre = torch.empty((rows, N), dtype=torch.bfloat16, device=x.device) if train and activation != "none" else None
        moe.moe_expert_matmul(x, weights, expert_offsets, out, bias, activation, residual, pre,
                              None if error is None else error[:1])
        ctx.activation, ctx.error = activation, error
        ctx.save_for_backward(x, weights, expert_offsets, pre)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_out):
        x, weights, offsets, pre = ctx.saved_tensors
        need_x, need_w, _, need_bias, _, need_residual = ctx.needs_input_grad[:6]
        grad_out = _whole(grad_out)
        grad_x = grad_w = grad_bias = None
        if need_x or need_w or need_bias:
            rows, (E, N, _) = x.shape[0], weights.shape
            grad_pre, workspace = grad_out, None
            if need_bias:
                grad_bias = torch.empty((E, N), dtype=torch.float32, device=x.device)
                workspace = torch.empty(moe.moe_expert_activation_backward_workspace_bytes(rows, N, E),
                                        dtype=torch.uint8, device=x.device)
            if pre is not None:
                grad_pre = torch.empty_like(pre)
            if pre is not None or need_bias:
                moe.moe_expert_activation_backward(pre, grad_out, offsets, None if pre is None else grad_pre,
                                                   ctx.activation, grad_bias, workspace, E=E)
            if need_x or need_w:
                grad_x = torch.empty_like(x) if need_x else None
                grad_w = torch.empty_like(weights) if need_w else None
                moe.moe_expert_matmul_backward(grad_pre, x, weights, offsets, grad_x, grad_w,
                                               dev_error=None if ctx.error is None else ctx.error[1:2])
        return grad_x, grad_w, None, grad_bias, None, grad_out if need_residual else None, None, None


def expert_linear(x: torch.Tensor, weights: torch.Tensor, expert_offsets: torch.Tensor,
                  bias: torch.Tensor | None = None, activation: str = "none", residual: torch.Tensor | None = None,
                  dev_error: torch.Tensor | None = None) -> torch.Tensor:
    """Packed rows [rows, H] times their experts' weights [E, N, H] (both bf16) as moe_expert_matmul has
    it, with gradients of x, weights, bias (E * N values) and residual.  The rows of no expert are unspecified,
    in the output and in x's gradient.  dev_error, [2] int32: the forward's error word and the backward's."""
    train = torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, weights, bias))
    least = 16 if activation == "swiglu" else 8
    if train and weights.shape[1] % least:
        raise ValueError(f"expert_linear: the gradient needs N % {least} == 0, N is {weights.shape[1]}")
    E, N, _ = weights.shape
    if bias is not None:
        bias = bias.float()
        if bias.shape != (E, N) and bias.numel() == E * N:
            bias = bias.reshape(E, N)
    if residual is not None and residual.shape[:-1] != x.shape[:1] and residual.numel() >= x.shape[0] * residual.shape[-1]:
        residual = residual.reshape(-1, residual.shape[-1])[:x.shape[0]]     # rows to spare: their gradient is 0
    return _ExpertLinear.apply(x, weights, expert_offsets, bias, activation, residual, dev_error, train)


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dst_row):
        packed = torch.empty((dst_row.numel(), x.shape[1]), dtype=torch.bfloat16, device=x.device)
        moe.moe_dispatch(_whole(x), dst_row, packed)
        ctx.save_for_backward(dst_row)
        return packed

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        dst_row, = ctx.saved_tensors
        T, H = dst_row.shape[0], grad.shape[1]
        out = torch.empty((T, H), dtype=torch.bfloat16, device=grad.device)
        # each token's K rows added up
        moe.moe_combine(_whole(grad), torch.ones(dst_row.shape, dtype=torch.float32, device=grad.device), dst_row, out)
        return out, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, topk_weights, dst_row):
        out = torch.empty((dst_row.shape[0], rows.shape[1]), dtype=torch.bfloat16, device=rows.device)
        topk_weights = topk_weights.contiguous()
        moe.moe_combine(_whole(rows), topk_weights, dst_row, out)
        ctx.save_for_backward(rows, topk_weights, dst_row)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        rows, weights, dst_row = ctx.saved_tensors
        need_rows, need_weights, _ = ctx.needs_input_grad
        kept, grad = dst_row >= 0, grad.float()
        at = dst_row.clamp(min=0).long()
        # an entry that has no row gets row 0's index with nothing in it: added, not copied
        grad_rows = torch.zeros_like(rows) if need_rows else None
        grad_weights = torch.empty_like(weights) if need_weights else None
        for k in range(dst_row.shape[1]):
            keep = kept[:, k, None]
            if need_rows:
                g = torch.where(keep, weights[:, k, None] * grad, 0.0)
                grad_rows.index_add_(0, at[:, k], g.to(rows.dtype))
            if need_weights:
                y = torch.where(keep, rows[at[:, k]].float(), 0.0)
                grad_weights[:, k] = (y * grad).sum(1)
        return grad_rows, grad_weights, None


class Experts:
    """A layer of gated experts in bf16, for training and serving: gate_up [E, 2 I, H] and down [E, H, I],
    with biases [E, 2 I] and [E, H] where the model has them.  shared: (gate_up [2 J, H], down [H, J]) of an
    expert that every token goes through.

    ``dev_error``, [9] int32 on the device, holds the last call's error words: the layout's
    (MOE_DEV_ERR_EXPERT_RANGE where an id is -1), then for each of the four products the forward's and
    the backward's, whose MOE_DEV_ERR_TIMEOUT says that the output or the gradient is unspecified.  Every
    call has words of its own, and its backward pass writes there: a step that makes several calls before
    it goes back gives each its words (``experts(x, ids, weights, dev_error=words[i])``), or keeps
    ``dev_error`` after each.

    A training step can be captured into a CUDA graph: after a warm-up on a side stream, with gradients
    from torch.autograd.grad, and with no output of an eager call on the same leaves still alive, since
    PyTorch cannot capture a backward pass that meets such a call's stream."""

    def __init__(self, gate_up: torch.Tensor, down: torch.Tensor, gate_up_bias: torch.Tensor | None = None,
                 down_bias: torch.Tensor | None = None, shared: tuple[torch.Tensor, torch.Tensor] | None = None,
                 ranks: int = 1):
        E, two_i, H = gate_up.shape
        if down.shape != (E, H, two_i // 2) or two_i % 2:
            raise ValueError("Experts: gate_up must be [E, 2 I, H] and down [E, H, I]")
        if shared is not None and (shared[0].dim() != 2 or shared[0].shape[1] != H or shared[0].shape[0] % 2
                                   or shared[1].shape != (H, shared[0].shape[0] // 2)):
            raise ValueError("Experts: shared must be gate_up [2 J, H] and down [H, J]")
        self.E, self.H, self.I, self.R = E, H, two_i // 2, ranks
        self.gate_up, self.down = gate_up, down
        self.gate_up_bias, self.down_bias, self.shared = gate_up_bias, down_bias, shared
        self.dev_error = None

    def __call__(self, x: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                 dev_error: torch.Tensor | None = None) -> torch.Tensor:
        """x [T, H] bf16 and its routing to [T, H] bf16.  dev_error, [9] int32: where this call and its
        backward pass write their error words (None: a new tensor); they are set to 0 first."""
        T, K, dev = x.shape[0], topk_ids.shape[1], x.device
        moe._refuse_other_devices("Experts", (("x", x), ("topk_ids", topk_ids), ("topk_weights", topk_weights)))
        if dev_error is None:
            dev_error = torch.zeros(9, dtype=torch.int32, device=dev)
        elif dev_error.shape != (9,) or dev_error.dtype != torch.int32 or dev_error.device != dev:
            raise ValueError("Experts: dev_error must be [9] int32 on x's device")
        else:
            dev_error.zero_()
        self.dev_error = err = dev_error
        lay = moe.LayoutBuffers(T, K, self.E, self.R, device=dev)
        lay.dev_error = err[:1]
        lay.run(topk_ids)
        rows = _Dispatch.apply(x, lay.dst_row)
        rows = expert_linear(rows, self.gate_up, lay.expert_offsets, self.gate_up_bias, "swiglu", dev_error=err[1:3])
        rows = expert_linear(rows, self.down, lay.expert_offsets, self.down_bias, dev_error=err[3:5])
        out = _Combine.apply(rows, topk_weights, lay.dst_row)
        if self.shared is None:
            return out
        every = torch.zeros(2, dtype=torch.int32, device=dev)
        every[1:].fill_(T)
        mid = expert_linear(x, self.shared[0][None], every, None, "swiglu", dev_error=err[5:7])
        return expert_linear(mid, self.shared[1][None], every, residual=out, dev_error=err[7:])


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
