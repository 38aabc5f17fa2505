"""layer.py on the CPU, with stand-ins for the library's calls: what autograd
keeps and refuses, and what the layer hands to the calls.  The stand-ins compute
the router by PyTorch, so a gradient is compared with one of the same operations
in the same type (equal but for the order of sums, 1e-6)."""
import gc
import weakref

import pytest
import torch

from combine_moe_layout_05_gb300 import _binding, layer


def _outputs(x, ids, counts, renormalize, coef):
    T, E = x.shape
    K = ids.shape[1]
    p = torch.softmax(x, 1)
    w = torch.where(ids >= 0, p.gather(1, ids.long().clamp(min=0)), torch.zeros((), dtype=x.dtype))
    if renormalize:
        w = w / w.sum(1, keepdim=True)
    return w, coef * E * (counts.to(x.dtype) / (K * T) * p.mean(0)).sum()


def _route(logits, topk_ids, topk_weights, expert_counts, routed_tokens, loss, renormalize=True, loss_coef=1.0,
           token_mask=None, workspace=None, stream=None):
    T, E = logits.shape
    K = topk_ids.shape[1]
    topk_ids.copy_(torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :K])
    expert_counts.copy_(torch.bincount(topk_ids.reshape(-1).long(), minlength=E))
    routed_tokens.fill_(T)
    w, value = _outputs(logits, topk_ids, expert_counts, renormalize, loss_coef)
    topk_weights.copy_(w)
    loss.copy_(value)


def _route_backward(logits, topk_ids, expert_counts, routed_tokens, grad_weights, grad_loss, grad_logits,
                    renormalize=True, loss_coef=1.0, stream=None):
    with torch.enable_grad():
        x = logits.detach().requires_grad_()
        w, value = _outputs(x, topk_ids, expert_counts, renormalize, loss_coef)
        grad_logits.copy_(torch.autograd.grad((w * grad_weights).sum() + value * grad_loss.reshape(()), x)[0])


@pytest.fixture
def calls(monkeypatch):
    monkeypatch.setattr(_binding, "moe_route", _route)
    monkeypatch.setattr(_binding, "moe_route_backward", _route_backward)
    monkeypatch.setattr(_binding, "moe_route_workspace_bytes", lambda T, E: 256)


class _Experts:
    """Stand-ins for the layout, int8 and combine calls; `timeouts` are the
    products (0, 1) whose error word is set."""

    def __init__(self, timeouts=()):
        self.timeouts, self.products = timeouts, 0

    def layout(self, topk_ids, E, R, expert_counts, expert_offsets, rank_offsets, src_token, dst_row, dev_error=None,
               workspace=None, stream=None):
        flat = topk_ids.reshape(-1).long()
        kept = flat >= 0
        expert_counts.copy_(torch.bincount(flat[kept], minlength=E))
        expert_offsets[0] = 0
        expert_offsets[1:] = torch.cumsum(expert_counts, 0)
        order = torch.argsort(torch.where(kept, flat, E), stable=True)
        dst = torch.empty_like(flat)
        dst[order] = torch.arange(flat.numel())
        dst_row.copy_(torch.where(kept, dst, -1).view(topk_ids.shape))
        if dev_error is not None:
            dev_error.fill_(0 if bool(kept.all()) else _binding.MOE_DEV_ERR_EXPERT_RANGE)

    def dispatch(self, tokens, dst_row, packed, scales, stream=None):
        for t, k in (dst_row >= 0).nonzero().tolist():
            scale = tokens[t].float().abs().max() / 127
            packed[dst_row[t, k]] = (tokens[t].float() / scale).round().to(torch.int8)
            scales[dst_row[t, k]] = scale

    def product(self, x, x_scales, weights, w_scales, expert_offsets, out, dev_error=None, stream=None):
        if x.shape[0] == 0:
            return
        for e in range(weights.shape[0]):
            r = slice(int(expert_offsets[e]), int(expert_offsets[e + 1]))
            y = x[r].float() @ weights[e].float().t()
            out[r] = (y * x_scales[r, None] * w_scales[e]).to(torch.bfloat16)
        if dev_error is not None:
            dev_error.fill_(_binding.MOE_DEV_ERR_TIMEOUT if self.products in self.timeouts else 0)
        self.products += 1

    def combine(self, expert_out, topk_weights, dst_row, out, stream=None):
        rows = expert_out[dst_row.clamp(min=0).long()].float() * (dst_row >= 0)[..., None]
        out.copy_((rows * topk_weights[..., None]).sum(1))


@pytest.fixture
def experts(calls, monkeypatch):
    def use(timeouts=()):
        e = _Experts(timeouts)
        monkeypatch.setattr(_binding, "moe_layout", e.layout)
        monkeypatch.setattr(_binding, "moe_dispatch_int8", e.dispatch)
        monkeypatch.setattr(_binding, "moe_expert_matmul_int8", e.product)
        monkeypatch.setattr(_binding, "moe_combine", e.combine)
        monkeypatch.setattr(_binding, "moe_layout_workspace_bytes", lambda T, K, E: 256)
        g = torch.Generator().manual_seed(1)
        return layer.Int8Experts(torch.randn((10, 32, 16), generator=g), torch.randn((10, 16, 16), generator=g))
    return use


def _logits(T=6, E=10):
    return torch.randn((T, E), generator=torch.Generator().manual_seed(0)).requires_grad_()


def test_gradient_through_the_stand_ins(calls):
    logits = _logits()
    ids, weights, counts, loss = layer.route(logits, 3, True, 0.5)
    pull = torch.arange(18.0).view(6, 3)
    ((weights * pull).sum() + 2 * loss).backward()
    x = logits.detach().clone().requires_grad_()
    w, value = _outputs(x, ids, counts, True, 0.5)
    ((w * pull).sum() + 2 * value).backward()
    assert torch.allclose(logits.grad, x.grad, rtol=0, atol=1e-6)


@pytest.mark.parametrize("which", ["ids", "counts"])
def test_an_edit_of_what_the_gradient_needs_is_an_error(calls, which):
    """Dropping entries by ids[...] = -1 must not change the gradient of weights
    that were computed with the old ids."""
    ids, weights, counts, loss = layer.route(_logits(), 3)
    (ids if which == "ids" else counts)[2] = -1
    with pytest.raises(RuntimeError, match="inplace operation"):
        (weights.sum() + loss).backward()


def test_edited_copies_weights_and_losses_are_fine(calls):
    logits = _logits()
    ids, weights, _, loss = layer.route(logits, 3, False)
    ids = ids.masked_fill(ids == 1, -1)
    weights *= 2.0
    loss *= 3.0
    (weights.sum() + loss).backward()
    a = logits.grad.clone()
    logits.grad = None
    _, weights, _, loss = layer.route(logits, 3, False)
    (2 * weights.sum() + 3 * loss).backward()
    assert torch.allclose(a, logits.grad, rtol=0, atol=1e-6)


@pytest.mark.parametrize("with_backward", [False, True])
def test_nothing_is_kept_in_a_cycle(calls, with_backward):
    """Buffers and logits go with the last reference, not with the collector."""
    gc.collect()
    gc.disable()
    try:
        ids, weights, counts, loss = layer.route(_logits(), 3)
        node = weakref.ref(weights.grad_fn)
        if with_backward:
            (weights.sum() + loss).backward()
        assert node() is not None
        del ids, weights, counts, loss
        assert node() is None
    finally:
        gc.enable()


def test_a_second_derivative_is_an_error(calls):
    """Not a term that is silently left out."""
    logits = _logits()
    _, weights, _, loss = layer.route(logits, 3)
    total = weights.square().sum() + loss
    (grad,) = torch.autograd.grad(total, logits, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (total + grad.square().sum()).backward()


def test_the_layer_refuses_to_cut_a_graph(experts):
    """It has no gradient: what would lose one is an error, outside no_grad."""
    run = experts()
    x = torch.randn(6, 16).to(torch.bfloat16)
    ids, weights, _, _ = layer.route(_logits(), 3)
    with pytest.raises(RuntimeError, match="no gradient"):
        run(x, ids, weights)
    with pytest.raises(RuntimeError, match="no gradient"):
        run(x.clone().requires_grad_(), ids, weights.detach())
    out = run(x, ids, weights.detach())
    with torch.no_grad():
        assert torch.equal(run(x.clone().requires_grad_(), ids, weights), out)
    assert not out.requires_grad and out.abs().max() > 0


@pytest.mark.parametrize("timeouts", [(), (0,), (1,), (0, 1)])
@pytest.mark.parametrize("dropped", [False, True])
def test_the_layer_keeps_every_error_word(experts, timeouts, dropped):
    """A wait that expired in either product, and the layout's word, can be read after the call."""
    run = experts(timeouts)
    ids, weights, _, _ = layer.route(_logits().detach(), 3)
    if dropped:
        ids = ids.masked_fill(ids == 1, -1)
    run(torch.randn(6, 16).to(torch.bfloat16), ids, weights)
    words = [_binding.MOE_DEV_ERR_EXPERT_RANGE if dropped else 0]
    words += [_binding.MOE_DEV_ERR_TIMEOUT if p in timeouts else 0 for p in (0, 1)]
    assert run.dev_error.dtype == torch.int32 and run.dev_error.tolist() == words


def test_the_error_words_of_no_token(experts):
    run = experts()
    out = run(torch.empty((0, 16), dtype=torch.bfloat16), torch.empty((0, 3), dtype=torch.int32), torch.empty((0, 3)))
    assert out.shape == (0, 16) and run.dev_error.tolist() == [0, 0, 0]


def test_channels_are_quantised_whatever_their_size():
    """127 codes either side of zero, from the largest channels to ones whose
    scale is subnormal; a channel of zeros has scale 0 and codes 0.  A weight is
    its code times the scale to half a scale, and the scale's own rounding (at
    most 2^-150) 127 times."""
    g = torch.Generator().manual_seed(2)
    w = torch.randn((1, 6, 64), generator=g)
    w *= torch.tensor([1e30, 1.0, 1e-30, 1e-36, 1e-38, 0.0])[None, :, None]
    q, scale = layer.quantize_channels(w)
    assert q.abs().amax(2).tolist() == [[127] * 5 + [0]] and scale[0, 5] == 0
    back = q.double() * scale.double()[..., None]
    assert bool(((back - w.double()).abs() <= 0.5001 * scale.double()[..., None] + 128 * 2.0 ** -150).all())
