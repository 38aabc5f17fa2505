"""expert_linear and Experts on the CPU, with stand-ins for the library's calls that
compute what the calls do by PyTorch in 32 bits, from the same arguments and with
the same readings of them.  Gradients of two calls that differ only in what the
calls do not use are equal."""
import pytest
import torch

from combine_moe_layout_05_gb300 import _binding, layer

bf16 = torch.bfloat16


def _aligned(*tensors):
    """The calls refuse matrices that do not start on 16 bytes."""
    for t in tensors:
        if t is not None and t.data_ptr() % 16:
            raise _binding.MoeError("stand-in", 2)


def _activate(z, activation):
    if activation == "swiglu":
        a, u = z.chunk(2, 1)
        return a * torch.sigmoid(a) * u
    if activation == "gelu":
        return torch.nn.functional.gelu(z, approximate="tanh")
    return z * torch.sigmoid(z) if activation == "silu" else z


def _ranges(offsets, E, rows):
    o = [max(0, min(rows, v)) for v in offsets.tolist()[:E + 1]]
    return [(e, slice(o[e], o[e + 1])) for e in range(E) if o[e + 1] > o[e]]


class _Products:
    """Stand-ins for the bf16 experts' calls.  late: the backward products report a wait that ran out."""

    def __init__(self):
        self.late = False

    def matmul(self, x, weights, expert_offsets, out, bias=None, activation="none", residual=None, pre=None, dev_error=None,
               stream=None):
        _aligned(x, weights, out, residual, pre)
        out.fill_(-77.0)
        for e, r in _ranges(expert_offsets, weights.shape[0], x.shape[0]):
            z = x[r].float() @ weights[e].float().t() + (0 if bias is None else bias.view(weights.shape[:2])[e])
            if pre is not None:
                pre[r] = z.to(bf16)
            y = _activate(z, activation)
            out[r] = (y if residual is None else y + residual[r].float()).to(bf16)
        if dev_error is not None:
            dev_error.fill_(0)

    def activation_backward(self, pre, grad_out, expert_offsets, grad_pre, activation, grad_bias=None, workspace=None,
                            stream=None, E=None):
        if E is None:
            E = expert_offsets.numel() - 1 if grad_bias is None else grad_bias.shape[0]
        _aligned(pre, grad_out, grad_pre)
        o = expert_offsets.tolist()
        # without the bias the calls' own reading: one run of rows, from the first expert's to the last one's
        parts = _ranges(expert_offsets, E, grad_out.shape[0]) if grad_bias is not None else [(0, slice(o[0], max(o[0], o[E])))]
        if grad_pre is not None:
            grad_pre.fill_(-77.0)
        if grad_bias is not None:
            grad_bias.zero_()
        for e, r in parts:
            z = grad_out[r].float() if pre is None else pre[r].float()
            with torch.enable_grad():
                z.requires_grad_()
                g, = torch.autograd.grad(_activate(z, activation), z, grad_out[r].float())
            if grad_pre is not None:
                grad_pre[r] = g.to(bf16)
            if grad_bias is not None:
                grad_bias[e] = g.sum(0)

    def matmul_backward(self, grad_pre, x, weights, expert_offsets, grad_x=None, grad_weights=None, accumulate=False,
                        dev_error=None, stream=None):
        _aligned(grad_pre, x, weights, grad_x, grad_weights)
        if grad_x is not None:
            grad_x.fill_(-77.0)
        if grad_weights is not None:
            grad_weights.zero_()
        for e, r in _ranges(expert_offsets, weights.shape[0], x.shape[0]):
            if grad_x is not None:
                grad_x[r] = (grad_pre[r].float() @ weights[e].float()).to(bf16)
            if grad_weights is not None:
                grad_weights[e] = (grad_pre[r].float().t() @ x[r].float()).to(bf16)
        if dev_error is not None:
            dev_error.fill_(_binding.MOE_DEV_ERR_TIMEOUT if self.late else 0)


def _layout(topk_ids, E, R, expert_counts, expert_offsets, rank_offsets, src_token, dst_row, dev_error=None, workspace=None,
            stream=None):
    flat = topk_ids.reshape(-1).long()
    expert_offsets[0] = 0
    expert_offsets[1:] = torch.cumsum(torch.bincount(flat, minlength=E), 0)
    dst = torch.empty_like(flat)
    dst[torch.argsort(flat, stable=True)] = torch.arange(flat.numel())
    dst_row.copy_(dst.view(topk_ids.shape))
    if dev_error is not None:
        dev_error.fill_(0)


def _dispatch(tokens, dst_row, packed, scales=None, fp8=False, stream=None):
    _aligned(tokens, packed)
    packed[dst_row.reshape(-1).long()] = tokens.repeat_interleave(dst_row.shape[1], 0)


def _combine(expert_out, topk_weights, dst_row, out, stream=None):
    _aligned(expert_out, out)
    out.copy_((expert_out[dst_row.long()].float() * topk_weights[..., None]).sum(1))


@pytest.fixture
def products(monkeypatch):
    monkeypatch.setattr(_binding, "moe_status_string", str)
    p = _Products()
    monkeypatch.setattr(_binding, "moe_expert_matmul", p.matmul)
    monkeypatch.setattr(_binding, "moe_expert_activation_backward", p.activation_backward)
    monkeypatch.setattr(_binding, "moe_expert_matmul_backward", p.matmul_backward)
    monkeypatch.setattr(_binding, "moe_expert_activation_backward_workspace_bytes", lambda rows, N, E: 256)
    monkeypatch.setattr(_binding, "moe_layout", _layout)
    monkeypatch.setattr(_binding, "moe_layout_workspace_bytes", lambda T, K, E: 256)
    monkeypatch.setattr(_binding, "moe_dispatch", _dispatch)
    monkeypatch.setattr(_binding, "moe_combine", _combine)
    return p


def _leaf(shape, seed, dtype=bf16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).requires_grad_()


@pytest.mark.parametrize("activation", ["none", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("tail", [[0, 0, 0], [9, 9], [4], [1 << 30]])
def test_offsets_longer_than_the_experts(products, activation, with_bias, tail):
    """What follows the first E + 1 offsets is not read, forward or backward."""
    counts, H, N = [4, 0, 5], 8, 16
    exact = torch.tensor([0, 4, 4, 9], dtype=torch.int32)

    def step(offsets):
        x, w = _leaf((9, H), 1), _leaf((len(counts), N, H), 2)
        b = _leaf((len(counts), N), 3, torch.float32) if with_bias else None
        out = layer.expert_linear(x, w, offsets, b, activation)
        out.backward(torch.ones_like(out))
        return [out.detach(), x.grad, w.grad] + ([b.grad] if with_bias else [])
    for a, c in zip(step(exact), step(torch.cat([exact, torch.tensor(tail, dtype=torch.int32)]))):
        assert torch.equal(a, c)


def test_bias_and_residual_of_other_shapes(products):
    """What the product takes by its size (a flat bias, a residual with rows to spare) has its own shape's gradient."""
    E, rows, H, N = 2, 6, 8, 16
    o = torch.tensor([0, 4, 6], dtype=torch.int32)

    def step(bias_shape, residual_shape):
        x, w = _leaf((rows, H), 1), _leaf((E, N, H), 2)
        b = _leaf((E, N), 3, torch.float32).detach().reshape(bias_shape).requires_grad_()
        r = torch.zeros(residual_shape, dtype=bf16)
        r.view(-1)[:rows * N] = _leaf((rows, N), 4).detach().view(-1)
        r.requires_grad_()
        out = layer.expert_linear(x, w, o, b, "silu", r)
        out.backward(_leaf((rows, N), 5).detach())
        assert b.grad.shape == torch.Size(bias_shape) and r.grad.shape == torch.Size(residual_shape)
        assert not r.grad.view(-1)[rows * N:].any()
        return [out.detach(), x.grad, w.grad, b.grad.view(-1), r.grad.view(-1)[:rows * N]]
    want = step((E, N), (rows, N))
    for bias_shape, residual_shape in (((E * N,), (rows, N)), ((E, 1, N), (rows + 3, N)), ((E, N), (2, rows, N)), ((N, E), (3, 4, N))):
        for a, c in zip(want, step(bias_shape, residual_shape)):
            assert torch.equal(a, c)


@pytest.mark.parametrize("given", [False, True])
def test_error_words_of_two_calls_before_their_backward_passes(products, given):
    """Two micro-batches forward, then both back: each one's words say what became of its gradients."""
    E, T, K, H, N = 4, 6, 2, 16, 16
    g = torch.Generator().manual_seed(1)
    experts = layer.Experts(_leaf((E, 2 * N, H), 1), _leaf((E, H, N), 2), shared=(_leaf((2 * N, H), 3), _leaf((H, N), 4)))
    words = torch.full((2, 9), 7, dtype=torch.int32)
    outs, kept = [], []
    for i in range(2):
        ids = torch.rand((T, E), generator=g).argsort(1)[:, :K].to(torch.int32)
        x = _leaf((T, H), 5 + i)
        outs.append(experts(x, ids, torch.full((T, K), 0.5), **(dict(dev_error=words[i]) if given else {})))
        kept.append(experts.dev_error)
        assert experts.dev_error.tolist() == [0] * 9 and (not given or words[i].tolist() == [0] * 9)
    late = _binding.MOE_DEV_ERR_TIMEOUT
    products.late = True
    outs[0].float().sum().backward()
    products.late = False
    outs[1].float().sum().backward()
    want = [[0] + [0, late] * 4, [0] * 9]
    assert [k.tolist() for k in kept] == want and (not given or words.tolist() == want)


@pytest.mark.parametrize("words", [torch.zeros(8, dtype=torch.int32), torch.zeros(9), torch.zeros((1, 9), dtype=torch.int32)])
def test_unfit_error_words_are_refused(products, words):
    experts = layer.Experts(_leaf((2, 16, 8), 1), _leaf((2, 8, 8), 2))
    with pytest.raises(ValueError):
        experts(_leaf((3, 8), 3), torch.zeros((3, 1), dtype=torch.int32), torch.ones((3, 1)), dev_error=words)


def _off(t):
    """The same values two bytes off the 16-byte grid, and contiguous."""
    flat = torch.zeros(t.numel() + 8, dtype=t.dtype)
    at = 1 + (-flat.data_ptr() // t.element_size()) % 8
    flat[at:at + t.numel()] = t.detach().reshape(-1)
    return flat[at:at + t.numel()].view(t.shape)


@pytest.mark.parametrize("activation", ["none", "silu", "swiglu"])
def test_tensors_off_the_16_byte_grid(products, activation):
    """Inputs that are views into larger buffers, and gradients that autograd hands on as such views (of
    torch.cat's, here behind three other values)."""
    E, rows, H, N = 2, 6, 8, 16
    C = N // 2 if activation == "swiglu" else N
    o = torch.tensor([0, 4, 6], dtype=torch.int32)

    def step(at, tail):
        x, w, r = (at(_leaf(s, i).detach()).requires_grad_() for i, s in enumerate(((rows, H), (E, N, H), (rows, C))))
        out = layer.expert_linear(x, w, o, None, activation, r)
        tail(out).backward()
        return [out.detach(), x.grad, w.grad, r.grad]
    pull = _leaf((rows * C,), 9).detach()

    def behind_others(out):
        return (torch.cat([torch.zeros(3, dtype=bf16), out.reshape(-1)])[3:] * pull).sum()
    want = step(lambda t: t, lambda out: (out.reshape(-1) * pull).sum())
    for got in (step(_off, lambda out: (out.reshape(-1) * pull).sum()), step(lambda t: t, behind_others), step(_off, behind_others)):
        assert all(torch.equal(a, c) for a, c in zip(want, got))


def test_experts_off_the_16_byte_grid(products):
    E, T, K, H, N = 4, 6, 2, 16, 16
    ids = torch.rand((T, E), generator=torch.Generator().manual_seed(1)).argsort(1)[:, :K].to(torch.int32)
    pull = _leaf((T * H,), 9).detach()

    def step(at, front):
        leaves = [at(_leaf(s, i).detach()).requires_grad_() for i, s in
                  enumerate(((E, 2 * N, H), (E, H, N), (2 * N, H), (H, N), (T, H)))]
        out = layer.Experts(leaves[0], leaves[1], shared=(leaves[2], leaves[3]))(leaves[4], ids, torch.full((T, K), 0.5))
        (torch.cat([torch.zeros(front, dtype=bf16), out.reshape(-1)])[front:] * pull).sum().backward()
        return [out.detach()] + [t.grad for t in leaves]
    want = step(lambda t: t, 8)
    for at in (lambda t: t, _off):
        assert all(torch.equal(a, c) for a, c in zip(want, step(at, 3)))
