"""The bf16 experts' calls and expert_linear where their arguments are unusual:
offsets longer than the experts, values near the type's largest.  Calls that differ
only in what is not used have to give the same bits."""
import math

import pytest
import torch

import combine_moe_layout_05_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_moe_layout_05_gb300 import build
    build.build()
    moe.load()


def normal(shape, seed, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def longer(offsets, tail):
    return torch.cat([offsets, torch.tensor(tail, dtype=torch.int32, device="cuda")])


TAILS = [[0, 0, 0], [70, 70], [4], [0] * 1200]


@pytest.mark.parametrize("activation", ["none", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("tail", TAILS)
def test_offsets_longer_than_the_experts(activation, with_bias, tail):
    from combine_moe_layout_05_gb300.layer import expert_linear
    exact = torch.tensor([0, 40, 40, 70], dtype=torch.int32, device="cuda")

    def step(offsets):
        x, w = normal((70, 72), 1).requires_grad_(), normal((3, 96, 72), 2, 0.1).requires_grad_()
        b = normal((3, 96), 3, dtype=torch.float32).requires_grad_() if with_bias else None
        out = expert_linear(x, w, offsets, b, activation)
        out.backward(normal(out.shape, 4))
        return [out.detach(), x.grad, w.grad] + ([b.grad] if with_bias else [])
    for a, c in zip(step(exact), step(longer(exact, tail))):
        assert torch.equal(a, c)


@pytest.mark.parametrize("activation", ["none", "swiglu"])
@pytest.mark.parametrize("tail", TAILS)
def test_activation_gradient_of_given_experts(activation, tail):
    exact = torch.tensor([2, 40, 40, 68], dtype=torch.int32, device="cuda")
    pre, dy = normal((70, 64), 1), normal((70, 32 if activation == "swiglu" else 64), 2)

    def call(offsets, **kw):
        out = torch.full_like(pre, -77.0)
        moe.moe_expert_activation_backward(pre, dy, offsets, out, activation, **kw)
        return out
    want = call(exact)
    assert bool((want[:2] == -77.0).all()) and bool((want[68:] == -77.0).all()) and not bool((want[2:68] == -77.0).all(1).any())
    assert torch.equal(want, call(longer(exact, tail), E=3)) and torch.equal(want, call(exact, E=3))
    with pytest.raises(ValueError):
        call(exact, E=4)
    with pytest.raises(ValueError):                      # the bias gradient's experts are another number
        call(exact, E=2, grad_bias=torch.empty((3, 64), device="cuda"))


@pytest.mark.parametrize("activation", ["silu", "gelu", "swiglu"])
def test_slopes_at_the_largest_values(activation):
    """Beyond |z| = 100 the slope is 1 or 0 to more than fp32's digits: SiLU's rest is below 1e-41, GELU's 0."""
    far = torch.tensor([100.0, 1e4, 1e10, 1.5e19, 2e19, 1e25, 1e38, 3.3895e38, 0.0], device="cuda")
    z = torch.cat([far, -far]).to(torch.bfloat16).repeat(8, 1).t().contiguous()        # [18, 8]
    rows, dy = z.shape[0], normal(z.shape, 1)
    pre = z if activation != "swiglu" else torch.cat([z, torch.full_like(z, 2.0)], 1)
    o, out = torch.tensor([0, rows], dtype=torch.int32, device="cuda"), torch.empty_like(pre)
    moe.moe_expert_activation_backward(pre, dy, o, out, activation)
    slope = torch.where(z > 0, 1.0, 0.0) + torch.where(z == 0, 0.5, 0.0)
    want = dy.double() * slope.double() * (2 if activation == "swiglu" else 1)
    assert bool(((out[:, :8].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-37).all())


def slope(z, activation):
    """a'(z) in 64 bits and the magnitude of its terms."""
    if activation == "none":
        return torch.ones_like(z), torch.ones_like(z)
    if activation == "gelu":
        k, c = 2 * math.sqrt(2 / math.pi), 0.044715
        s = torch.sigmoid(k * (z + c * z ** 3))
        return s + z * s * (1 - s) * k * (1 + 3 * c * z * z), 1 + z.abs() * (1 + z * z)
    s = torch.sigmoid(z)
    return s * (1 + z * (1 - s)), 1 + z.abs()


@pytest.mark.parametrize("activation", ["none", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("N", [16, 64, 528, 4112])
@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 17, 1], [127, 128, 129, 0, 700], [4] * 256])
def test_every_activation_gradient_is_within_its_bound(counts, N, activation, with_bias):
    """Each value, so that a NaN is outside: terms that cancel to 2^-17 of their magnitudes (the sigmoid's
    relative error is below (|u| + 6) 2^-24, |z| < 60 here), then one rounding to bf16."""
    E, rows, C = len(counts), sum(counts), N // 2 if activation == "swiglu" else N
    o = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
    z, dy = normal((rows, N), N, 2.0), normal((rows, C), N + 1)
    out, gb = torch.full_like(z, float("nan")), torch.full((E, N), float("nan"), device="cuda") if with_bias else None
    ws = torch.empty(moe.moe_expert_activation_backward_workspace_bytes(rows, N, E), dtype=torch.uint8, device="cuda")
    moe.moe_expert_activation_backward(z, dy, o, out, activation, grad_bias=gb, workspace=ws)
    g, z = dy.double(), z.double()
    if activation == "swiglu":
        a, u = z.chunk(2, 1)
        d, m = slope(a, "silu")
        s = torch.sigmoid(a)
        want, size = torch.cat([g * u * d, g * a * s], 1), torch.cat([(g * u).abs() * m, (g * a).abs()], 1)
    else:
        d, m = slope(z, activation)
        want, size = g * d, g.abs() * m
    off = 1.01 * 2.0 ** -17 * size
    assert bool(((out.double() - want).abs() <= off + 2.0 ** -8 * want.abs()).all())
    if with_bias:
        e = torch.repeat_interleave(torch.arange(E, device="cuda"), torch.tensor(counts, device="cuda"))

        def per_expert(t):
            return torch.zeros((E, N), dtype=torch.float64, device="cuda").index_add_(0, e, t)
        room = per_expert(off) + 1.01 * torch.tensor(counts, device="cuda")[:, None] * 2.0 ** -24 * per_expert(want.abs())
        assert bool(((gb.double() - per_expert(want)).abs() <= room).all())


def off_the_grid(t):
    """The same values, contiguous, two bytes past a multiple of 16."""
    flat = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
    flat[1:] = t.reshape(-1)
    return flat[1:].view(t.shape)


@pytest.mark.parametrize("activation", ["none", "swiglu"])
def test_tensors_and_gradients_off_the_16_byte_grid(activation):
    """Views into larger buffers, and gradients that torch.cat hands on as such views."""
    from combine_moe_layout_05_gb300.layer import expert_linear
    rows, H, N = 50, 72, 96
    C = N // 2 if activation == "swiglu" else N
    o = torch.tensor([0, 20, 50], dtype=torch.int32, device="cuda")
    pull = normal((rows * C,), 9)

    def step(at, front):
        x, w, r = (at(normal(s, i)).requires_grad_() for i, s in enumerate(((rows, H), (2, N, H), (rows, C))))
        out = expert_linear(x, w, o, None, activation, r)
        (torch.cat([pull.new_zeros(front), out.reshape(-1)])[front:] * pull).sum().backward()
        return [out.detach(), x.grad, w.grad, r.grad]
    want = step(lambda t: t, 8)
    for at, front in ((off_the_grid, 8), (lambda t: t, 3), (off_the_grid, 3)):
        assert all(torch.equal(a, c) for a, c in zip(want, step(at, front)))


@pytest.mark.parametrize("activation", ["none", "silu", "gelu"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_activation_gradient_in_its_own_gradients_place(activation, with_bias):
    """grad_pre may be grad_out itself where not gated."""
    o = torch.tensor([2, 100, 100, 297], dtype=torch.int32, device="cuda")
    pre, dy = normal((300, 264), 1), normal((300, 264), 2)
    ws = torch.empty(moe.moe_expert_activation_backward_workspace_bytes(300, 264, 3), dtype=torch.uint8, device="cuda")

    def call(to, src):
        gb = torch.zeros((3, 264), device="cuda") if with_bias else None
        moe.moe_expert_activation_backward(pre, src, o, to, activation, grad_bias=gb, workspace=ws)
        return gb
    want, place = dy.clone(), dy.clone()
    a, b = call(want, dy), call(place, place)
    assert torch.equal(want, place) and (not with_bias or torch.equal(a, b))


def test_experts_when_no_token_is_routed():
    """All ids -1: nothing for the experts, zero gradients, and the shared expert's output alone."""
    from combine_moe_layout_05_gb300.layer import Experts
    T, E, H, N = 20, 4, 64, 32
    leaves = [normal(s, i, 0.1).requires_grad_() for i, s in enumerate(((E, 2 * N, H), (E, H, N), (2 * N, H), (H, N), (T, H)))]
    ids = torch.full((T, 2), -1, dtype=torch.int32, device="cuda")
    weights = torch.ones((T, 2), device="cuda", requires_grad=True)
    alone = Experts(leaves[0], leaves[1])(leaves[4], ids, weights)
    assert not bool(alone.any())
    out = Experts(leaves[0], leaves[1], shared=(leaves[2], leaves[3]))(leaves[4], ids, weights)
    out.backward(torch.ones_like(out))
    assert not bool(leaves[0].grad.any()) and not bool(leaves[1].grad.any()) and not bool(weights.grad.any())
    a, u = (leaves[4].detach().double() @ leaves[2].detach().double().t()).chunk(2, 1)
    want = (a * torch.sigmoid(a) * u) @ leaves[3].detach().double().t()
    assert float((out.detach().double() - want).norm()) <= 3 * 2.0 ** -8 * float(want.norm())
    assert all(bool(t.grad.isfinite().all()) and bool(t.grad.any()) for t in leaves[2:])
