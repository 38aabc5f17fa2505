"""The grouped router, the bf16 experts and a shared expert run together, forward
and backward, against autograd in 64 bits on the same choice of experts.

Values pass through bf16 at the packed rows' products (twice), the combine and the
shared expert's two products; gradients at as many places and at the inputs.
Each rounding moves a tensor by at most 2^-8 of its size (normwise), and a chain
of n of them, each of which a well-scaled product passes on, by about n 2^-8:
held to 8 2^-8 normwise."""
import pytest
import torch

import combine_moe_layout_05_gb300 as moe

pytestmark = pytest.mark.gpu

TOL = 8 * 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_moe_layout_05_gb300 import build
    build.build()
    moe.load()


def leaf(shape, g, std, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype).requires_grad_()


def swiglu(z):
    a, b = z.chunk(2, -1)
    return a * torch.sigmoid(a) * b


def reference(p, x, ids, bias, scale, coef, mask):
    """The layer and its loss in 64 bits, the choice given."""
    T, (E, H) = x.shape[0], p["router"].shape
    K = ids.shape[1]
    live = torch.ones(T, dtype=torch.bool, device="cuda") if mask is None else mask
    s = torch.sigmoid(x @ p["router"].t()) * live[:, None]
    taken = ids >= 0
    w = torch.where(taken, s.gather(1, ids.clamp(min=0)), torch.zeros((), dtype=torch.float64, device="cuda"))
    w = scale * w / w.sum(1, keepdim=True).clamp(min=1e-300)
    counts = torch.bincount((ids + 1).reshape(-1), minlength=E + 1)[1:]
    n = int(live.sum())
    probs = s / s.sum(1, keepdim=True).clamp(min=1e-300)
    loss = coef * E * (counts.double() / (K * n) * probs.sum(0) / n).sum()
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        y = swiglu(x[t] @ p["gate_up"][e].t() + p["gate_up_bias"][e]) @ p["down"][e].t() + p["down_bias"][e]
        out = out.index_add(0, t, w[t, k, None] * y)
    return out + swiglu(x @ p["shared_gate_up"].t()) @ p["shared_down"].t(), loss


@pytest.mark.parametrize("T,H,I,J,E,K,groups,top,masked", [
    (5, 64, 48, 32, 8, 2, 1, 1, False),
    (130, 264, 104, 72, 16, 4, 4, 2, True),
    (700, 512, 136, 256, 24, 6, 8, 3, True),
])
def test_training_step(T, H, I, J, E, K, groups, top, masked):
    from combine_moe_layout_05_gb300.layer import Experts, move_balance_bias, route_grouped
    g = torch.Generator(device="cuda").manual_seed(T)
    p = dict(router=leaf((E, H), g, H ** -0.5, torch.float32), gate_up=leaf((E, 2 * I, H), g, H ** -0.5),
             down=leaf((E, H, I), g, I ** -0.5), gate_up_bias=leaf((E, 2 * I), g, 0.2, torch.float32),
             down_bias=leaf((E, H), g, 0.2, torch.float32), shared_gate_up=leaf((2 * J, H), g, H ** -0.5),
             shared_down=leaf((H, J), g, J ** -0.5))
    x = leaf((T, H), g, 1.0)
    bias = torch.randint(-20, 21, (E,), generator=g, device="cuda").float() * 0.01
    mask = torch.rand(T, generator=g, device="cuda") > 0.25 if masked else None
    ids, weights, counts, loss = route_grouped(x.float() @ p["router"].t(), K, bias, groups=groups, top_groups=top, scale=1.5,
                                               loss_coef=0.3, token_mask=mask)
    layer = Experts(p["gate_up"], p["down"], p["gate_up_bias"], p["down_bias"], (p["shared_gate_up"], p["shared_down"]))
    out = layer(x, ids, weights)
    pull = torch.randn((T, H), generator=g, device="cuda")
    ((out.float() * pull).sum() + 50 * loss).backward()
    assert layer.dev_error.tolist() == [1 if masked else 0] + [0] * 8
    # the same in 64 bits
    q = {k: v.detach().double().requires_grad_() for k, v in p.items()}
    x64 = x.detach().double().requires_grad_()
    want, want_loss = reference(q, x64, ids.long(), bias, 1.5, 0.3, mask)
    ((want * pull.double()).sum() + 50 * want_loss).backward()

    def near(a, b, name):
        assert float((a.detach().double() - b).norm()) <= TOL * float(b.norm()), name
    near(out, want.detach(), "out")
    assert abs(loss.item() - want_loss.item()) <= 1e-5 * want_loss.item()
    near(x.grad, x64.grad, "x")
    for k in p:
        near(p[k].grad, q[k].grad, k)
    # the balance bias moves against the load
    before = bias.clone()
    move_balance_bias(bias, counts, 0.01)
    mean = counts.float().mean()
    assert torch.equal(bias > before, counts < mean) and torch.equal(bias < before, counts > mean)


def test_serving_matches_training_and_replays():
    from combine_moe_layout_05_gb300.layer import Experts, route_grouped
    g = torch.Generator(device="cuda").manual_seed(3)
    T, H, I, E, K = 40, 256, 112, 16, 4
    gate_up, down, x = leaf((E, 2 * I, H), g, H ** -0.5), leaf((E, H, I), g, I ** -0.5), leaf((T, H), g, 1.0)
    router = torch.randn((E, H), generator=g, device="cuda") / H ** 0.5
    layer = Experts(gate_up, down)

    def run(rows):
        ids, weights, _, _ = route_grouped(rows.float() @ router.t(), K, groups=4, top_groups=2)
        return layer(rows, ids, weights)
    trained = run(x).detach()
    with torch.no_grad():
        assert torch.equal(run(x), trained)
        static, side = x.detach().clone(), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run(static)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run(static)
        for seed in (1, 2):
            static.copy_(torch.randn((T, H), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
            graph.replay()
            assert torch.equal(out, run(static))


def test_one_token_and_no_token():
    from combine_moe_layout_05_gb300.layer import Experts, route_grouped
    g = torch.Generator(device="cuda").manual_seed(4)
    H, I, E, K = 64, 32, 8, 2
    layer = Experts(leaf((E, 2 * I, H), g, 0.1), leaf((E, H, I), g, 0.1))
    for T in (1, 0):
        x = leaf((T, H), g, 1.0)
        ids, weights, _, loss = route_grouped(torch.randn((T, E), generator=g, device="cuda").requires_grad_(), K)
        out = layer(x, ids, weights)
        assert out.shape == (T, H)
        (out.float().sum() + loss).backward()
        assert x.grad.shape == (T, H) and bool(torch.isfinite(layer.gate_up.grad.float()).all())


@pytest.mark.parametrize("activation", ["none", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("frozen", ["", "x", "weights", "bias"])
def test_expert_linear_gradients(activation, frozen):
    from combine_moe_layout_05_gb300.layer import expert_linear
    g = torch.Generator(device="cuda").manual_seed(5)
    counts, H, N = [20, 0, 150, 3], 72, 96
    o = torch.tensor([0, 20, 20, 170, 173], dtype=torch.int32, device="cuda")
    C = N // 2 if activation == "swiglu" else N
    t = dict(x=leaf((173, H), g, 1.0), weights=leaf((4, N, H), g, H ** -0.5), bias=leaf((4, N), g, 0.3, torch.float32),
             residual=leaf((173, C), g, 1.0))
    if frozen:
        t[frozen].requires_grad_(False)
    out = expert_linear(t["x"], t["weights"], o, t["bias"], activation, t["residual"])
    pull = torch.randn((173, C), generator=g, device="cuda")
    (out.float() * pull).sum().backward()
    q = {k: v.detach().double().requires_grad_(v.requires_grad) for k, v in t.items()}
    parts = []
    for e in range(4):
        r = slice(int(o[e]), int(o[e + 1]))
        z = q["x"][r] @ q["weights"][e].t() + q["bias"][e]
        if activation == "swiglu":
            z = swiglu(z)
        elif activation == "silu":
            z = z * torch.sigmoid(z)
        elif activation == "gelu":
            z = torch.nn.functional.gelu(z, approximate="tanh")
        parts.append(z + q["residual"][r])
    (torch.cat(parts) * pull.double()).sum().backward()
    for k in t:
        if k == frozen:
            assert t[k].grad is None
        else:
            assert float((t[k].grad.double() - q[k].grad).norm()) <= TOL * float(q[k].grad.norm()), k


def test_second_derivatives_and_unfit_widths_are_refused():
    from combine_moe_layout_05_gb300.layer import expert_linear, route_grouped
    g = torch.Generator(device="cuda").manual_seed(6)
    o = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    x, w = leaf((4, 16), g, 1.0), leaf((1, 16, 16), g, 1.0)
    grad, = torch.autograd.grad(expert_linear(x, w, o).float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        grad.float().sum().backward()
    with pytest.raises(ValueError):
        expert_linear(x, leaf((1, 12, 16), g, 1.0), o)
    with torch.no_grad():
        assert expert_linear(x, leaf((1, 12, 16), g, 1.0), o).shape == (4, 12)
    logits = torch.randn((4, 8), generator=g, device="cuda").requires_grad_()
    grad, = torch.autograd.grad(route_grouped(logits, 2)[1].square().sum(), logits, create_graph=True)
    with pytest.raises(RuntimeError):
        grad.sum().backward()


def test_edits_of_what_the_gradient_needs_are_errors():
    from combine_moe_layout_05_gb300.layer import expert_linear, route_grouped
    g = torch.Generator(device="cuda").manual_seed(7)
    o = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    x, w = leaf((4, 16), g, 1.0), leaf((1, 16, 16), g, 1.0)
    rows = x * 1
    out = expert_linear(rows, w, o, activation="silu")
    rows.zero_()
    with pytest.raises(RuntimeError):
        out.float().sum().backward()
    logits = torch.randn((4, 8), generator=g, device="cuda").requires_grad_()
    ids, weights, counts, loss = route_grouped(logits, 2)
    ids.fill_(0)
    with pytest.raises(RuntimeError):
        weights.sum().backward()


def test_weights_gradients_of_two_batches_add_up():
    """Autograd adds the second batch's gradients; each is one bf16 rounding off (2^-8), their sum another."""
    from combine_moe_layout_05_gb300.layer import expert_linear
    g = torch.Generator(device="cuda").manual_seed(8)
    w = leaf((2, 32, 24), g, 1.0)
    want = torch.zeros((2, 32, 24), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for counts in ((30, 9), (0, 70)):
        o = torch.tensor([0, counts[0], sum(counts)], dtype=torch.int32, device="cuda")
        x, pull = leaf((sum(counts), 24), g, 1.0), torch.randn((sum(counts), 32), generator=g, device="cuda")
        pull = pull.to(torch.bfloat16)
        expert_linear(x, w, o).backward(pull)
        for e in range(2):
            r = slice(int(o[e]), int(o[e + 1]))
            part = pull[r].double().t() @ x.detach()[r].double()
            want[e] += part
            size[e] += part.abs()
    assert bool(((w.grad.double() - want).abs() <= 2.0 ** -8 * (size + want.abs()) * 1.01 + 1e-5).all())


def test_captured_training_step_replays():
    """Forward and backward of the router, the experts and the shared expert in one graph, replayed on
    new rows, against the same step run eagerly: the layer's sums have one order, so the same bits."""
    from combine_moe_layout_05_gb300.layer import Experts, route_grouped
    g = torch.Generator(device="cuda").manual_seed(9)
    T, H, I, E, K = 50, 128, 72, 8, 2
    leaves = [leaf(s, g, s[-1] ** -0.5) for s in ((E, 2 * I, H), (E, H, I), (2 * 40, H), (H, 40))]
    leaves.append(leaf((E, 2 * I), g, 0.1, torch.float32))
    router = leaf((E, H), g, H ** -0.5, torch.float32)
    layer = Experts(leaves[0], leaves[1], leaves[4], shared=(leaves[2], leaves[3]))
    static, pull = leaf((T, H), g, 1.0), torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)

    def step():
        ids, weights, _, loss = route_grouped(static.float() @ router.t(), K, groups=2, top_groups=1)
        out = layer(static, ids, weights)
        grads = torch.autograd.grad((out.float() * pull).sum() + loss, leaves + [router, static])
        return [out.detach(), loss.detach()] + list(grads)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (1, 2):
        rows = torch.randn((T, H), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")
        with torch.no_grad():
            static.copy_(rows)
        graph.replay()
        # copies: the eager step below is another call of the same layer
        held = [t.clone() for t in got]
        for a, b in zip(held, step()):
            assert torch.equal(a, b)
