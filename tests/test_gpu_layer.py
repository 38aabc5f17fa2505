"""The layer built from the calls: route -> layout -> int8 dispatch -> product
-> gate -> int8 rows -> product -> combine, and the router under autograd.

Up to the combine every step of the plain form is the same single operations
(codes and scales by IEEE division, integer sums below 2^24, one rounding to
bf16), so only the last sum differs: K fp32 terms against 64 bits, at most
(K + 1) 2^-24 of their magnitudes, and the rounding to bf16, 2^-8 of the
result.  Gradients: the terms' errors of the routing tests, 1.6e-5 of the
magnitudes, of which autograd's own fp32 sums may have as much."""
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


def quantize_rows(x):
    s = x.float().abs().amax(1) / 127.0
    q = torch.round(x.float() / torch.where(s == 0, torch.ones_like(s), s)[:, None])
    return q.clamp(-127, 127), s


def product(q, s, w, ws):
    """[n, H] codes with row scales times [N, H] codes with channel scales."""
    return ((q.double() @ w.double().t()).float() * s[:, None] * ws).to(torch.bfloat16)


@pytest.mark.parametrize("T,H,I,E,K", [(1, 64, 48, 8, 2), (37, 256, 112, 16, 4), (300, 512, 144, 24, 6)])
def test_layer(T, H, I, E, K):
    from combine_moe_layout_05_gb300.layer import Int8Experts, route
    g = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    x = rand(T, H).to(torch.bfloat16)
    router, gate_up, down = rand(E, H) / H ** 0.5, rand(E, 2 * I, H) / H ** 0.5, rand(E, H, I) / I ** 0.5
    ids, weights, counts, loss = route(x.float() @ router.t(), K, loss_coef=0.01)
    experts = Int8Experts(gate_up, down)
    out = experts(x, ids, weights)
    q, s = quantize_rows(x)
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for e in range(E):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        mid = product(q[t], s[t], experts.gate_up[e], experts.gate_up_scales[e])
        act = torch.nn.functional.silu(mid[:, :I]) * mid[:, I:]
        y = product(*quantize_rows(act), experts.down[e], experts.down_scales[e]).double()
        w = weights[t, k].double()[:, None]
        want.index_add_(0, t, w * y)
        size.index_add_(0, t, (w * y).abs())
    tol = 2.0 ** -8 * want.abs() + (K + 1) * 2.0 ** -24 * size + 1e-30
    assert bool(((out.double() - want).abs() <= tol).all())
    assert int(counts.sum()) == T * K and float(loss) > 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_under_autograd(dtype):
    from combine_moe_layout_05_gb300.layer import route
    T, E, K, coef = 200, 48, 4, 0.05
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = (torch.randn(T, E, generator=g, device="cuda") * 2).to(dtype).requires_grad_()
    pull = torch.randn(T, K, generator=g, device="cuda")
    ids, w, counts, loss = route(logits, K, True, coef)
    ((w * pull).sum() + 3.0 * loss).backward()
    z = logits.detach().double().requires_grad_()
    p = torch.softmax(z, 1)
    v = p.gather(1, ids.long())
    v = v / v.sum(1, keepdim=True)
    aux = coef * E * (counts.double() / (K * T) * p.mean(0)).sum()
    ((v * pull).sum() + 3.0 * aux).backward()
    # each entry's terms are at most |w| (|pull| + sum w |pull|) and p (a + sum p a)
    a = 3.0 * coef * E * counts.double() / (K * T * T)
    size = p.detach() * (a + (p.detach() * a).sum(1, keepdim=True))
    inner = (v.detach() * pull.abs()).sum(1, keepdim=True)
    size.scatter_add_(1, ids.long(), v.detach() * (pull.abs() + inner))
    tol = 3.2e-5 * size + (2.0 ** -8 * z.grad.abs() if dtype == torch.bfloat16 else 0)
    assert bool(((logits.grad.double() - z.grad).abs() <= tol).all())
    assert logits.grad.dtype == dtype


def test_unrouted_tokens_pass_through_as_zeros():
    """Padding: a masked token's ids are -1, so no expert sees it and its output is 0."""
    from combine_moe_layout_05_gb300.layer import Int8Experts, route
    T, H, I, E, K = 20, 64, 32, 8, 2
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    experts = Int8Experts(torch.randn(E, 2 * I, H, generator=g, device="cuda"),
                          torch.randn(E, H, I, generator=g, device="cuda"))
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    mask[5:9] = False
    logits = torch.randn(T, E, generator=g, device="cuda")
    ids, w, _, _ = route(logits, K, token_mask=mask)
    out = experts(x, ids, w)
    assert torch.count_nonzero(out[5:9]) == 0
    keep = mask.nonzero()[:, 0]
    ids2, w2, _, _ = route(logits[keep], K)
    assert torch.equal(out[keep], experts(x[keep].contiguous(), ids2, w2))
