"""moe_route and moe_route_backward against their definition in 64 bits.

Tolerances, from the arithmetic: x - m rounds to a relative 2^-24, so exp has a
relative error of |x - m| 2^-24 + 2 ulp, at most 4e-6 for |x - m| <= 60; the
row's sum, the quotients and the sums over tokens (short chains a lane, then a
tree) add less than as much again: 8e-6 relative for weights and loss.  A
gradient entry is a difference of terms with that error each, so its error is
at most 1.6e-5 of the sum of the terms' magnitudes; a bf16 gradient has to lie
between the roundings of that interval's ends (rounding keeps the order)."""
import numpy as np
import pytest
import torch

import combine_moe_layout_05_gb300 as moe

pytestmark = pytest.mark.gpu

REL = 8e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_moe_layout_05_gb300 import build
    build.build()
    moe.load()


def reference(x, K, renorm, coef, mask=None):
    """numpy, 64 bits, token by token."""
    T, E = x.shape
    p = np.zeros((T, E))
    ids = np.full((T, K), -1, np.int64)
    w = np.zeros((T, K))
    for t in range(T):
        live = np.flatnonzero(x[t] > -np.inf) if mask is None or mask[t] else np.array([], int)
        if live.size == 0:
            continue
        z = np.exp(x[t, live] - x[t, live].max())
        p[t, live] = z / z.sum()
        chosen = live[np.argsort(-x[t, live], kind="stable")][:K]
        ids[t, :chosen.size] = chosen
        w[t, :chosen.size] = p[t, chosen]
        if renorm:
            w[t] /= w[t].sum()
    counts = np.bincount(ids[ids >= 0], minlength=E)
    n = int((ids[:, 0] >= 0).sum())
    loss = coef * E * (counts / (K * max(n, 1)) * p.sum(0) / max(n, 1)).sum()
    return p, ids, w, counts, n, loss


def gradient(p, ids, w, counts, n, renorm, coef, dw, dl):
    """The formula, and the sum of its terms' magnitudes."""
    T, E = p.shape
    K = ids.shape[1]
    a = dl * coef * E * counts / (K * max(n, 1) ** 2)
    g = p * (a - (p * a).sum(1, keepdims=True))
    big = p * (np.abs(a) + (p * np.abs(a)).sum(1, keepdims=True))
    inner = (w * dw).sum(1, keepdims=True)
    ibig = (w * np.abs(dw)).sum(1, keepdims=True)
    if not renorm:
        g -= p * inner
        big += p * ibig
    for k in range(K):
        t = np.flatnonzero(ids[:, k] >= 0)
        e = ids[t, k]
        v = w[t, k] * (dw[t, k] - (inner[t, 0] if renorm else 0))
        np.add.at(g, (t, e), v)
        np.add.at(big, (t, e), w[t, k] * (np.abs(dw[t, k]) + (ibig[t, 0] if renorm else 0)))
    return g, big


def make(T, E, dtype, seed, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, E), generator=g) * scale).to(dtype)


def run(x, K, renorm, coef, mask=None, stream=None):
    b = moe.RouteBuffers(x.shape[0], K, x.shape[1])
    for t in (b.topk_ids, b.expert_counts, b.routed_tokens):
        t.fill_(-77)
    b.topk_weights.fill_(float("nan"))
    b.workspace.fill_(0xAB)
    return b.run(x, renorm, coef, mask, stream)


def check(x, K, renorm, coef=0.01, mask=None, seed=0):
    xd = x.cuda()
    md = None if mask is None else torch.from_numpy(mask).cuda()
    b = run(xd, K, renorm, coef, md)
    x64 = x.double().numpy()
    p, ids, w, counts, n, loss = reference(x64, K, renorm, coef, mask)
    assert np.array_equal(b.topk_ids.cpu().numpy(), ids)
    assert np.array_equal(b.expert_counts.cpu().numpy(), counts)
    assert b.routed_tokens.item() == n
    assert np.all(np.abs(b.topk_weights.cpu().double().numpy() - w) <= REL * w + 1e-37)
    assert abs(b.loss.item() - loss) <= REL * loss
    rng = np.random.default_rng(seed)
    dw = rng.standard_normal(w.shape).astype(np.float32)
    dl = np.float32(0.7)
    grad = torch.full_like(xd, float("nan"))
    b.backward(xd, torch.from_numpy(dw).cuda(), torch.full((1,), float(dl), device="cuda"), grad, renorm, coef)
    g, big = gradient(p, ids, w, counts, n, renorm, coef, dw.astype(float), float(dl))
    tol = 2 * REL * big + 1e-37
    got = grad.cpu().double().numpy()
    low, high = (torch.from_numpy(v.astype(np.float32)).to(x.dtype).double().numpy() for v in (g - tol, g + tol))
    assert np.all((low <= got) & (got <= high)), float(np.maximum(low - got, got - high).max())
    return b


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,K", [(1, 8, 2), (1, 256, 8), (3, 1, 1), (9, 33, 32), (17, 64, 6), (65, 65, 4),
                                   (128, 256, 8), (300, 384, 8), (40, 513, 8), (33, 1024, 32), (2500, 128, 8)])
def test_shapes(T, E, K, renorm, dtype):
    check(make(T, E, dtype, T * 7 + E), K, renorm)


def test_ties_take_the_lowest_index():
    x = torch.zeros(6, 100)
    x[1, 50:] = 1.0
    x[2, ::3] = -0.0                      # the two zeros are equal
    x[3] = -5.0
    x[4, 99] = x[4, 0] = 2.0
    x[5, 40:60] = torch.arange(20).div(4, rounding_mode="floor").float()
    check(x, 8, True)
    check(x.to(torch.bfloat16), 8, False)


@pytest.mark.parametrize("renorm", [True, False])
def test_closed_experts_and_masked_tokens(renorm):
    x = make(50, 40, torch.float32, 3)
    x[:, 5] = x[:, 17] = -torch.inf
    x[3] = -torch.inf                     # nothing is left
    x[4, :35] = -torch.inf                # fewer open (5) than K
    x[4, 36] = -torch.inf
    x[7] = torch.finfo(torch.float32).min # the type's lowest value is an ordinary logit
    x[8, 1:] = torch.finfo(torch.float32).min
    mask = np.ones(50, bool)
    mask[10:20] = mask[49] = False
    x[11] = torch.nan                     # in masked places they do not matter
    x[12, 3] = torch.inf
    ref = x.clone()
    ref[11] = ref[12] = 0.0
    b = check(ref, 6, renorm, mask=mask)
    c = run(x.cuda(), 6, renorm, 0.01, torch.from_numpy(mask).cuda())
    for name in ("topk_ids", "topk_weights", "expert_counts", "routed_tokens", "loss"):
        assert torch.equal(getattr(b, name), getattr(c, name)), name
    grad = torch.full_like(x, torch.nan).cuda()
    c.backward(x.cuda(), torch.ones(50, 6, device="cuda"), None, grad, renorm, 0.01)
    assert torch.count_nonzero(grad[torch.from_numpy(~mask).cuda()]) == 0
    assert torch.count_nonzero(grad[3]) == 0 and bool(torch.isfinite(grad).all())


def test_every_token_masked_and_no_token():
    x = make(20, 16, torch.float32, 1).cuda()
    b = run(x, 4, True, 1.0, torch.zeros(20, dtype=torch.bool, device="cuda"))
    assert bool((b.topk_ids == -1).all()) and torch.count_nonzero(b.topk_weights) == 0
    assert b.loss.item() == 0 and b.routed_tokens.item() == 0 and torch.count_nonzero(b.expert_counts) == 0
    grad = torch.full_like(x, torch.nan)
    b.backward(x, torch.ones(20, 4, device="cuda"), torch.ones(1, device="cuda"), grad)
    assert torch.count_nonzero(grad) == 0
    b = run(x[:0], 4, True, 1.0)
    assert b.loss.item() == 0 and b.routed_tokens.item() == 0 and torch.count_nonzero(b.expert_counts) == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("renorm", [True, False])
def test_bad_logits_show(bad, renorm):
    x = make(12, 24, torch.float32, 2)
    x[5, 7] = bad
    b = run(x.cuda(), 4, renorm, 1.0)
    w = b.topk_weights.cpu()
    assert bool(torch.isnan(w[5]).all()) and bool(torch.isfinite(w[torch.arange(12) != 5]).all())
    assert np.isnan(b.loss.item())
    ids = b.topk_ids.cpu()
    assert bool(((ids >= 0) & (ids < 24)).all())
    if bad != bad:
        assert not bool((ids[5] == 7).any())


def test_gradient_against_differences():
    """Central differences of the 64-bit forward, with the choice and the counts held."""
    T, E, K, coef, h = 5, 12, 3, 0.5, 1e-6
    x = make(T, E, torch.float32, 4)
    dw = np.random.default_rng(0).standard_normal((T, K))
    for renorm in (True, False):
        b = run(x.cuda(), K, renorm, coef)
        grad = torch.empty(T, E, device="cuda")
        b.backward(x.cuda(), torch.from_numpy(dw).float().cuda(), torch.ones(1, device="cuda"), grad, renorm, coef)
        ids, counts = b.topk_ids.cpu().numpy(), b.expert_counts.cpu().numpy()

        def value(z):
            q = np.exp(z - z.max(1, keepdims=True))
            q /= q.sum(1, keepdims=True)
            w = np.take_along_axis(q, ids, 1)
            if renorm:
                w = w / w.sum(1, keepdims=True)
            return (w * dw.astype(np.float32)).sum() + coef * E * (counts / (K * T) * q.sum(0) / T).sum()
        x64 = x.double().numpy()
        for t in range(T):
            for e in range(E):
                up, down = x64.copy(), x64.copy()
                up[t, e] += h
                down[t, e] -= h
                # differences: h^2 of the third derivative and 1e-16 / h of rounding, about 1e-9
                assert abs(grad[t, e].item() - (value(up) - value(down)) / (2 * h)) < 1e-5


def test_parts_of_the_gradient_and_repeated_ids():
    x = make(30, 20, torch.float32, 6).cuda()
    b = run(x, 4, False, 1.0)
    dw, dl = torch.randn(30, 4, device="cuda"), torch.ones(1, device="cuda")
    both, a, c = (torch.empty_like(x) for _ in range(3))
    b.backward(x, dw, dl, both, False)
    b.backward(x, dw, None, a, False)
    b.backward(x, None, dl, c, False)
    assert torch.allclose(both, a + c, rtol=0, atol=1e-6)
    # the caller's own ids, one twice: both entries' parts are added
    b.topk_ids[3] = torch.tensor([7, 2, 7, 7], device="cuda")
    b.backward(x, dw, None, a, False)
    p = torch.softmax(x[3].double(), 0)
    d = dw[3].double()
    g = torch.zeros(20, dtype=torch.float64, device="cuda")
    for k, e in enumerate([7, 2, 7, 7]):
        g -= p * p[e] * d[k]
        g[e] += p[e] * d[k]
    assert torch.allclose(a[3].double(), g, rtol=0, atol=1e-5)


def test_same_bits_again_on_another_stream_and_in_a_graph():
    x = make(5000, 96, torch.float32, 8).cuda()
    first = run(x, 8, True, 1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = run(x, 8, True, 1.0)
    with torch.cuda.stream(side):
        second.topk_weights.zero_()
        second.run(x, True, 1.0)
    torch.cuda.current_stream().wait_stream(side)
    third = moe.RouteBuffers(5000, 8, 96)
    third.run(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third.run(x)
    third.loss.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for other in (second, third):
        for name in ("topk_ids", "topk_weights", "expert_counts", "routed_tokens", "loss"):
            assert torch.equal(getattr(first, name), getattr(other, name)), name


def test_counts_are_the_layouts():
    x = make(3000, 64, torch.bfloat16, 9).cuda()
    b = run(x, 6, True, 1.0)
    lay = moe.LayoutBuffers(3000, 6, 64, 8).run(b.topk_ids)
    assert torch.equal(lay.expert_counts, b.expert_counts) and lay.dev_error.item() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,K", [(70, 64, 4), (70, 250, 8), (700, 384, 8), (9, 512, 3)])
def test_rows_off_the_16_byte_grid(T, E, K, dtype):
    """Views that start one value in: the same results as aligned copies, bit for bit."""
    x = make(T, E, dtype, 5).cuda()
    flat = torch.empty(T * E + 1, dtype=dtype, device="cuda")
    view = flat[1:].view(T, E)
    view.copy_(x)
    a, b = run(x, K, True, 0.1), run(view, K, True, 0.1)
    assert torch.equal(a.topk_ids, b.topk_ids) and torch.equal(a.expert_counts, b.expert_counts)
    assert torch.allclose(a.topk_weights, b.topk_weights, rtol=REL, atol=0)
    assert abs(a.loss.item() - b.loss.item()) <= REL * a.loss.item()
    dw, dl = torch.randn(T, K, device="cuda"), torch.ones(1, device="cuda")
    ga, gb = torch.empty_like(x), torch.empty(T * E + 1, dtype=dtype, device="cuda")[1:].view(T, E)
    a.backward(x, dw, dl, ga, True, 0.1)
    b.backward(view, dw, dl, gb, True, 0.1)
    # each side is within 2 REL of its terms' magnitudes, at most 3 |dw| here; bf16 rounds by 2^-8
    tol = 4 * REL * 3 * dw.abs().max() + (2.0 ** -7 * ga.float().abs() if dtype == torch.bfloat16 else 0)
    assert bool(((ga.float() - gb.float()).abs() <= tol).all())


def test_past_32_bit_offsets():
    """More than 2^31 logits: the last rows' addresses need 64 bits."""
    E, K, tail = 256, 4, 500
    T = 2 ** 31 // E + tail
    x = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    last = make(tail, E, torch.bfloat16, 3)
    x[T - tail:] = last.cuda()
    b = run(x, K, True, 1.0)
    p, ids, w, counts, n, loss = reference(last.double().numpy(), K, True, 1.0)
    assert np.array_equal(b.topk_ids[T - tail:].cpu().numpy(), ids)
    assert np.all(np.abs(b.topk_weights[T - tail:].cpu().double().numpy() - w) <= REL * w)
    assert bool((b.topk_ids[: T - tail] == torch.arange(K, device="cuda")).all())
    total = counts.copy()
    total[:K] += T - tail
    assert np.array_equal(b.expert_counts.cpu().numpy(), total) and b.routed_tokens.item() == T
    grad = torch.full_like(x, torch.nan)
    dw = torch.zeros((T, K), device="cuda")
    dw[T - 1, 0] = 1.0
    b.backward(x, dw, None, grad)
    assert torch.count_nonzero(grad[: T - 1]) == 0
    want = np.zeros(E)
    want[ids[-1]] -= w[-1] * w[-1, 0]
    want[ids[-1, 0]] += w[-1, 0]
    got = grad[T - 1].cpu().double().numpy()
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 4 * REL)
