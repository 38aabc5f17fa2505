"""moe_route_grouped and its gradient against their definitions in 64 bits.

Ids and counts have to be equal.  A sigmoid score's relative error is at most
(|x| + 8) u, u = 2^-24, a softmax score's (|x - m| + 64) u; renormalising adds
the error of a sum of at most 32 such scores, its 5 additions and a quotient of
2 ulp, and the scale one product: weights are held to twice the score's bound and
16 u.  The loss sums T x E values of that error in fp32; each partial sum is over
at most T terms, in chains of (T / warps + 8 + 8 + 64) additions: 1e-5 relative.
The gradient's terms are products of a few such values: 2 (z + 64) u + 64 u of the
magnitudes' sum, z the largest distance or logit, then one rounding."""
import math

import pytest
import torch

import combine_moe_layout_05_gb300 as moe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
NINF = -math.inf


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_moe_layout_05_gb300 import build
    build.build()
    moe.load()


def scores(x, live, scoring):
    s = torch.sigmoid(x) if scoring == "sigmoid" else torch.softmax(x.masked_fill(~live, NINF), 1).nan_to_num(nan=0.0)
    return s.masked_fill(~live, 0.0)


def choose(x, live, bias, K, scoring, groups, top_groups, group_top):
    c = scores(x, live, scoring)
    key = c + bias.double() if bias is not None else c
    if bias is None and top_groups == groups:
        key = x                                          # the same order, where scores are equal in 64 bits too
    key = key.masked_fill(~live, NINF)
    T, E = x.shape
    if top_groups < groups:
        parts = torch.sort(key.view(T, groups, -1), dim=2, descending=True)[0]
        value = parts[:, :, 0].clone()
        if group_top == 2 and E > groups:
            second = parts[:, :, 1]
            value += torch.where(second > NINF, second, torch.zeros_like(second))
        kept = torch.sort(value, dim=1, descending=True, stable=True)[1][:, :top_groups]
        keep = torch.zeros((T, groups), dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        key = key.masked_fill(~keep.repeat_interleave(E // groups, 1), NINF)
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    return ids[:, :K].masked_fill(top[:, :K] == NINF, -1)


def bound(x, live, scoring):
    if scoring == "sigmoid":
        return (x.abs().masked_fill(~live, 0.0) + 8) * U
    m = x.masked_fill(~live, NINF).amax(1, keepdim=True)
    return ((m - x).masked_fill(~live, 0.0) + 64) * U


def run(x, bias, K, scoring="sigmoid", groups=1, top_groups=1, group_top=2, renorm=True, scale=1.0, coef=0.5, mask=None):
    T, E = x.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    r = dict(topk_ids=torch.full((T, K), -9, **i32), topk_weights=torch.full((T, K), -9.0, device="cuda"),
             expert_counts=torch.full((E,), -9, **i32), routed_tokens=torch.full((1,), -9, **i32),
             loss=torch.full((1,), -9.0, device="cuda"))
    ws = torch.empty(moe.moe_route_grouped_workspace_bytes(T, E), dtype=torch.uint8, device="cuda").fill_(0xAB)
    moe.moe_route_grouped(x, bias, **r, scoring=scoring, groups=groups, top_groups=top_groups, group_top=group_top,
                          renormalize=renorm, scale=scale, loss_coef=coef, token_mask=mask, workspace=ws)
    return r


def check(x, bias, K, scoring="sigmoid", groups=1, top_groups=1, group_top=2, renorm=True, scale=1.0, coef=0.5, mask=None):
    T, E = x.shape
    r = run(x, bias, K, scoring, groups, top_groups, group_top, renorm, scale, coef, mask)
    x = x.double()
    live = x > NINF
    if mask is not None:
        live &= mask[:, None]
    ids = choose(x, live, bias, K, scoring, groups, top_groups, group_top)
    assert torch.equal(r["topk_ids"].long(), ids), (r["topk_ids"].long() != ids).any(1).nonzero()[:5].tolist()
    s = scores(x, live, scoring)
    w = torch.where(ids >= 0, s.gather(1, ids.clamp(min=0)), torch.zeros((), dtype=torch.float64, device="cuda"))
    if renorm:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    off = 2 * bound(x, live, scoring).gather(1, ids.clamp(min=0)).amax(1, keepdim=True) + 16 * U
    assert bool(((r["topk_weights"].double() - scale * w).abs() <= off * (scale * w).abs() + 1e-37).all())
    counts = torch.bincount((ids + 1).reshape(-1), minlength=E + 1)[1:]
    assert torch.equal(r["expert_counts"].long(), counts)
    n = int(live.any(1).sum())
    assert r["routed_tokens"].item() == n
    p = s / s.sum(1, keepdim=True).clamp(min=1e-300)
    loss = coef * E * torch.dot(counts.double(), p.sum(0)).item() / (K * max(n, 1) ** 2)
    assert abs(r["loss"].item() - loss) <= 1e-5 * abs(loss)
    return r


def logits(T, E, seed, dtype=torch.float32, spread=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((T, E), generator=g, device="cuda") * spread).to(dtype)


def steps(E, seed, unit=0.001):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-60, 61, (E,), generator=g, device="cuda").float() * unit


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [True, False])
@pytest.mark.parametrize("T,E,K,groups,top_groups,group_top", [
    (1, 256, 8, 8, 4, 2), (7, 16, 2, 4, 1, 2), (300, 64, 6, 8, 3, 1), (777, 250, 6, 5, 2, 2), (129, 384, 8, 1, 1, 1),
    (1000, 128, 8, 8, 8, 2), (513, 160, 6, 8, 3, 2), (65, 1000, 32, 20, 5, 2), (40, 1024, 31, 32, 16, 1),
    (2000, 512, 8, 16, 4, 2), (33, 33, 5, 11, 7, 2), (90, 24, 3, 12, 2, 2), (50, 32, 1, 32, 5, 2), (17, 5, 5, 1, 1, 2),
    (200, 1, 1, 1, 1, 2), (64, 96, 8, 2, 1, 2),
])
def test_against_the_definition(T, E, K, groups, top_groups, group_top, with_bias, scoring, dtype):
    bias = steps(E, E) if with_bias else None
    check(logits(T, E, T + E, dtype), bias, K, scoring, groups, top_groups, group_top, renorm=T % 2 == 0, scale=2.5)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T", [16384, 4097])
def test_large_batch(T, scoring):
    check(logits(T, 256, T), steps(256, 1), 8, scoring, 8, 4, 2, scale=2.5)
    check(logits(T, 384, T), steps(384, 2), 8, scoring)


@pytest.mark.parametrize("E,groups,top_groups", [(256, 8, 4), (64, 1, 1), (40, 5, 3), (512, 16, 4), (1000, 10, 3)])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_keys_nearer_than_fp32_rounding(E, groups, top_groups, scoring):
    """A bias that undoes the first token's scores: its keys differ by less than a unit in the last place."""
    x = logits(24, E, E)
    s = scores(x.double(), torch.ones_like(x, dtype=torch.bool), scoring)
    check(x, (0.75 - s[0]).float(), 8, scoring, groups, top_groups, 2)
    x[1::2] = x[::2] + 0                                 # the same row again, and one in which two experts change places
    x[3, [0, 1]] = x[2, [1, 0]]
    check(x, (0.75 - s[2]).float(), 8, scoring, groups, top_groups, 1)


@pytest.mark.parametrize("K,groups,top_groups", [(8, 1, 1), (8, 8, 4), (32, 4, 2)])
def test_ties_go_to_the_lowest_index(K, groups, top_groups):
    x = torch.zeros((50, 256), device="cuda")
    check(x, torch.zeros(256, device="cuda"), K, "sigmoid", groups, top_groups)
    check(x, None, K, "softmax", groups, top_groups)
    x = logits(500, 256, 3, torch.bfloat16, 0.5)         # many equal logits
    check(x, torch.zeros(256, device="cuda"), K, "sigmoid", groups, top_groups)
    check(x, steps(256, 4, 0.25).round(), K, "sigmoid", groups, top_groups)


def test_biases_that_differ_by_a_rounding():
    """Two neighbours in fp32 of 0.003: equal keys in fp32, not in exact arithmetic."""
    x = torch.ones((40, 64), device="cuda")
    a = torch.tensor(0.003, device="cuda")
    b = torch.nextafter(a, torch.tensor(1.0, device="cuda"))
    bias = torch.where(torch.arange(64, device="cuda") % 3 == 1, a, b)
    assert a.item() != b.item()
    check(x, bias, 8)
    check(x, bias, 6, "sigmoid", 8, 2, 2)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (8, 3)])
def test_closed_experts_and_masked_tokens(scoring, groups, top_groups):
    x = logits(600, 64, 5)
    x[:, [3, 17, 18]] = NINF
    x[10] = NINF                                         # nothing open
    x[11, 1:] = NINF                                     # one open
    x[12, :40] = NINF                                    # whole groups closed
    x[13] = NINF
    x[13, ::8] = 1.0                                     # one open expert a group
    x[14, :] = NINF
    x[14, 9:12] = 2.0                                    # fewer than K
    mask = torch.rand(600, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") > 0.3
    mask[10:15] = True
    check(x, steps(64, 1), 8, scoring, groups, top_groups, 2, mask=mask)
    check(x, None, 8, scoring, groups, top_groups, 2, renorm=False, mask=mask)
    check(x, steps(64, 1), 8, scoring, groups, top_groups, 1, mask=torch.zeros_like(mask))


def test_scores_far_from_zero():
    """Scores of 1e-30 and of 1 less than a rounding: the bias alone, then the logits, decide."""
    x = logits(200, 64, 6, spread=1.0)
    check(x - 60, steps(64, 2), 8)
    check(x - 60, None, 8)
    check(x + 12, steps(64, 2), 8)
    check(x * 20, steps(64, 2), 8, "softmax")
    check(x + 60, None, 8, renorm=False)                 # equal in 64 bits, ordered by the logits


def test_large_bias():
    bias = torch.linspace(-50, 50, 64, device="cuda")
    check(logits(300, 64, 7), bias[torch.randperm(64, device="cuda")], 8, "sigmoid", 4, 2, 2)


def test_nan_and_infinity():
    x = logits(64, 32, 8)
    x[3, 5] = math.nan
    x[4] = math.nan
    x[5, 7] = math.inf
    for groups, top in ((1, 1), (4, 2)):
        for bias in (None, steps(32, 1)):
            r = run(x, bias, 4, "sigmoid", groups, top)
            ids = r["topk_ids"].long()
            assert 5 not in ids[3].tolist() and bool(torch.isfinite(r["topk_weights"][3]).all())
            assert ids[4].tolist() == [0, 1, 2, 3] and bool(torch.isnan(r["topk_weights"][4]).all())
            if bias is None:
                assert ids[5, 0].item() == 7 or groups == 4
            keep = torch.ones(64, dtype=torch.bool, device="cuda")
            keep[3:5] = False
            good = choose(x.double(), x > NINF, bias, 4, "sigmoid", groups, top, 2)
            assert torch.equal(ids[keep], good[keep]) and bool(torch.isnan(r["loss"]).all())
            assert r["routed_tokens"].item() == 64 and r["expert_counts"].sum().item() == 256
    y = x.clone()
    y[5, 7] = 0
    r = run(y, None, 4, "softmax")
    assert bool(torch.isnan(r["topk_weights"][3:5]).all()) and bool(torch.isfinite(r["topk_weights"][5:]).all())
    for row in (3, 4):
        assert len(set(r["topk_ids"][row].tolist())) == 4 and r["topk_ids"][row].min() >= 0


def test_no_tokens():
    r = run(torch.empty((0, 16), device="cuda"), None, 2)
    assert bool((r["expert_counts"] == 0).all()) and r["loss"].item() == 0 and r["routed_tokens"].item() == 0


@pytest.mark.parametrize("shift", [1, 2, 3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_off_the_16_byte_grid(shift, dtype):
    flat = logits(1, 100 * 64 + 8, shift, dtype).view(-1)
    check(flat[shift:shift + 6400].view(100, 64), steps(64, 1), 6, "sigmoid", 8, 4)


def test_same_bits_every_time_and_as_moe_route():
    x = logits(3000, 128, 9)
    a, b = (run(x, steps(128, 1), 8, "sigmoid", 8, 4) for _ in range(2))
    assert all(torch.equal(a[k], b[k]) for k in a)
    c = run(x, None, 8, "softmax")
    d = moe.RouteBuffers(3000, 8, 128).run(x, loss_coef=0.5)
    assert torch.equal(c["topk_ids"], d.topk_ids) and torch.equal(c["expert_counts"], d.expert_counts)


def reference_gradient(x, live, ids, counts, n, dw, dl, scoring, renorm, scale, coef):
    """The formula, and the sum of its terms' magnitudes."""
    T, E = x.shape
    K = ids.shape[1]
    s = scores(x, live, scoring)
    S = s.sum(1, keepdim=True)
    S = torch.where(S == 0, torch.ones_like(S), S)
    p = s / S
    a = dl * coef * E * counts.double() / (K * max(n, 1) ** 2)
    g, m = (a - (p * a).sum(1, keepdim=True)) / S, (a.abs() + (p * a.abs()).sum(1, keepdim=True)) / S
    taken, at = ids >= 0, ids.clamp(min=0).long()
    w = torch.where(taken, s.gather(1, at), torch.zeros((), dtype=torch.float64, device="cuda"))
    d = torch.where(taken, dw.double() * scale, torch.zeros_like(w))
    dm = d.abs()
    if renorm:
        sk = w.sum(1, keepdim=True).clamp(min=1e-300)
        d, dm = (d - (w / sk * d).sum(1, keepdim=True)) / sk * taken, (dm + (w / sk * dm).sum(1, keepdim=True)) / sk * taken
    g, m = g.scatter_add(1, at, d), m.scatter_add(1, at, dm)
    if scoring == "sigmoid":
        slope = s * torch.sigmoid(-x).masked_fill(~live, 0.0)
        return slope * g, slope * m
    return s * (g - (s * g).sum(1, keepdim=True)), s * (m + (s * m).sum(1, keepdim=True))


def check_gradient(x, K, scoring, renorm, scale=2.5, coef=0.5, mask=None, bias=None, groups=1, top_groups=1, seed=0,
                   loss=True):
    T, E = x.shape
    r = run(x, bias, K, scoring, groups, top_groups, 2, renorm, scale, coef, mask)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dw = torch.randn((T, K), generator=gen, device="cuda")
    dl = torch.full((1,), 100.0, device="cuda") if loss else None
    grad = torch.full_like(x, -9.0)
    moe.moe_route_grouped_backward(x, r["topk_ids"], r["expert_counts"], r["routed_tokens"], dw, dl, grad, scoring=scoring,
                                   renormalize=renorm, scale=scale, loss_coef=coef)
    y = x.double()
    live = y > NINF
    if mask is not None:
        live &= mask[:, None]
    want, size = reference_gradient(y, live, r["topk_ids"].long(), r["expert_counts"], r["routed_tokens"].item(), dw,
                                    100.0 if loss else 0.0, scoring, renorm, scale, coef)
    off = (2 * bound(y, live, scoring).amax(1, keepdim=True) + 192 * U) * size
    rounding = 2.0 ** -8 if x.dtype == torch.bfloat16 else U
    assert bool(((grad.double() - want).abs() <= 1.01 * off + rounding * want.abs() + 1e-37).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,K", [(1, 256, 8), (7, 16, 2), (777, 250, 6), (129, 384, 8), (65, 1000, 32), (3000, 128, 6),
                                   (33, 33, 5), (40, 7, 7), (20, 1, 1)])
def test_gradient(T, E, K, renorm, scoring, dtype):
    check_gradient(logits(T, E, T + E, dtype), K, scoring, renorm, bias=steps(E, 1))


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_gradient_of_closed_masked_and_grouped(scoring):
    x = logits(400, 64, 5)
    x[:, [3, 17]] = NINF
    x[10] = NINF
    x[11, 1:] = NINF
    mask = torch.rand(400, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") > 0.3
    for renorm in (True, False):
        check_gradient(x, 6, scoring, renorm, mask=mask, groups=8, top_groups=3)
        check_gradient(x, 6, scoring, renorm, mask=mask, loss=False)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_by_differences(scoring, renorm):
    """Of the kernel's own outputs, with the choice held: step 1/64, fp32 outputs of
    size 1 off by 64 u (64 u * 64 over the step), third derivatives below 2."""
    x = logits(40, 32, 11)
    K, coef, h = 4, 0.5, 1 / 64
    bias = torch.zeros(32, device="cuda")
    bias[[1, 9, 20, 30]] = 10.0                          # these four are chosen whatever x is
    gen = torch.Generator(device="cuda").manual_seed(1)
    pull = torch.randn((40, K), generator=gen, device="cuda").double()
    r = run(x, bias, K, scoring, renorm=renorm, coef=coef)
    grad = torch.empty_like(x)
    order = r["topk_ids"].long()
    moe.moe_route_grouped_backward(x, r["topk_ids"], r["expert_counts"], r["routed_tokens"], pull.float(),
                                   torch.ones(1, device="cuda"), grad, scoring=scoring, renormalize=renorm, loss_coef=coef)
    pulls = torch.zeros((40, 32), dtype=torch.float64, device="cuda").scatter_(1, order, pull)

    def total(z):
        q = run(z, bias, K, scoring, renorm=renorm, coef=coef)
        return (q["topk_weights"].double() * pulls.gather(1, q["topk_ids"].long())).sum().item() + q["loss"].double().item()
    size = pulls.abs().sum(1).amax().item()
    for t, e in ((0, 1), (0, 2), (3, 9), (17, 30), (39, 31), (20, 20)):
        up, down = x.clone(), x.clone()
        up[t, e] += h
        down[t, e] -= h
        slope = (total(up) - total(down)) / (up[t, e] - down[t, e]).item()
        # one token's weights change; the others' and the loss are equal but for fp32's rounding
        room = 64 * U * 2 * (size + 1) / h + 2 * size * h * h / 6 + 2e-5
        assert abs(slope - grad[t, e].item()) <= room, (t, e)


def test_gradient_without_pulls_is_zero():
    x = logits(50, 64, 1)
    r = run(x, None, 4)
    grad = torch.full_like(x, 9.0)
    moe.moe_route_grouped_backward(x, r["topk_ids"], r["expert_counts"], r["routed_tokens"], None, None, grad)
    assert torch.count_nonzero(grad) == 0


def test_side_stream_and_graph():
    x, bias = logits(2000, 256, 1), steps(256, 1)
    K, T, E = 8, 2000, 256
    i32 = dict(dtype=torch.int32, device="cuda")

    def buffers():
        return [torch.zeros((T, K), **i32), torch.zeros((T, K), device="cuda"), torch.zeros(E, **i32),
                torch.zeros(1, **i32), torch.zeros(1, device="cuda")]
    ws = torch.empty(moe.moe_route_grouped_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")

    def go(b):
        moe.moe_route_grouped(x, bias, *b, groups=8, top_groups=4, workspace=ws)
    a, c = buffers(), buffers()
    go(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go(c)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, c))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(c)
    x.copy_(logits(2000, 256, 2))
    go(a)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, c))
