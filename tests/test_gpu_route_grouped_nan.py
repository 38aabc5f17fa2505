"""moe_route_grouped's choice where keys are NaN or at the ends of fp32: a NaN key
ranks below every number, a group's value with a NaN in it below every number's and
above a group without an open expert, equal ones go to the lowest index."""
import math

import pytest
import torch

import combine_moe_layout_05_gb300 as moe

pytestmark = pytest.mark.gpu

LAST = -1e300                                            # NaN's place: below every number, above what is not open
LOWEST = torch.finfo(torch.float32).min


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_moe_layout_05_gb300 import build
    build.build()
    moe.load()


def choose(x, bias, K, scoring, groups, top_groups, group_top):
    """ids [T, K] by the definition, in 64 bits."""
    x = x.double()
    T, E = x.shape
    live = x != -math.inf
    s = torch.sigmoid(x) if scoring == "sigmoid" else torch.softmax(x.masked_fill(~live, -math.inf), 1)
    c = torch.where(live, (s + bias.double()).nan_to_num(nan=LAST, posinf=math.inf, neginf=-math.inf), -math.inf)
    parts = torch.sort(c.view(T, groups, -1), dim=2, descending=True)[0]
    value = parts[:, :, 0].clone()
    if group_top == 2 and E > groups:
        second = parts[:, :, 1]
        value = torch.where(second == LAST, LAST, torch.where(second > -math.inf, value + second, value))
    kept = torch.sort(value, dim=1, descending=True, stable=True)[1][:, :top_groups]
    keep = torch.zeros((T, groups), dtype=torch.bool, device=x.device).scatter_(1, kept, True)
    alike = bool((bias == bias[0]).all())                # then logits have the keys' order
    key = torch.where(live, x.nan_to_num(nan=LAST, posinf=math.inf, neginf=-math.inf), -math.inf) if alike else c
    key = key.masked_fill(~keep.repeat_interleave(E // groups, 1), -math.inf)
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    return ids[:, :K].masked_fill(top[:, :K] == -math.inf, -1), s


def check(x, bias, K, scoring, groups, top_groups, group_top):
    T, E = x.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, weights = torch.full((T, K), -9, **i32), torch.full((T, K), -9.0, device="cuda")
    counts, routed, loss = torch.full((E,), -9, **i32), torch.full((1,), -9, **i32), torch.full((1,), -9.0, device="cuda")
    ws = torch.empty(moe.moe_route_grouped_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")
    moe.moe_route_grouped(x, bias, ids, weights, counts, routed, loss, scoring=scoring, groups=groups, top_groups=top_groups,
                          group_top=group_top, renormalize=False, workspace=ws)
    b = torch.zeros(E, device="cuda") if bias is None else bias
    want, s = choose(x, b, K, scoring, groups, top_groups, group_top)
    wrong = (ids.long() != want).any(1).nonzero()[:3, 0].tolist()
    assert not wrong, [(t, x[t].tolist(), ids[t].tolist(), want[t].tolist()) for t in wrong]
    picked = torch.where(want >= 0, s.gather(1, want.clamp(min=0)), 0.0)
    assert torch.equal(torch.isnan(weights), torch.isnan(picked))
    assert routed.item() == int((x != -math.inf).any(1).sum())
    assert torch.equal(counts.long(), torch.bincount((want + 1).reshape(-1), minlength=E + 1)[1:])


def rows(T, E, groups, seed):
    """Rows in which groups and experts are closed, and others NaN, at random."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def coin(shape, p):
        return torch.rand(shape, generator=g, device="cuda") < p
    x = torch.randn((T, E), generator=g, device="cuda")
    nan = coin((T, E), 0.5) & coin((T, groups), 0.5).repeat_interleave(E // groups, 1) & coin((T, 1), 0.7)
    nan |= coin((T, groups), 0.2).repeat_interleave(E // groups, 1) & coin((T, 1), 0.5)
    closed = coin((T, E), 0.2) | coin((T, groups), 0.3).repeat_interleave(E // groups, 1)
    return x.masked_fill(nan, math.nan).masked_fill(closed, -math.inf)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("E,groups,top_groups,K", [(32, 8, 1, 4), (32, 8, 3, 5), (96, 12, 2, 6), (256, 8, 4, 8), (512, 16, 2, 8)])
@pytest.mark.parametrize("bias", ["none", "steps"])
def test_nan_in_groups(E, groups, top_groups, K, group_top, scoring, bias):
    g = torch.Generator(device="cuda").manual_seed(E)
    b = None if bias == "none" else torch.randint(-60, 61, (E,), generator=g, device="cuda").float() * 0.001
    check(rows(400, E, groups, E + top_groups), b, K, scoring, groups, top_groups, group_top)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_an_open_group_of_nan_is_before_a_closed_one(scoring):
    x = torch.full((3, 16), -math.inf, device="cuda")
    x[0, 8:12] = math.nan
    x[1, 4:] = 1.0
    x[1, 13] = math.nan
    x[2, [9, 10]] = torch.tensor([math.nan, 1.0], device="cuda")
    check(x, None, 2, scoring, 4, 1, 2)
    check(x, torch.linspace(0, 0.1, 16, device="cuda"), 2, scoring, 4, 1, 2)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("value", [LOWEST, -LOWEST, -2.5e38, 2.5e38])
def test_biases_at_the_ends_of_fp32(value, scoring):
    """Sums of two such keys leave fp32's range; experts with the lowest bias come last, before NaN."""
    x = rows(300, 64, 8, 5)
    bias = torch.zeros(64, device="cuda")
    bias[::3] = value
    bias[8:12] = value
    for top_groups, group_top, K in ((1, 2, 6), (3, 2, 8), (3, 1, 8), (8, 1, 8)):
        check(x, bias, K, scoring, 8, top_groups, group_top)


@pytest.mark.parametrize("renorm", [True, False])
def test_scores_below_the_smallest_number(renorm):
    """Sigmoid scores below 2^-126 are 0: where all of a token's are, so are its weights, its part of the
    loss and its gradient; the choice goes by the logits, or by the bias."""
    T, E, K = 6, 64, 4
    x = -torch.linspace(88, 200, E, device="cuda").repeat(T, 1)
    x[3:, 7] = 1.0
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, weights = torch.empty((T, K), **i32), torch.empty((T, K), device="cuda")
    counts, routed, loss = torch.empty(E, **i32), torch.empty(1, **i32), torch.empty(1, device="cuda")
    ws = torch.empty(moe.moe_route_grouped_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")
    for bias, rest in ((None, [0, 1, 2, 3]), (torch.linspace(0, 0.5, E, device="cuda"), [63, 62, 61, 60])):
        moe.moe_route_grouped(x, bias, ids, weights, counts, routed, loss, renormalize=renorm, workspace=ws)
        assert ids[0].tolist() == rest and ids[5].tolist() == [7] + rest[:3]
        assert not bool(weights[:3].any()) and not bool(weights[3:, 1:].any()) and routed.item() == T
        s = 1 / (1 + math.exp(-1.0))
        assert bool(((weights[3:, 0] - (1.0 if renorm else s)).abs() <= 1e-6).all())
        want = E * 3 / (K * T) * 3 / T                   # expert 7: chosen three times, all of three tokens' probability
        assert abs(loss.item() - want) <= 1e-5 * want
        grad = torch.full_like(x, -9.0)
        moe.moe_route_grouped_backward(x, ids, counts, routed, torch.ones_like(weights), torch.ones(1, device="cuda"), grad,
                                       renormalize=renorm)
        assert not bool(grad[:3].any()) and bool(grad.isfinite().all())
