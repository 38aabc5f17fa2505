"""moe_route and its gradient on rows whose logits are NaN, or number fewer than
K: a NaN logit is open, ranks below every number and shows in the token's
weights, its gradient and what the experts' outputs are combined to.  Nothing is
compared but ids, counts and which values are NaN."""
import numpy as np
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


def expected_ids(row, K):
    """Numbers above -inf, largest first, then NaN, each to the lowest index; -1 after them."""
    numbers = np.flatnonzero(row > -np.inf)
    order = numbers[np.argsort(-row[numbers], kind="stable")]
    ids = np.concatenate([order, np.flatnonzero(np.isnan(row))])[:K]
    return np.concatenate([ids, np.full(K - ids.size, -1)]).astype(np.int32)


def nan_rows(T, E, K, dtype):
    """Rows: 1 all NaN; 2 NaN but for fewer than K numbers; 3 NaN and closed
    experts alone; 4 one NaN, and K - 1 experts open in all; T - 1 masked and NaN."""
    g = torch.Generator().manual_seed(E + K)
    x = torch.randn((T, E), generator=g).to(dtype).float()
    x[1] = torch.nan
    x[2, torch.randperm(E, generator=g)[: E - (K - 1)]] = torch.nan
    x[3] = -torch.inf
    x[3, E // 2] = x[3, E - 1] = torch.nan
    x[4, K - 1:] = -torch.inf
    x[4, 0] = torch.nan
    x[T - 1] = torch.nan
    mask = torch.ones(T, dtype=torch.bool)
    mask[T - 1] = False
    return x.to(dtype), mask


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,K", [(12, 24, 4), (700, 128, 8), (3000, 250, 6), (40, 384, 8), (33, 513, 8),
                                   (20, 1000, 32), (9, 2, 2)])
def test_nan_rows_show(T, E, K, renorm, dtype):
    x, mask = nan_rows(T, E, K, dtype)
    b = moe.RouteBuffers(T, K, E)
    b.run(x.cuda(), renorm, 1.0, mask.cuda())
    rows = x.float().numpy()
    ids = np.stack([expected_ids(rows[t], K) if mask[t] else np.full(K, -1, np.int32) for t in range(T)])
    assert np.array_equal(b.topk_ids.cpu().numpy(), ids)
    assert np.array_equal(b.expert_counts.cpu().numpy(), np.bincount(ids[ids >= 0], minlength=E))
    assert b.routed_tokens.item() == T - 1
    bad = np.isnan(rows).any(1) & mask.numpy()
    w = b.topk_weights.cpu().numpy()
    assert np.array_equal(np.isnan(w), bad[:, None] & (ids >= 0)) and np.all(w[ids < 0] == 0)
    assert np.isnan(b.loss.item())
    grad = torch.zeros((T, E), dtype=dtype, device="cuda")
    b.backward(x.cuda(), torch.ones(T, K, device="cuda"), torch.ones(1, device="cuda"), grad, renorm)
    grad = grad.float().cpu().numpy()
    assert np.isnan(grad[bad]).all() and np.isfinite(grad[~bad]).all() and np.all(grad[T - 1] == 0)


def test_nan_rows_reach_the_layers_output():
    """A NaN hidden state: NaN logits, and NaN where its output is."""
    from combine_moe_layout_05_gb300.layer import Int8Experts, route
    T, H, I, E, K = 30, 64, 32, 8, 2
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    x, router = rand(T, H).to(torch.bfloat16), rand(E, H)
    x[7] = torch.nan
    experts = Int8Experts(rand(E, 2 * I, H), rand(E, H, I))
    ids, weights, _, _ = route(x.float() @ router.t(), K)
    nan = torch.isnan(experts(x, ids, weights))
    assert bool(nan[7].all()) and int(nan.sum()) == H
