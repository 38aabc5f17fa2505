"""moe_route_grouped and its gradient in the forms that the widest rows take: 32
values a lane, read one by one where rows are off the 16-byte grid, and 8 at a time
in bf16.  Against the definitions and bounds of test_gpu_route_grouped.py."""
import math

import pytest
import torch

import combine_moe_layout_05_gb300 as moe
from test_gpu_route_grouped import check, check_gradient, logits, scores, steps

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_moe_layout_05_gb300 import build
    build.build()
    moe.load()


# experts, picks, groups: off the grid in both types (not multiples of 4), and on it past 384 and, in bf16, past 512
SIZES = [(257, 8, 1, 1), (333, 6, 9, 4), (383, 8, 1, 1), (495, 8, 15, 3), (1001, 8, 13, 5), (1001, 32, 11, 11), (1023, 7, 31, 2),
         (1022, 1, 2, 1), (448, 8, 8, 3), (1000, 8, 8, 3), (1024, 8, 32, 5), (1024, 31, 1, 1), (520, 8, 13, 6)]


def closed_and_masked(x, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x[:, 5] = -math.inf
    x[torch.rand(x.shape, generator=g, device="cuda") < 0.05] = -math.inf
    x[0] = -math.inf
    x[1, 2:] = -math.inf
    return x, torch.rand(x.shape[0], generator=g, device="cuda") > 0.2


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [True, False])
@pytest.mark.parametrize("E,K,groups,top_groups", SIZES)
def test_choice(E, K, groups, top_groups, with_bias, scoring, dtype):
    bias = steps(E, E) if with_bias else None
    check(logits(301, E, E, dtype), bias, K, scoring, groups, top_groups, 2, renorm=with_bias, scale=2.5)
    x, mask = closed_and_masked(logits(301, E, E + 1, dtype), E)
    check(x, bias, K, scoring, groups, top_groups, 1, scale=2.5, mask=mask)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,K,groups,top_groups", SIZES)
def test_gradient(E, K, groups, top_groups, renorm, scoring, dtype):
    check_gradient(logits(301, E, E, dtype), K, scoring, renorm, bias=steps(E, 1), groups=groups, top_groups=top_groups)
    x, mask = closed_and_masked(logits(301, E, E + 1, dtype), E)
    check_gradient(x, K, scoring, renorm, mask=mask, groups=groups, top_groups=top_groups)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,groups", [(384, 8), (512, 16), (1024, 8)])
def test_rows_that_start_off_the_grid(E, groups, dtype):
    flat = logits(1, 100 * E + 8, E, dtype).view(-1)
    x = flat[1:1 + 100 * E].view(100, E)
    check(x, steps(E, 1), 8, "sigmoid", groups, 3)
    check_gradient(x, 8, "softmax", True, groups=groups, top_groups=3)


@pytest.mark.parametrize("E,groups,top_groups", [(333, 9, 4), (383, 1, 1), (1001, 13, 5)])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_keys_nearer_than_fp32_rounding(E, groups, top_groups, scoring):
    """A bias that undoes the first token's scores: its keys differ by less than a unit in the last place."""
    x = logits(24, E, E)
    s = scores(x.double(), torch.ones_like(x, dtype=torch.bool), scoring)
    check(x, (0.75 - s[0]).float(), 8, scoring, groups, top_groups, 2)
    x[1::2] = x[::2] + 0
    check(x, (0.75 - s[2]).float(), 8, scoring, groups, top_groups, 1)
