"""The largest sizes that moe_route, moe_route_backward and
moe_expert_matmul_int8 take: their kernels step through tokens, rows and
channels in 32 bits, a grid's stride or a tile past the last one.  Refused on
the host, before any CUDA call; a size at the limit gets past the size checks
to the next refusal."""
import ctypes

import pytest

import combine_moe_layout_05_gb300 as moe
from combine_moe_layout_05_gb300 import build as moe_build

FAKE = 0x10000            # never dereferenced: the checks come first
P = ctypes.c_void_p
INVALID, ALIGNMENT, WORKSPACE = 1, 2, 4
MOST = 2 ** 31 - 65536
PAST = [MOST + 1, 2 ** 31 - 4864, 2 ** 31 - 16, 2 ** 31 - 2, 2 ** 31 - 1]


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.load()


@pytest.mark.parametrize("T", PAST)
def test_tokens_past_the_limit(lib, T):
    p = P(FAKE)
    assert lib.moe_route(p, 1, T, 1, 1, 1, 1.0, None, p, p, p, p, p, p, 1 << 20, None) == INVALID
    assert lib.moe_route_backward(p, 1, T, 1, 1, 1, 1.0, p, p, p, p, p, p, None) == INVALID
    assert moe.moe_route_workspace_bytes(T, 1) == 0


@pytest.mark.parametrize("n", PAST)
def test_rows_and_channels_past_the_limit(lib, n):
    p = P(FAKE)
    assert lib.moe_expert_matmul_int8(p, p, p, p, p, n, 16, 1, 1, p, None, None) == INVALID
    assert lib.moe_expert_matmul_int8(p, p, p, p, p, 1, 16, n, 1, p, None, None) == INVALID
    assert lib.moe_expert_matmul_int8(p, p, p, p, p, 1, 16, n // 2 + 1, 2, p, None, None) == INVALID


def test_at_the_limit(lib):
    p, off = P(FAKE), P(FAKE + 1)
    assert moe.moe_route_workspace_bytes(MOST, 1) > 0
    assert lib.moe_route(p, 1, MOST, 1, 1, 1, 1.0, None, p, p, p, p, p, p, 0, None) == WORKSPACE
    assert lib.moe_route_backward(p, 1, MOST, 1, 1, 1, 1.0, off, p, p, p, p, p, None) == ALIGNMENT
    assert lib.moe_expert_matmul_int8(p, off, p, p, p, MOST, 16, 1, 1, p, None, None) == ALIGNMENT
    assert lib.moe_expert_matmul_int8(p, off, p, p, p, 1, 16, MOST, 1, p, None, None) == ALIGNMENT
