"""moe_dispatch_int8 against its definition: the scale (a product with the fp32
1/127) and the quotient are single IEEE fp32 operations, so codes and scales are compared bit for bit."""
import numpy as np
import pytest
import torch

import combine_moe_layout_05_gb300 as moe

from gpu_util import i32_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_moe_layout_05_gb300 import build
    build.build()
    moe.load()


def reference(x, dst, rows):
    """numpy fp32 (IEEE): packed codes and scales; -99 and NaN where nothing is written."""
    T, H = x.shape
    q = np.full((rows, H), -99, np.int8)
    s = np.full(rows, np.nan, np.float32)
    amax = np.abs(x).max(1).astype(np.float32)
    for t in range(T):
        scale = np.float32(amax[t] * (np.float32(1) / np.float32(127)))
        code = np.zeros(H, np.int8)
        if not np.isfinite(amax[t]):
            scale = np.float32(np.nan)
        elif scale > 0:
            code = np.clip(np.rint(x[t] / scale), -127, 127).astype(np.int8)
        for r in dst[t]:
            if 0 <= r < rows:
                q[r], s[r] = code, scale
    return q, s


def run(x, dst):
    T, H = x.shape
    K = dst.shape[1]
    q = torch.full((T * K, H), -99, dtype=torch.int8, device="cuda")
    s = torch.full((T * K,), float("nan"), device="cuda")
    moe.moe_dispatch_int8(x.cuda(), i32_dev(dst), q, s)
    return q.cpu().numpy(), s.cpu().numpy()


def check(x, dst):
    q, s = run(x, dst)
    eq, es = reference(x.float().numpy(), dst, dst.size)
    assert np.array_equal(s.view(np.uint32)[~np.isnan(es)], es.view(np.uint32)[~np.isnan(es)])
    assert np.array_equal(np.isnan(s), np.isnan(es))
    assert np.array_equal(q, eq)


@pytest.mark.parametrize("T,H,K", [(1, 16, 1), (1, 7168, 8), (3, 48, 2), (128, 7168, 8), (33, 4096, 6), (70, 2064, 32),
                                   (5, 8192, 4), (9, 10256, 3), (2, 70000, 2), (1000, 272, 5)])
def test_shapes(T, H, K):
    g = torch.Generator().manual_seed(T + H)
    x = (torch.randn((T, H), generator=g) * torch.exp(3 * torch.randn((T, 1), generator=g))).to(torch.bfloat16)
    check(x, np.random.default_rng(T).permutation(T * K).astype(np.int32).reshape(T, K))


def test_zero_rows_skipped_slots_and_extreme_rows():
    g = torch.Generator().manual_seed(0)
    x = torch.randn((8, 128), generator=g)
    x[0] = 0.0
    x[1] = 0.0
    x[1, 5] = -3.0
    x[2] *= 1e38
    x[3] *= 1e-37
    x[4] = -2.0
    x[5, 17] = float("nan")
    x[6, 100] = -float("inf")
    dst = np.random.default_rng(1).permutation(16).astype(np.int32).reshape(8, 2)
    dst[7, 0] = -1
    dst[4, 1] = 16
    check(x.to(torch.bfloat16), dst)


def test_codes_at_the_ties():
    """Rows whose quotients are at or next to k + 1/2 (scale 1): ties go to even."""
    x = torch.zeros(1, 256)
    x[0, 0] = 127.0
    x[0, 1:200] = torch.arange(199) * 0.5 - 50
    check(x.to(torch.bfloat16), np.zeros((1, 1), np.int32))


def test_subnormal_scale():
    x = torch.full((1, 16), 2.0 ** -126)
    x[0, 3] = -(2.0 ** -130)
    check(x.to(torch.bfloat16), np.zeros((1, 1), np.int32))


def test_side_stream_and_offset_view():
    g = torch.Generator().manual_seed(5)
    x = torch.randn((40, 512), generator=g).to(torch.bfloat16)
    dst = np.random.default_rng(2).permutation(72).astype(np.int32).reshape(36, 2)
    big, d = x.cuda(), i32_dev(dst)
    q = torch.empty((72, 512), dtype=torch.int8, device="cuda")
    s = torch.empty(72, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.moe_dispatch_int8(big[4:], d, q, s)
    side.synchronize()
    eq, es = reference(x[4:].float().numpy(), dst, 72)
    assert np.array_equal(q.cpu().numpy(), eq) and np.array_equal(s.cpu().numpy(), es)


def test_past_32_bit_offsets():
    """More than 2^31 values: the last rows' addresses need 64 bits."""
    T, H = 33000, 65536
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(1)
    tail = torch.randn((6, H), generator=g).to(torch.bfloat16)
    x[T - 6:] = tail.cuda()
    q = torch.full((T, H), -99, dtype=torch.int8, device="cuda")
    s = torch.full((T,), float("nan"), device="cuda")
    moe.moe_dispatch_int8(x, torch.arange(T, dtype=torch.int32, device="cuda").view(T, 1), q, s)
    eq, es = reference(tail.float().numpy(), np.arange(6).reshape(6, 1), 6)
    assert np.array_equal(q[T - 6:].cpu().numpy(), eq) and np.array_equal(s[T - 6:].cpu().numpy(), es)
    assert torch.count_nonzero(s[:T - 6]) == 0 and torch.count_nonzero(q[::997]) <= 6 * H
