"""moe_expert_matmul against 64-bit products.

Products of bf16 values are exact in fp32; the sum's error is held to 2^-23 of
the magnitudes' sum S for every 16 terms (each instruction may round or
truncate to 24 bits), and one such step each for the bias and the start:
d = (H / 16 + 3) 2^-23 S.  The activations' slopes are below 1.13 (SiLU 1.1,
GELU's tanh form 1.13), their own error is a relative (|u| + 6) 2^-24 of the
sigmoid, |u| < 60 here: below 2^-17.  Each output is then rounded to bf16 once:
2^-8 of the value."""
import math

import numpy as np
import pytest
import torch

import combine_moe_layout_05_gb300 as moe

pytestmark = pytest.mark.gpu

SLOPE, OWN, BF16 = 1.13, 2.0 ** -17, 2.0 ** -8
ACTS = ["none", "silu", "gelu", "swiglu"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_moe_layout_05_gb300 import build
    build.build()
    moe.load()


def normal(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)


def offsets_of(counts, first=0):
    o = np.full(len(counts) + 1, first, np.int32)
    o[1:] += np.cumsum(counts).astype(np.int32)
    return torch.from_numpy(o).cuda()


def values(x, w, o, bias):
    """z and the bound on its error, [rows, N] in 64 bits; NaN where no expert owns the row."""
    rows, H = x.shape
    E, N, _ = w.shape
    z = torch.full((rows, N), math.nan, dtype=torch.float64, device="cuda")
    d = z.clone()
    lo = o.tolist()
    for e in range(E):
        a, b = max(0, min(rows, lo[e])), max(0, min(rows, lo[e + 1]))
        if b <= a:
            continue
        xe, we = x[a:b].double(), w[e].double()
        add = bias[e].double() if bias is not None else torch.zeros(N, dtype=torch.float64, device="cuda")
        z[a:b] = xe @ we.t() + add
        d[a:b] = (H / 16 + 3) * 2.0 ** -23 * (xe.abs() @ we.abs().t() + add.abs())
    return z, d


def expected(z, d, act, residual):
    """The output in 64 bits and what the kernel's may be off."""
    def gelu(v):
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if act == "swiglu":
        n = z.shape[1] // 2
        g, u, dg, du = z[:, :n], z[:, n:], d[:, :n], d[:, n:]
        s = g * torch.sigmoid(g)
        y, off = s * u, SLOPE * dg * (u.abs() + du) + s.abs() * du
    elif act == "none":
        y, off = z, d
    else:
        y, off = (z * torch.sigmoid(z) if act == "silu" else gelu(z)), SLOPE * d
    off = off + OWN * y.abs()
    if residual is not None:
        y = y + residual.double()
        off = off + 2.0 ** -24 * y.abs()
    return y, (1 + BF16) * off + BF16 * y.abs()


def check(counts, H, N, act="none", bias=False, residual=False, pre=False, seed=0, spare=0, first=0):
    E, rows = len(counts), first + int(sum(counts)) + spare
    C = N // 2 if act == "swiglu" else N
    o = offsets_of(counts, first)
    x, w = normal((rows, H), seed), normal((E, N, H), seed + 1, H ** -0.5)
    b = torch.randn((E, N), generator=torch.Generator(device="cuda").manual_seed(seed + 2), device="cuda") if bias else None
    r = normal((rows, C), seed + 3) if residual else None
    out = torch.full((rows, C), -77.0, dtype=torch.bfloat16, device="cuda")
    p = torch.full((rows, N), -77.0, dtype=torch.bfloat16, device="cuda") if pre else None
    err = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    moe.moe_expert_matmul(x, w, o, out, bias=b, activation=act, residual=r, pre=p, dev_error=err)
    z, d = values(x, w, o, b)
    y, off = expected(z, d, act, r)
    owned = torch.zeros(rows, dtype=torch.bool, device="cuda")
    owned[first:rows - spare] = True
    worst = ((out.double() - y).abs() - off)[owned]
    assert worst.numel() == 0 or bool((worst <= 0).all()), float(worst.max())
    assert bool((out[~owned] == -77.0).all())
    if pre:
        assert bool(((p.double() - z).abs() <= (1 + BF16) * d + BF16 * z.abs())[owned].all())
        assert bool((p[~owned] == -77.0).all())
    if rows:
        assert err.item() == 0


@pytest.mark.parametrize("H", [8, 64, 72, 128, 520])
@pytest.mark.parametrize("N", [2, 8, 64, 130, 250, 256])
@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 17, 1], [16, 33, 250, 0]])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_small(counts, H, N, act):
    check(counts, H, N, act, seed=H + N)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias,residual,pre", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 1)])
@pytest.mark.parametrize("counts,H,N", [
    ([5, 0, 30, 2], 200, 96),            # a few rows an expert
    ([60, 33, 0, 128], 136, 272),        # tens
    ([700, 129, 1], 264, 528),           # hundreds
    ([7], 2112, 100),                    # the contraction shared out
])
def test_epilogue(counts, H, N, act, bias, residual, pre):
    check(counts, H, N, act, bias, residual, pre, seed=H, spare=3)


@pytest.mark.parametrize("N", [1, 3, 7, 33, 129, 1001])
@pytest.mark.parametrize("counts", [[3, 0, 9], [40, 90], [600, 17], [0, 12]])
def test_odd_channels(counts, N):
    """Rows off the 16-byte grid: stored value by value."""
    check(counts, 104, N, "gelu", True, True, True, seed=N)
    check(counts, 2056, N, "silu", True, True, True, seed=N, spare=1)
    check(counts, 104, 2 * N, "swiglu", True, True, True, seed=N, spare=2)
    check(counts, 2056, 2 * N, "swiglu", True, True, True, seed=N)


@pytest.mark.parametrize("act,H,N", [("swiglu", 1032, 520), ("none", 512, 264), ("gelu", 576, 1024)])
@pytest.mark.parametrize("counts", [
    [1] * 8 + [0] * 24,                                  # one token's experts
    [4] * 256,                                           # a decode batch
    [1000, 0, 3, 515, 64, 127, 128, 129],                # rows around every tile edge
    [0, 0, 0],                                           # nobody
    [4097],                                              # one expert: the plain product
    [31, 32, 33, 63, 64, 65, 255, 256, 257, 511, 513],
])
def test_groups(counts, act, H, N):
    check(counts, H, N, act, True, False, True, seed=len(counts), spare=5)


@pytest.mark.parametrize("each", [1, 40, 300])
def test_the_most_experts(each):
    """The experts' table takes the most shared memory, in each form."""
    check([each + (e % 5 == 0) for e in range(1024)], 48, 24, "swiglu", seed=each)


@pytest.mark.parametrize("rows", [1, 15, 16, 17, 32])
@pytest.mark.parametrize("act,H,N", [("none", 2048, 100), ("swiglu", 4104, 130), ("gelu", 7168, 257)])
def test_contraction_split_over_blocks(rows, act, H, N):
    check([rows], H, N, act, True, True, True, seed=rows + H)
    check([0, rows, 3, 0, 1], H, N, act, False, True, False, seed=rows + N, spare=2)


def test_rows_before_the_first_expert_are_left():
    check([5, 40], 64, 64, "silu", first=7, spare=9)


def test_offsets_outside_the_rows_are_cut():
    x, w = normal((10, 32), 1), normal((3, 16, 32), 2)
    a, b = torch.empty(10, 16, dtype=torch.bfloat16, device="cuda"), torch.empty(10, 16, dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_matmul(x, w, torch.tensor([0, 4, 4, 10], dtype=torch.int32, device="cuda"), a)
    moe.moe_expert_matmul(x, w, torch.tensor([-3, 4, 4, 1000], dtype=torch.int32, device="cuda"), b)
    assert torch.equal(a, b)


def test_no_rows():
    check([0, 0], 64, 32, "none")


@pytest.mark.parametrize("counts,act", [([20, 1], "gelu"), ([90, 70], "none"), ([600], "swiglu"), ([9], "silu")])
def test_residual_in_place(counts, act):
    H, N = 2056, 144
    C = N // 2 if act == "swiglu" else N
    o, rows = offsets_of(counts), sum(counts)
    x, w, r = normal((rows, H), 1), normal((len(counts), N, H), 2, H ** -0.5), normal((rows, C), 3)
    out = torch.empty_like(r)
    moe.moe_expert_matmul(x, w, o, out, activation=act, residual=r)
    moe.moe_expert_matmul(x, w, o, r, activation=act, residual=r)
    assert torch.equal(out, r)


@pytest.mark.parametrize("counts", [[20, 5], [100, 60], [300, 260]])
def test_a_row_of_nan_and_infinity_stays_alone(counts):
    """Neighbours in a tile, of the same expert and of the next, are not touched."""
    H, N = 136, 96
    o, rows = offsets_of(counts), sum(counts)
    x, w = normal((rows, H), 1), normal((2, N, H), 2, H ** -0.5)
    clean, out = (torch.empty((rows, N), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    moe.moe_expert_matmul(x, w, o, clean)
    bad = [2, counts[0] - 1, counts[0]]
    x[bad] = math.nan
    w[1, 5] = math.inf
    moe.moe_expert_matmul(x, w, o, out)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[bad] = False
    assert bool(torch.isnan(out[bad].float()).all())
    same = out[keep] == clean[keep]
    second = torch.arange(rows, device="cuda")[keep] >= counts[0]
    same[second, 5] = True
    assert bool(same.all()) and not bool(torch.isfinite(out[counts[0]:, 5].float()).any())


@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu"])
def test_large_values_before_the_activation(act):
    """z up to 1e5: the sigmoid is 0 or 1, and z or 0 (a zero of its sign) comes out."""
    x = torch.zeros((40, 8), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.tensor([-1e5, -2000.0, -100.0, -90.0, 0.0, 50.0, 100.0, 1e5], device="cuda").repeat(5)
    w = torch.ones((1, 16, 8), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((40, 8 if act == "swiglu" else 16), dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_matmul(x, w, offsets_of([40]), out, activation=act)
    z = x[:, :1].double()
    y, off = expected(z.repeat(1, 2) if act == "swiglu" else z, torch.zeros((40, 2), device="cuda").double(), act, None)
    # below u = -87.3 the power of 2 overflows and the value, under 2^-118 |z|, is 0
    assert bool(((out.double() - y).abs() <= off[:, :1] + 1e-25).all())


def test_weights_past_32_bit_offsets():
    """More than 2^32 weight bytes: the last experts' addresses need 64 bits."""
    E, N, H = 40, 4096, 14336
    counts = [0] * E
    counts[0], counts[E - 1] = 3, 5
    check(counts, H, N, "swiglu", seed=9)


def test_outputs_past_32_bit_offsets():
    rows, H, N = 1_060_000, 16, 2048
    x, w = normal((rows, H), 1), normal((2, N, H), 2)
    o = torch.tensor([0, 1000, rows], dtype=torch.int32, device="cuda")
    out = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_matmul(x, w, o, out)
    for a, b in ((0, 300), (900, 1100), (rows - 3000, rows)):
        part = (o - a).clamp(0, b - a)
        z, d = values(x[a:b], w, part, None)
        assert bool(((out[a:b].double() - z).abs() <= (1 + BF16) * d + BF16 * z.abs()).all())


def test_longest_contraction():
    check([5, 0, 40], 65536, 40, seed=11)
    check([20] * 30, 65536, 24, "swiglu", seed=12)


def test_side_stream_graph_and_repeat():
    x, w, b = normal((300, 512), 1), normal((4, 512, 512), 2, 0.05), torch.randn(4, 512, device="cuda")
    o = torch.tensor([0, 100, 101, 290, 300], dtype=torch.int32, device="cuda")
    a, c = (torch.zeros((300, 256), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def go(to):
        moe.moe_expert_matmul(x, w, o, to, bias=b, activation="swiglu")
    go(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go(c)
    side.synchronize()
    assert torch.equal(a, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(c)
    for n in range(3):
        c.zero_()
        if n == 2:                                       # a replay sees new rows and new ranges
            x.copy_(normal((300, 512), 7))
            o.copy_(torch.tensor([0, 0, 290, 290, 300], dtype=torch.int32))
            go(a)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, c)
