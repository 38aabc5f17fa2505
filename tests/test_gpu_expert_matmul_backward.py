"""moe_expert_matmul_backward and moe_expert_activation_backward against 64 bits.

A sum of n products of bf16 values is held to (n / 16 + 2) 2^-23 of the
magnitudes' sum (test_gpu_expert_matmul.py), then a rounding to bf16 (2^-8) or
one to fp32 (2^-24, and as much for the addition to what was there).  The
activation's gradient: its factors are fp32 with a relative error of the sigmoid
below (|u| + 6) 2^-24; terms that cancel are held to 2^-17 of their magnitudes
(|z| < 60 in the tests: a slope's terms are at most (1 + |z|) and, for GELU, |z|
(1 + z^2))."""
import math

import numpy as np
import pytest
import torch

import combine_moe_layout_05_gb300 as moe

pytestmark = pytest.mark.gpu

BF16, F32 = 2.0 ** -8, 2.0 ** -24


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


def ranges(o, rows):
    lo = [max(0, min(rows, v)) for v in o.tolist()]
    return [(e, lo[e], lo[e + 1]) for e in range(len(lo) - 1) if lo[e + 1] > lo[e]]


def check_products(counts, H, N, f32=False, accumulate=False, seed=0, spare=0, first=0):
    E, rows = len(counts), first + int(sum(counts)) + spare
    o = offsets_of(counts, first)
    g, x, w = normal((rows, N), seed), normal((rows, H), seed + 1), normal((E, N, H), seed + 2, H ** -0.5)
    if spare:
        g[rows - spare:] = math.nan                      # rows of no expert are not read into a sum
        x[rows - spare:] = math.inf
    gx = torch.full((rows, H), -77.0, dtype=torch.bfloat16, device="cuda")
    dt = torch.float32 if f32 else torch.bfloat16
    gw = torch.randn((E, N, H), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dt)
    before = gw.double() if accumulate else torch.zeros((E, N, H), dtype=torch.float64, device="cuda")
    err = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    moe.moe_expert_matmul_backward(g, x, w, o, grad_x=gx, grad_weights=gw, accumulate=accumulate, dev_error=err)
    owned = torch.zeros(rows, dtype=torch.bool, device="cuda")
    owned[first:rows - spare] = True
    assert bool((gx[~owned] == -77.0).all())
    with_rows = {e: (a, b) for e, a, b in ranges(o, rows)}
    for e in range(E):
        if e not in with_rows:
            assert torch.equal(gw[e].double(), before[e])
            continue
        a, b = with_rows[e]
        ge, xe, we = g[a:b].double(), x[a:b].double(), w[e].double()
        y, s = ge @ we, ge.abs() @ we.abs()
        assert bool(((gx[a:b].double() - y).abs() <= 1.01 * (N / 16 + 2) * 2.0 ** -23 * s + BF16 * y.abs()).all()), ("x", e)
        y, s = ge.t() @ xe + before[e], ge.t().abs() @ xe.abs()
        off = 1.01 * ((b - a) / 16 + 2) * 2.0 ** -23 * s + (F32 if f32 else BF16) * y.abs() * (1.01 if f32 else 1.0)
        assert bool(((gw[e].double() - y).abs() <= off).all()), ("w", e)
    assert err.item() == 0


@pytest.mark.parametrize("H", [8, 64, 72, 264])
@pytest.mark.parametrize("N", [8, 64, 136, 264])
@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 17, 1], [16, 33, 250, 0]])
def test_small_products(counts, H, N):
    check_products(counts, H, N, seed=H + N)


@pytest.mark.parametrize("f32,accumulate", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("counts,H,N", [
    ([5, 0, 30, 2], 200, 96),
    ([60, 33, 0, 128, 64], 136, 272),
    ([700, 129, 1, 63, 65, 0], 520, 1032),
    ([4] * 100, 512, 264),
    ([2049], 1024, 512),
    ([0, 0, 0], 72, 40),
    ([1, 2, 3, 15, 16, 17, 47, 48, 49, 63, 64, 65, 79, 80, 81], 264, 392),       # every kind of last step
])
def test_products(counts, H, N, f32, accumulate):
    check_products(counts, H, N, f32, accumulate, seed=H, spare=3, first=2)


@pytest.mark.parametrize("each", [1, 40, 300])
def test_products_of_the_most_experts(each):
    check_products([each + (e % 5 == 0) for e in range(1024)], 48, 24, seed=each)


def test_an_experts_nan_rows_stay_in_it():
    """The last step of a sum reaches into the next expert's rows, which are cleared."""
    counts, H, N = [70, 50, 40], 136, 72
    o, rows = offsets_of(counts), 160
    g, x = normal((rows, N), 1), normal((rows, H), 2)
    clean, gw = (torch.empty((3, N, H), dtype=torch.float32, device="cuda") for _ in range(2))
    moe.moe_expert_matmul_backward(g, x, None, o, grad_weights=clean)
    g[70:120], x[70:120] = math.nan, math.inf
    moe.moe_expert_matmul_backward(g, x, None, o, grad_weights=gw)
    assert torch.equal(gw[0], clean[0]) and torch.equal(gw[2], clean[2])
    assert bool(torch.isnan(gw[1]).all())


def test_weights_of_the_next_expert_stay_out():
    """The contraction over N ends inside a step: the next expert's weights are not reached."""
    counts, H, N = [40, 30], 64, 72
    o = offsets_of(counts)
    g, w = normal((70, N), 1), normal((2, N, H), 2)
    a, b = (torch.empty((70, H), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    moe.moe_expert_matmul_backward(g, None, w, o, grad_x=a)
    w[1] = math.nan
    moe.moe_expert_matmul_backward(g, None, w, o, grad_x=b)
    assert torch.equal(a[:40], b[:40]) and bool(torch.isnan(b[40:].float()).all())


def test_no_rows():
    g, x, w = normal((0, 16), 1), normal((0, 24), 1), normal((3, 16, 24), 2)
    o = torch.zeros(4, dtype=torch.int32, device="cuda")
    gw = torch.ones((3, 16, 24), dtype=torch.float32, device="cuda")
    moe.moe_expert_matmul_backward(g, x, w, o, grad_x=x, grad_weights=gw, accumulate=True)
    assert bool((gw == 1).all())
    moe.moe_expert_matmul_backward(g, x, w, o, grad_x=x, grad_weights=gw)
    assert bool((gw == 0).all())


def test_one_gradient_alone():
    counts, H, N = [40, 0, 300], 200, 136
    o, rows = offsets_of(counts), 340
    g, x, w = normal((rows, N), 1), normal((rows, H), 2), normal((3, N, H), 3)
    gx, gx2 = torch.empty_like(x), torch.empty_like(x)
    gw, gw2 = torch.empty_like(w), torch.empty_like(w)
    moe.moe_expert_matmul_backward(g, x, w, o, grad_x=gx, grad_weights=gw)
    moe.moe_expert_matmul_backward(g, None, w, o, grad_x=gx2)
    moe.moe_expert_matmul_backward(g, x, None, o, grad_weights=gw2)
    assert torch.equal(gx, gx2) and torch.equal(gw, gw2)


def test_gradients_past_32_bit_offsets():
    """More than 2^32 bytes of weights and of their gradient."""
    E, N, H = 40, 4096, 14336
    counts = [0] * E
    counts[0], counts[E - 1] = 3, 70
    o, rows = offsets_of(counts), 73
    g, x, w = normal((rows, N), 1), normal((rows, H), 2), normal((E, N, H), 3, H ** -0.5)
    gx, gw = torch.empty_like(x), torch.empty_like(w)
    moe.moe_expert_matmul_backward(g, x, w, o, grad_x=gx, grad_weights=gw)
    ge, xe, we = g[3:].double(), x[3:].double(), w[E - 1].double()
    y, s = ge @ we, ge.abs() @ we.abs()
    assert bool(((gx[3:].double() - y).abs() <= 1.01 * (N / 16 + 2) * 2.0 ** -23 * s + BF16 * y.abs()).all())
    y, s = ge.t() @ xe, ge.t().abs() @ xe.abs()
    assert bool(((gw[E - 1].double() - y).abs() <= 8 * 2.0 ** -23 * s + BF16 * y.abs()).all())
    assert torch.count_nonzero(gw[1:E - 1]) == 0


def slopes(z, act):
    """a'(z) in 64 bits and the magnitude of its terms."""
    if act == "none":
        return torch.ones_like(z), torch.ones_like(z)
    if act == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s)), 1 + z.abs()
    k, c = 2 * math.sqrt(2 / math.pi), 0.044715
    s = torch.sigmoid(k * (z + c * z ** 3))
    return s + z * s * (1 - s) * k * (1 + 3 * c * z * z), 1 + z.abs() * (1 + z * z)


def check_activation(counts, N, act, bias=True, seed=0, spare=0, first=0, alias=False):
    E, rows = len(counts), first + int(sum(counts)) + spare
    o = offsets_of(counts, first)
    C = N // 2 if act == "swiglu" else N
    z, dy = normal((rows, N), seed, 2.0), normal((rows, C), seed + 1)
    kept = z.clone()
    gz = z if alias else torch.full((rows, N), -77.0, dtype=torch.bfloat16, device="cuda")
    gb = torch.full((E, N), -77.0, device="cuda") if bias else None
    ws = torch.empty(moe.moe_expert_activation_backward_workspace_bytes(rows, N, E), dtype=torch.uint8, device="cuda")
    ws.fill_(0xAB)
    moe.moe_expert_activation_backward(z, dy, o, gz, act, grad_bias=gb, workspace=ws if bias else None)
    z64, g = kept.double(), dy.double()
    if act == "swiglu":
        a, u = z64[:, :C], z64[:, C:]
        d, m = slopes(a, "silu")
        s = torch.sigmoid(a)
        want, size = torch.cat([g * u * d, g * a * s], 1), torch.cat([(g * u).abs() * m, (g * a).abs()], 1)
    else:
        d, m = slopes(z64, act)
        want, size = g * d, g.abs() * m
    off = 2.0 ** -17 * size
    owned = torch.zeros(rows, dtype=torch.bool, device="cuda")
    owned[first:rows - spare] = True
    bad = (gz.double() - want).abs() > 1.01 * off + BF16 * want.abs()
    assert not bool(bad[owned].any())
    assert torch.equal(gz[~owned], kept[~owned] if alias else torch.full_like(gz[~owned], -77.0))
    if bias:
        sums, room = torch.zeros((E, N), dtype=torch.float64, device="cuda"), torch.zeros((E, N), dtype=torch.float64, device="cuda")
        for e, a, b in ranges(o, rows):
            sums[e] = want[a:b].sum(0)
            room[e] = (off[a:b].sum(0) + (b - a) * F32 * want[a:b].abs().sum(0)) * 1.01
        assert bool(((gb.double() - sums).abs() <= room).all())


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("N", [16, 64, 528, 4112])
@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 17, 1], [127, 128, 129, 0, 700], [4] * 256])
def test_activation(counts, N, act, bias):
    check_activation(counts, N, act, bias, seed=N, spare=3, first=2)


@pytest.mark.parametrize("act", ["silu", "swiglu"])
def test_activation_in_place(act):
    check_activation([100, 0, 200], 272, act, seed=1, spare=2, alias=True)


@pytest.mark.parametrize("N", [8, 24, 1000])
def test_activation_odd_rows_of_eight(N):
    check_activation([33, 200, 0, 5], N, "gelu", seed=N)


def test_activation_of_the_most_experts():
    check_activation([3 + (e % 7 == 0) for e in range(1024)], 48, "swiglu", seed=3)


def test_activation_without_rows():
    gb = torch.full((3, 32), 5.0, device="cuda")
    ws = torch.empty(moe.moe_expert_activation_backward_workspace_bytes(0, 32, 3), dtype=torch.uint8, device="cuda")
    e = torch.empty((0, 32), dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_activation_backward(e, e, torch.zeros(4, dtype=torch.int32, device="cuda"), e, "silu", grad_bias=gb,
                                       workspace=ws)
    assert bool((gb == 0).all())


def test_bias_gradient_alone():
    o = offsets_of([200, 0, 313])
    dy = normal((513, 264), 1)
    gb, gb2, gz = torch.empty((3, 264), device="cuda"), torch.empty((3, 264), device="cuda"), torch.empty_like(dy)
    ws = torch.empty(moe.moe_expert_activation_backward_workspace_bytes(513, 264, 3), dtype=torch.uint8, device="cuda")
    moe.moe_expert_activation_backward(None, dy, o, None, "none", grad_bias=gb, workspace=ws)
    moe.moe_expert_activation_backward(dy, dy, o, gz, "none", grad_bias=gb2, workspace=ws)
    assert torch.equal(gb, gb2) and torch.equal(gz, dy)


def test_activation_gradient_by_differences():
    """(a(z + h) - a(z - h)) / 2h through moe_expert_matmul itself: one row a value,
    weights 1, z = x in bf16; h = 1/8 keeps bf16's rounding (2^-8 |a| / h) and the
    third derivative's share (h^2 / 6, it is below 1) small."""
    v = torch.arange(-48, 49, device="cuda").float() / 8
    rows, h = v.numel(), 0.125
    w = torch.zeros((1, 8, 8), dtype=torch.bfloat16, device="cuda")
    w[0, 0, 0] = 1
    o = offsets_of([rows])

    def value(x, act):
        xb = torch.zeros((rows, 8), dtype=torch.bfloat16, device="cuda")
        xb[:, 0] = x
        out = torch.empty((rows, 8), dtype=torch.bfloat16, device="cuda")
        moe.moe_expert_matmul(xb, w, o, out, activation=act)
        return out[:, 0].double()
    for act in ("silu", "gelu"):
        up, down = value(v + h, act), value(v - h, act)
        z = torch.zeros((rows, 8), dtype=torch.bfloat16, device="cuda")
        z[:, 0] = v
        gz = torch.empty_like(z)
        moe.moe_expert_activation_backward(z, torch.ones_like(z), o, gz, act)
        room = BF16 * (up.abs() + down.abs()) / (2 * h) + h * h / 6 + BF16 * 1.2
        assert bool((((up - down) / (2 * h) - gz[:, 0].double()).abs() <= room).all()), act


def test_graph_replay_with_new_rows():
    counts, H, N = [100, 0, 60, 140], 264, 272
    o, rows = offsets_of(counts), 300
    z, dy, x, w = normal((rows, N), 1), normal((rows, N // 2), 2), normal((rows, H), 3), normal((4, N, H), 4, 0.06)
    ws = torch.empty(moe.moe_expert_activation_backward_workspace_bytes(rows, N, 4), dtype=torch.uint8, device="cuda")

    def buffers():
        return (torch.zeros_like(z), torch.zeros((4, N), device="cuda"), torch.zeros_like(x), torch.zeros_like(w))

    def go(b):
        moe.moe_expert_activation_backward(z, dy, o, b[0], "swiglu", grad_bias=b[1], workspace=ws)
        moe.moe_expert_matmul_backward(b[0], x, w, o, grad_x=b[2], grad_weights=b[3])
    a, c = buffers(), buffers()
    go(a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(c)
    for n in range(3):
        for t in c:
            t.zero_()
        if n == 2:
            z.copy_(normal((rows, N), 9))
            o.copy_(torch.tensor([0, 0, 290, 290, 300], dtype=torch.int32))
            for t in a[1:]:
                t.zero_()
            go(a)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(a, c))
