"""moe_expert_matmul_int8 against the integer sums.

While no partial sum can reach 2^24 the kernel's sum is the integer, and the
result is bf16(fp32(fp32(s * x_scale) * w_scale)): compared bit for bit.  Past
2^24 each of the sum's steps may round or truncate to 24 bits: its error is
held to 2^-23 of the magnitudes' sum for every 16 terms, and the output's
rounding adds 2^-8 of the result."""
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


def codes(shape, seed, lo=-128, hi=128):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int8)


def offsets_of(counts):
    o = np.zeros(len(counts) + 1, np.int32)
    o[1:] = np.cumsum(counts)
    return o


def sums(x, w, o):
    """[rows, N] integer sums in float64 (exact), NaN where no expert owns the row."""
    s = torch.full((x.shape[0], w.shape[1]), float("nan"), dtype=torch.float64, device="cuda")
    for e in range(w.shape[0]):
        a, b = int(o[e]), int(o[e + 1])
        if b > a:
            s[a:b] = x[a:b].double() @ w[e].double().t()
    return s


def scales(rows, E, N, seed):
    g = torch.Generator(device="cuda").manual_seed(seed + 1000)
    return (torch.rand(rows, generator=g, device="cuda") * 0.1 + 0.001,
            torch.rand((E, N), generator=g, device="cuda") * 0.02 + 1e-4)


def run(x, xs, w, ws, o):
    out = torch.full((x.shape[0], w.shape[1]), -77.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_expert_matmul_int8(x, xs, w, ws, torch.from_numpy(np.asarray(o, np.int32)).cuda(), out)
    return out


def check(counts, H, N, seed=0, spare=0, lim=None):
    E, rows = len(counts), int(sum(counts)) + spare
    o = offsets_of(counts)
    # magnitudes that keep H products' sum below 2^24
    lim = lim or max(1, min(127, int((2 ** 24 / H) ** 0.5)))
    x, w = codes((rows, H), seed, -lim, lim + 1), codes((E, N, H), seed + 1, -lim, lim + 1)
    xs, ws = scales(rows, E, N, seed)
    out = run(x, xs, w, ws, o)
    s = sums(x, w, o)
    owned = ~torch.isnan(s[:, 0])
    per_row = torch.zeros((rows, N), device="cuda")
    for e in range(E):
        per_row[int(o[e]):int(o[e + 1])] = ws[e]
    want = (s.float() * xs[:, None] * per_row).to(torch.bfloat16)
    assert torch.equal(out[owned], want[owned])
    assert bool((out[~owned] == -77.0).all())            # rows of no expert are left alone


@pytest.mark.parametrize("H", [16, 64, 128, 144, 1040])
@pytest.mark.parametrize("N", [1, 7, 64, 129, 250, 256])
@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 17, 1], [16, 33, 250, 0]])
def test_small(counts, H, N):
    check(counts, H, N, seed=H + N)


@pytest.mark.parametrize("counts,H,N", [
    ([1] * 8 + [0] * 24, 7168, 256),                     # one token's experts
    ([4] * 256, 1024, 264),                              # a decode batch
    ([1000, 0, 3, 515, 64, 127, 128, 129], 512, 520),    # rows around every tile edge
    ([0, 0, 0], 64, 64),                                 # nobody
    ([4097], 256, 1000),                                 # one expert: the plain product
    ([0] * 1023 + [5], 32, 16),                          # the most experts
    ([31, 32, 33, 63, 64, 65, 255, 256, 257, 511, 513], 192, 384),
])
def test_groups(counts, H, N):
    check(counts, H, N, seed=len(counts), spare=5)


@pytest.mark.parametrize("H,N", [(1040, 2600), (144, 2568), (64, 3001), (4112, 2560)])
@pytest.mark.parametrize("counts", [[1500, 700], [0, 2049], [129, 0, 2500, 513, 96, 1]])
def test_many_rows(counts, H, N):
    """Full and ragged tiles of many rows, channels that end inside a tile."""
    check(counts, H, N, seed=H + N, spare=3)


@pytest.mark.parametrize("H,N", [(2560, 2600), (2576, 257), (2752, 2561), (3984, 1), (2816, 520)])
@pytest.mark.parametrize("counts", [[385], [900, 33, 410], [0, 255, 2049, 1, 256, 257, 17]])
def test_many_rows_and_a_long_contraction(counts, H, N):
    check(counts, H, N, seed=H + N, spare=2)


@pytest.mark.parametrize("H,N", [(272, 2600), (1040, 2049), (64, 3000)])
@pytest.mark.parametrize("counts", [[33, 64, 65, 96, 97, 127, 128, 129, 160], [20, 0, 250, 1, 40, 48], [17] * 40])
def test_tens_of_rows(counts, H, N):
    check(counts, H, N, seed=H + N, spare=1)


@pytest.mark.parametrize("each", [3, 40, 520])
def test_the_most_experts_of_few_and_many_rows(each):
    """The experts' table takes the most shared memory, in each form."""
    check([each + (e % 5 == 0) for e in range(1024)], 48, 24, seed=each)


@pytest.mark.parametrize("rows", [1, 15, 16, 17, 31, 32])
@pytest.mark.parametrize("H,N", [(528, 100), (1008, 129), (2064, 40), (7168, 130), (1040, 1000)])
def test_contraction_split_over_blocks(rows, H, N):
    """A few tiles: their contraction is shared out, in uneven parts at these H."""
    check([rows], H, N, seed=rows + H)
    check([0, rows, 3, 0, 1], H, N, seed=rows + N, spare=2)


def test_full_codes_below_the_exact_bound():
    """All 256 codes, -128 among them: 1008 * 128 * 128 < 2^24."""
    o = offsets_of([40, 0, 90])
    x, w = codes((130, 1008), 3), codes((3, 200, 1008), 4)
    assert int(x.min()) == -128 == int(w.min())
    xs, ws = scales(130, 3, 200, 5)
    out = run(x, xs, w, ws, o)
    per_row = torch.cat([ws[0].expand(40, -1), ws[2].expand(90, -1)])
    assert torch.equal(out, (sums(x, w, o).float() * xs[:, None] * per_row).to(torch.bfloat16))


@pytest.mark.parametrize("kind", ["random", "all_127", "up_then_down"])
def test_sums_past_24_bits(kind):
    rows, H, N = 70, 7168, 136
    x, w = codes((rows, H), 1, -127, 128), codes((1, N, H), 2, -127, 128)
    if kind != "random":
        x.fill_(127)
        w.fill_(127)
    if kind == "up_then_down":
        w[..., H // 2:] = -126
    xs, ws = torch.ones(rows, device="cuda"), torch.ones(1, N, device="cuda")
    out = run(x, xs, w, ws, [0, rows]).double()
    s = x.double() @ w[0].double().t()
    big = x.double().abs() @ w[0].double().abs().t()
    tol = (H / 16) * 2.0 ** -23 * big + 2.0 ** -8 * s.abs()
    assert bool(((out - s).abs() <= tol).all())


def test_scales_pass_through():
    x, w = codes((20, 64), 1), codes((2, 24, 64), 2)
    xs, ws = scales(20, 2, 24, 3)
    xs[4], xs[5] = float("nan"), 0.0
    ws[1, 3] = float("inf")
    out = run(x, xs, w, ws, [0, 10, 20]).float()
    assert bool(torch.isnan(out[4]).all()) and torch.count_nonzero(out[5]) == 0
    assert not bool(torch.isfinite(out[10:, 3]).any()) and bool(torch.isfinite(out[10:, 4]).all())


def test_offsets_outside_the_rows_are_cut():
    x, w = codes((10, 32), 1), codes((3, 16, 32), 2)
    xs, ws = scales(10, 3, 16, 3)
    good = run(x, xs, w, ws, [0, 4, 4, 10])
    assert torch.equal(run(x, xs, w, ws, [-3, 4, 4, 1000]), good)


def test_long_weights_pass_32_bit_offsets():
    """More than 2^31 weight bytes: the last experts' addresses need 64 bits."""
    E, N, H = 40, 4096, 14336
    counts = [0] * E
    counts[0], counts[E - 1] = 3, 5
    check(counts, H, N, seed=9)


def test_longest_contraction():
    check([5, 0, 40], 65536, 40, seed=11)
    check([20] * 30, 65536, 24, seed=12)


def test_outputs_past_32_bit_offsets():
    """More than 2^31 outputs: the last rows' addresses need 64 bits."""
    rows, H, N = 1_060_000, 16, 2048
    x, w = codes((rows, H), 1), codes((2, N, H), 2)
    xs, ws = scales(rows, 2, N, 3)
    o = [0, 1000, rows]
    out = run(x, xs, w, ws, o)
    for r in (slice(0, 300), slice(900, 1100), slice(rows - 3000, rows)):
        at = torch.arange(rows, device="cuda")[r]
        e = (at >= 1000).long()
        s = torch.einsum("rh,rnh->rn", x[r].double(), w[e].double())
        assert torch.equal(out[r], (s.float() * xs[r, None] * ws[e]).to(torch.bfloat16))


def test_error_word_is_cleared():
    x, w = codes((20, 64), 1), codes((2, 24, 64), 2)
    xs, ws = scales(20, 2, 24, 3)
    err = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    out = torch.empty((20, 24), dtype=torch.bfloat16, device="cuda")
    o = torch.tensor([0, 10, 20], dtype=torch.int32, device="cuda")
    moe.moe_expert_matmul_int8(x, xs, w, ws, o, out, dev_error=err)
    assert err.item() == 0


def test_side_stream_graph_and_repeat():
    x, w = codes((300, 512), 1, -60, 61), codes((4, 512, 512), 2, -60, 61)
    xs, ws = scales(300, 4, 512, 3)
    o = torch.tensor([0, 100, 101, 290, 300], dtype=torch.int32, device="cuda")
    a = run(x, xs, w, ws, o.cpu().numpy())
    b = torch.zeros_like(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.moe_expert_matmul_int8(x, xs, w, ws, o, b)
    side.synchronize()
    assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_expert_matmul_int8(x, xs, w, ws, o, b)
    for n in range(3):
        b.zero_()
        if n == 2:                                       # a replay sees new rows and new ranges
            x.copy_(codes((300, 512), 7, -60, 61))
            o.copy_(torch.tensor([0, 0, 290, 290, 300], dtype=torch.int32))
            a = run(x, xs, w, ws, o.cpu().numpy())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, b)
