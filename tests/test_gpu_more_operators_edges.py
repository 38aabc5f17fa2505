"""The grouped router and the bf16 expert operators where their memory is unusual:
tensors that start on 16 bytes and no more, element offsets past 32 bits, calls on
two streams at once, and ids listed twice."""
import pytest
import torch

import combine_moe_layout_05_gb300 as moe

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_moe_layout_05_gb300 import build
    build.build()
    moe.load()


def normal(shape, seed, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def shifted(t):
    """The same values 16 bytes into a buffer."""
    k = 16 // t.element_size()
    flat = torch.empty(t.numel() + k, dtype=t.dtype, device="cuda")
    flat[k:].copy_(t.reshape(-1))
    return flat[k:].view(t.shape)


@pytest.mark.parametrize("counts", [[3, 0, 5], [40, 90], [300, 0, 260]])
@pytest.mark.parametrize("f32", [False, True])
def test_tensors_that_start_on_16_bytes(counts, f32):
    E, H, N, rows = len(counts), 264, 272, sum(counts)
    o = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
    x, w, b = normal((rows, H), 1), normal((E, N, H), 2, 0.06), normal((E, N), 3, dtype=torch.float32)
    r, dy = normal((rows, N // 2), 4), normal((rows, N // 2), 5)

    def run(at):
        x1, w1, r1, dy1 = at(x), at(w), at(r), at(dy)
        out, pre = at(torch.zeros_like(r)), at(torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda"))
        moe.moe_expert_matmul(x1, w1, o, out, bias=b, activation="swiglu", residual=r1, pre=pre)
        gz, gb = at(torch.zeros_like(pre)), torch.zeros_like(b)
        ws = torch.empty(moe.moe_expert_activation_backward_workspace_bytes(rows, N, E), dtype=torch.uint8, device="cuda")
        moe.moe_expert_activation_backward(pre, dy1, o, gz, "swiglu", grad_bias=gb, workspace=ws)
        gx, gw = at(torch.zeros_like(x)), at(torch.zeros((E, N, H), dtype=torch.float32 if f32 else torch.bfloat16, device="cuda"))
        moe.moe_expert_matmul_backward(gz, x1, w1, o, gx, gw, accumulate=f32)
        return out, pre, gz, gb, gx, gw
    for a, c in zip(run(lambda t: t.clone()), run(shifted)):
        assert torch.equal(a, c)


def test_two_streams_at_once():
    counts, H, N = [200, 0, 700, 60], 1032, 1040
    o = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
    w = normal((4, N, H), 2, 0.03)
    xs = [normal((960, H), s) for s in (1, 2)]
    logits = [normal((4000, 256), s, dtype=torch.float32) for s in (3, 4)]

    def run(x, lo):
        out = torch.empty((960, N // 2), dtype=torch.bfloat16, device="cuda")
        gx, gw = torch.empty_like(x), torch.empty_like(w)
        r = moe.RouteBuffers(4000, 8, 256)
        ws = torch.empty(moe.moe_route_grouped_workspace_bytes(4000, 256), dtype=torch.uint8, device="cuda")
        for _ in range(5):
            moe.moe_expert_matmul(x, w, o, out, activation="swiglu")
            moe.moe_expert_matmul_backward(torch.ones((960, N), dtype=torch.bfloat16, device="cuda"), x, w, o, gx, gw)
            moe.moe_route_grouped(lo, None, r.topk_ids, r.topk_weights, r.expert_counts, r.routed_tokens, r.loss,
                                  groups=8, top_groups=4, workspace=ws)
        return out, gx, gw, r.topk_ids, r.topk_weights, r.expert_counts, r.loss
    want = [run(x, lo) for x, lo in zip(xs, logits)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in xs], []
    for s, x, lo in zip(streams, xs, logits):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(run(x, lo))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_activation_offsets_past_32_bits():
    rows, N = 1_060_000, 2048                            # 2.2e9 elements
    z, dy = normal((rows, N), 1), normal((rows, N), 2)
    o = torch.tensor([0, 500, rows - 300, rows], dtype=torch.int32, device="cuda")
    gz, gb = torch.empty_like(z), torch.empty((3, N), device="cuda")
    ws = torch.empty(moe.moe_expert_activation_backward_workspace_bytes(rows, N, 3), dtype=torch.uint8, device="cuda")
    moe.moe_expert_activation_backward(z, dy, o, gz, "silu", grad_bias=gb, workspace=ws)
    for a, b, e in ((0, 500, 0), (rows - 300, rows, 2)):
        x, g = z[a:b].double(), dy[a:b].double()
        s = torch.sigmoid(x)
        want, size = g * s * (1 + x * (1 - s)), g.abs() * (1 + x.abs())
        off = 2.0 ** -17 * size
        assert bool(((gz[a:b].double() - want).abs() <= 1.01 * off + BF16 * want.abs()).all())
        room = 1.01 * (off.sum(0) + (b - a) * 2.0 ** -24 * want.abs().sum(0))
        assert bool(((gb[e].double() - want.sum(0)).abs() <= room).all())


def test_router_offsets_past_32_bits():
    T, E, K = 8_500_000, 256, 2                          # 2.2e9 logits
    x = normal((T, E), 1)
    r = moe.RouteBuffers(T, K, E)
    ws = torch.empty(moe.moe_route_grouped_workspace_bytes(T, E), dtype=torch.uint8, device="cuda")
    moe.moe_route_grouped(x, None, r.topk_ids, r.topk_weights, r.expert_counts, r.routed_tokens, r.loss, workspace=ws)
    grad = torch.empty_like(x)
    dw = torch.ones((T, K), device="cuda")
    dw[:, 1] = 0
    moe.moe_route_grouped_backward(x, r.topk_ids, r.expert_counts, r.routed_tokens, dw, None, grad)
    assert r.expert_counts.sum().item() == T * K and r.routed_tokens.item() == T
    for a in (0, T - 500):
        y = x[a:a + 500].double()
        ids = torch.sort(y, dim=1, descending=True, stable=True)[1][:, :K]
        assert torch.equal(r.topk_ids[a:a + 500].long(), ids)
        s = torch.sigmoid(y).gather(1, ids)
        w = s / s.sum(1, keepdim=True)
        assert torch.allclose(r.topk_weights[a:a + 500].double(), w, rtol=1e-5, atol=0)
        d = torch.stack([w[:, 0] * w[:, 1] * torch.sigmoid(-y.gather(1, ids)[:, 0]),
                         -w[:, 0] * w[:, 1] * torch.sigmoid(-y.gather(1, ids)[:, 1])], 1)
        want = torch.zeros_like(y).scatter_(1, ids, d)
        assert bool(((grad[a:a + 500].double() - want).abs() <= 1e-5 + 1.01 * BF16 * want.abs()).all())


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_ids_listed_twice_add_up(scoring):
    """Not what the router gives, but what the gradient's formula says of it (without renormalising)."""
    x = normal((50, 32), 1, dtype=torch.float32)
    ids = torch.tensor([[3, 3, 7, 3]], dtype=torch.int32, device="cuda").repeat(50, 1)
    dw = normal((50, 4), 2, dtype=torch.float32)
    counts, n = torch.zeros(32, dtype=torch.int32, device="cuda"), torch.full((1,), 50, dtype=torch.int32, device="cuda")
    grad = torch.empty_like(x)
    moe.moe_route_grouped_backward(x, ids, counts, n, dw, None, grad, scoring=scoring, renormalize=False)
    y = x.double().requires_grad_()
    s = torch.sigmoid(y) if scoring == "sigmoid" else torch.softmax(y, 1)
    want = torch.autograd.grad((s.gather(1, ids.long()) * dw.double()).sum(), y)[0]
    # terms of size |dw|, a few of them: 2 (8 + 64) and some 2^-24 of each
    assert bool(((grad.double() - want).abs() <= 200 * 2.0 ** -24 * dw.abs().sum(1, keepdim=True)).all())
