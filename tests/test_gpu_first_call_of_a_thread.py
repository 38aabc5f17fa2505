"""The routers' and the experts' calls as the first CUDA work of a thread, as autograd's
own thread makes them where a gradient comes straight from the caller: same bits as here."""
import threading

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


def in_a_thread(call):
    failed = []

    def go():
        try:
            call()
        except Exception as e:
            failed.append(e)
    t = threading.Thread(target=go)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not failed, failed


def normal(shape, seed):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("what", ["forward", "backward", "int8"])
@pytest.mark.parametrize("rows", [5, 400])
def test_products(what, rows):
    o = torch.tensor([0, 3, rows], dtype=torch.int32, device="cuda")
    x, w, g = normal((rows, 128), 1), normal((2, 64, 128), 2), normal((rows, 64), 3)
    x8, w8 = (t.mul(20).clamp(-127, 127).to(torch.int8) for t in (x, w))
    ones, scales = torch.ones(rows, device="cuda"), torch.ones((2, 64), device="cuda")
    outs = [[torch.empty_like(t) for t in (g, x, w)] for _ in range(2)]

    def call(out):
        if what == "forward":
            moe.moe_expert_matmul(x, w, o, out[0])
        elif what == "backward":
            moe.moe_expert_matmul_backward(g, x, w, o, out[1], out[2])
        else:
            moe.moe_expert_matmul_int8(x8, ones, w8, scales, o, out[0])
    for out in outs:
        for t in out:
            t.zero_()
    torch.cuda.synchronize()
    in_a_thread(lambda: call(outs[1]))
    call(outs[0])
    assert all(torch.equal(a, b) for a, b in zip(*outs)) and any(bool(t.any()) for t in outs[0])


def test_gradient_given_by_the_caller():
    """The backward pass in a thread that has done nothing before."""
    from combine_moe_layout_05_gb300.layer import expert_linear
    o = torch.tensor([0, 3, 9], dtype=torch.int32, device="cuda")
    x, w, g = normal((9, 128), 1).requires_grad_(), normal((2, 64, 128), 2).requires_grad_(), normal((9, 64), 3)
    out = expert_linear(x, w, o)
    out.backward(g)
    gx, gw = torch.empty_like(x), torch.empty_like(w)
    moe.moe_expert_matmul_backward(g, x.detach(), w.detach(), o, gx, gw)
    assert torch.equal(x.grad, gx) and torch.equal(w.grad, gw)


@pytest.mark.parametrize("what", ["route", "route_backward", "activation"])
@pytest.mark.parametrize("rows", [5, 4000])
def test_other_calls(what, rows):
    x, bias = normal((rows, 64), 1).float(), torch.linspace(0, 0.1, 64, device="cuda")
    o = torch.tensor([0, 3, rows], dtype=torch.int32, device="cuda")
    pre, dy, dw = normal((rows, 64), 2), normal((rows, 64), 3), torch.ones((rows, 4), device="cuda")
    route = moe.RouteBuffers(rows, 4, 64).run(x)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(2):
        r = moe.RouteBuffers(rows, 4, 64)
        outs.append(dict(route=[r.topk_ids, r.topk_weights, r.expert_counts, r.routed_tokens, r.loss],
                         route_backward=[torch.zeros_like(x)],
                         activation=[torch.zeros_like(pre), torch.zeros((2, 64), device="cuda")])[what])
        for t in outs[-1]:
            t.zero_()

    def call(out):
        if what == "route":
            moe.moe_route_grouped(x, bias, *out, groups=8, top_groups=4, workspace=ws)
        elif what == "route_backward":
            moe.moe_route_grouped_backward(x, route.topk_ids, route.expert_counts, route.routed_tokens, dw, route.loss, *out)
        else:
            moe.moe_expert_activation_backward(pre, dy, o, out[0], "silu", grad_bias=out[1], workspace=ws)
    torch.cuda.synchronize()
    in_a_thread(lambda: call(outs[1]))
    call(outs[0])
    assert all(torch.equal(a, b) for a, b in zip(*outs)) and any(bool(t.any()) for t in outs[0])
