"""moe_route_grouped, its gradient, moe_expert_matmul, its gradients and
moe_expert_activation_backward refuse bad arguments on the host, before any CUDA
call (so these run without a GPU), and the binding refuses wrong types, sizes,
layouts and names."""
import ctypes

import pytest
import torch

import combine_moe_layout_05_gb300 as moe
from combine_moe_layout_05_gb300 import build as moe_build

FAKE = 0x10000            # never dereferenced: the checks come first
P = ctypes.c_void_p
INVALID, ALIGNMENT, WORKSPACE = 1, 2, 4
MOST = 2 ** 31 - 65536
bf16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.load()


def test_route_grouped(lib):
    def f(logits=FAKE, bf16=0, T=4, E=16, K=2, scoring=1, bias=FAKE, groups=4, top=2, group_top=2, renorm=1, mask=None,
          ids=FAKE, w=FAKE, cnt=FAKE, n=FAKE, loss=FAKE, ws=FAKE, wsb=1 << 20):
        return lib.moe_route_grouped(P(logits), bf16, T, E, K, scoring, P(bias), groups, top, group_top, renorm, 1.0, 1.0,
                                     P(mask), P(ids), P(w), P(cnt), P(n), P(loss), P(ws), wsb, None)
    for kw in (dict(T=-1), dict(E=0), dict(E=1025), dict(K=0), dict(K=17), dict(K=33, E=64), dict(bf16=2), dict(renorm=-1),
               dict(scoring=2), dict(scoring=-1), dict(groups=0), dict(groups=3), dict(groups=64, E=64, top=2),
               dict(top=0), dict(top=5), dict(group_top=0), dict(group_top=3), dict(K=9), dict(K=5, top=1),
               dict(logits=0), dict(ids=0), dict(w=0), dict(cnt=0), dict(n=0), dict(loss=0), dict(T=2 ** 28, K=8),
               dict(T=MOST + 1, E=1, K=1, groups=1, top=1)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(logits=FAKE + 2), dict(bf16=1, logits=FAKE + 1), dict(ids=FAKE + 2), dict(w=FAKE + 1), dict(bias=FAKE + 2),
               dict(cnt=FAKE + 2), dict(n=FAKE + 2), dict(loss=FAKE + 2), dict(ws=FAKE + 8)):
        assert f(**kw) == ALIGNMENT, kw
    need = moe.moe_route_grouped_workspace_bytes(4, 16)
    assert need > 0 and f(wsb=need - 1) == WORKSPACE and f(ws=0) == WORKSPACE
    assert moe.moe_route_grouped_workspace_bytes(4, 1025) == 0 == moe.moe_route_grouped_workspace_bytes(-1, 16)
    assert moe.moe_route_grouped_workspace_bytes(MOST + 1, 16) == 0 < moe.moe_route_grouped_workspace_bytes(MOST, 16)


def test_route_grouped_backward(lib):
    def f(logits=FAKE, bf16=0, T=4, E=16, K=2, scoring=0, renorm=1, ids=FAKE, cnt=FAKE, n=FAKE, dw=FAKE, dl=FAKE, grad=FAKE):
        return lib.moe_route_grouped_backward(P(logits), bf16, T, E, K, scoring, renorm, 1.0, 1.0, P(ids), P(cnt), P(n),
                                              P(dw), P(dl), P(grad), None)
    for kw in (dict(T=-1), dict(E=0), dict(E=1025), dict(K=0), dict(K=17), dict(bf16=3), dict(renorm=2), dict(scoring=2),
               dict(logits=0), dict(ids=0), dict(cnt=0), dict(n=0), dict(grad=0)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(logits=FAKE + 2), dict(grad=FAKE + 2), dict(ids=FAKE + 2), dict(dw=FAKE + 2),
               dict(dl=FAKE + 1), dict(bf16=1, grad=FAKE + 1)):
        assert f(**kw) == ALIGNMENT, kw
    assert f(T=0, logits=0, grad=0) == 0                 # T == 0: no-op


BAD_SIZES = (dict(rows=-1), dict(H=0), dict(H=12), dict(H=65544), dict(N=0), dict(E=0), dict(E=1025),
             dict(E=1024, N=2 ** 21), dict(rows=MOST + 1), dict(rows=2 ** 31 - 1))


def test_expert_matmul(lib):
    def f(x=FAKE, w=FAKE, b=FAKE, off=FAKE, rows=4, H=32, N=8, E=2, act=0, res=FAKE, pre=FAKE, out=FAKE, err=0):
        return lib.moe_expert_matmul(P(x), P(w), P(b), P(off), rows, H, N, E, act, P(res), P(pre), P(out), P(err), None)
    for kw in BAD_SIZES + (dict(act=-1), dict(act=4), dict(act=3, N=7), dict(x=0), dict(w=0), dict(off=0), dict(out=0)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(x=FAKE + 8), dict(w=FAKE + 8), dict(out=FAKE + 8), dict(res=FAKE + 8), dict(pre=FAKE + 8),
               dict(b=FAKE + 2), dict(off=FAKE + 2), dict(err=FAKE + 2), dict(rows=MOST, x=FAKE + 2),
               dict(N=MOST, E=1, x=FAKE + 2)):
        assert f(**kw) == ALIGNMENT, kw
    assert f(rows=0, x=0, out=0) == 0


def test_expert_matmul_backward(lib):
    def f(g=FAKE, x=FAKE, w=FAKE, off=FAKE, rows=4, H=32, N=8, E=2, gx=FAKE, gw=FAKE, f32=0, acc=0, err=0):
        return lib.moe_expert_matmul_backward(P(g), P(x), P(w), P(off), rows, H, N, E, P(gx), P(gw), f32, acc, P(err), None)
    for kw in BAD_SIZES + (dict(N=12), dict(f32=2), dict(acc=2), dict(acc=1), dict(g=0), dict(x=0), dict(w=0), dict(off=0),
                           dict(gx=0, gw=0)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(g=FAKE + 8), dict(x=FAKE + 8), dict(w=FAKE + 8), dict(gx=FAKE + 8), dict(gw=FAKE + 8),
               dict(off=FAKE + 2), dict(err=FAKE + 2)):
        assert f(**kw) == ALIGNMENT, kw
    assert f(rows=0, g=0, x=0, gw=0) == 0 and f(rows=0, f32=1, acc=1, g=0, x=0) == 0


def test_expert_activation_backward(lib):
    def f(pre=FAKE, g=FAKE, off=FAKE, rows=4, N=16, E=2, act=1, gp=FAKE, gb=FAKE, ws=FAKE, wsb=1 << 20):
        return lib.moe_expert_activation_backward(P(pre), P(g), P(off), rows, N, E, act, P(gp), P(gb), P(ws), wsb, None)
    for kw in (dict(rows=-1), dict(N=0), dict(N=12), dict(N=8, act=3), dict(E=0), dict(E=1025), dict(act=-1), dict(act=4),
               dict(rows=MOST + 1), dict(pre=0), dict(g=0), dict(off=0), dict(gp=0, gb=0)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(pre=FAKE + 8), dict(g=FAKE + 8), dict(gp=FAKE + 8), dict(gb=FAKE + 2), dict(off=FAKE + 2),
               dict(ws=FAKE + 8)):
        assert f(**kw) == ALIGNMENT, kw
    need = moe.moe_expert_activation_backward_workspace_bytes(4, 16, 2)
    assert need > 0 and f(wsb=need - 1) == WORKSPACE and f(ws=0) == WORKSPACE
    assert f(rows=0, gb=0, g=0, pre=0) == 0
    assert moe.moe_expert_activation_backward_workspace_bytes(-1, 16, 2) == 0
    assert moe.moe_expert_activation_backward_workspace_bytes(4, 16, 1025) == 0


@pytest.mark.parametrize("rows,N,E", [(1, 8, 1), (131072, 4096, 128), (4662, 1032, 48), (5, 8, 1024), (10 ** 6, 8, 3)])
def test_activation_workspace_holds_every_split(rows, N, E):
    """Chunks of at least 32 rows, one more for each expert that has rows, and a table of the experts."""
    need = moe.moe_expert_activation_backward_workspace_bytes(rows, N, E)
    assert 4 * (E + 1) + 4 * N * (rows // 128) <= need <= 4 * (E + 1) + 512 + 4 * N * (rows // 32 + min(rows, E) + 1)


def test_binding_types_sizes_and_names(lib):
    T, E, K = 4, 16, 2
    i32 = torch.int32
    route = [torch.zeros(T, K, dtype=i32), torch.zeros(T, K), torch.zeros(E, dtype=i32), torch.zeros(1, dtype=i32),
             torch.zeros(1)]
    x = torch.zeros(T, E)
    with pytest.raises(TypeError):
        moe.moe_route_grouped(x.half(), None, *route)
    with pytest.raises(ValueError, match="scoring"):
        moe.moe_route_grouped(x, None, *route, scoring="tanh")
    with pytest.raises(ValueError):
        moe.moe_route_grouped(x, None, *route)           # host tensors
    with pytest.raises(ValueError):
        moe.moe_route_grouped(torch.zeros(E, T).t(), None, *route)
    with pytest.raises(TypeError):
        moe.moe_route_grouped_backward(x.double(), route[0], route[2], route[3], None, None, x.double())
    rows, w = torch.zeros(4, 32, dtype=bf16), torch.zeros(2, 16, 32, dtype=bf16)
    off, out = torch.zeros(3, dtype=i32), torch.zeros(4, 16, dtype=bf16)
    with pytest.raises(TypeError):
        moe.moe_expert_matmul(rows.float(), w, off, out)
    with pytest.raises(ValueError, match="activation"):
        moe.moe_expert_matmul(rows, w, off, out, activation="relu")
    with pytest.raises(ValueError):
        moe.moe_expert_matmul(rows, w, off, out)         # host tensors
    with pytest.raises(TypeError):
        moe.moe_expert_matmul_backward(out.float(), rows, w, off, rows, w)
    with pytest.raises(TypeError):
        moe.moe_expert_activation_backward(out.float(), out, off, out, "silu")
    with pytest.raises(ValueError, match="activation"):
        moe.moe_expert_activation_backward(out, out, off, out, "SiLU")


@pytest.mark.gpu
def test_binding_sizes_on_the_gpu(lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    d = dict(device="cuda")
    i32 = dict(dtype=torch.int32, **d)
    x = torch.zeros(4, 16, **d)
    route = [torch.zeros(4, 2, **i32), torch.zeros(4, 2, **d), torch.zeros(16, **i32), torch.zeros(1, **i32), torch.zeros(1, **d)]
    ws = torch.empty(moe.moe_route_grouped_workspace_bytes(4, 16), dtype=torch.uint8, **d)
    with pytest.raises(moe.MoeError):
        moe.moe_route_grouped(x, None, *route)           # no workspace
    with pytest.raises(moe.MoeError):
        moe.moe_route_grouped(x, None, *route, groups=3, workspace=ws)
    with pytest.raises(ValueError):
        moe.moe_route_grouped(x, torch.zeros(15, **d), *route, workspace=ws)
    with pytest.raises(TypeError):
        moe.moe_route_grouped(x, torch.zeros(16, dtype=bf16, **d), *route, workspace=ws)
    with pytest.raises(ValueError):
        moe.moe_route_grouped(x, None, *route, token_mask=torch.ones(3, dtype=torch.bool, **d), workspace=ws)
    with pytest.raises(ValueError):
        moe.moe_route_grouped(x, None, *route, workspace=ws.cpu())
    r, w, off = torch.zeros(4, 32, dtype=bf16, **d), torch.zeros(2, 16, 32, dtype=bf16, **d), torch.zeros(3, **i32)
    out = torch.zeros(4, 16, dtype=bf16, **d)
    for kw in (dict(out=out[:3]), dict(weights=w[:, :, :16].contiguous()), dict(expert_offsets=off[:2]),
               dict(bias=torch.zeros(2, 8, **d)), dict(residual=out[:2]), dict(pre=out[:3]), dict(activation="swiglu")):
        a = dict(x=r, weights=w, expert_offsets=off, out=out)
        a.update(kw)
        with pytest.raises(ValueError):
            moe.moe_expert_matmul(**a)
    with pytest.raises(TypeError):
        moe.moe_expert_matmul(r, w, off, out, bias=torch.zeros(2, 16, dtype=bf16, **d))
    for kw in (dict(grad_x=r[:3]), dict(grad_weights=w[:1]), dict(x=r[:2]), dict(expert_offsets=off[:1])):
        a = dict(grad_pre=out, x=r, weights=w, expert_offsets=off, grad_x=r.clone(), grad_weights=w.clone())
        a.update(kw)
        with pytest.raises(ValueError):
            moe.moe_expert_matmul_backward(**a)
    with pytest.raises(moe.MoeError):
        moe.moe_expert_matmul_backward(out, r, w, off, r.clone(), w.clone(), accumulate=True)   # bf16 is not added to
    with pytest.raises(moe.MoeError):
        moe.moe_expert_activation_backward(out, out, off, out.clone(), "silu", grad_bias=torch.zeros(2, 16, **d))
    with pytest.raises(ValueError):
        moe.moe_expert_activation_backward(out, out[:, :8].contiguous(), off, out.clone(), "silu")
