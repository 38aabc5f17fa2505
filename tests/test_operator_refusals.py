"""moe_route, moe_route_backward, moe_dispatch_int8 and moe_expert_matmul_int8
refuse bad arguments on the host, before any CUDA call (so these run without
a GPU), and the binding refuses wrong types, sizes and layouts."""
import ctypes

import pytest
import torch

import combine_moe_layout_05_gb300 as moe
from combine_moe_layout_05_gb300 import build as moe_build

FAKE = 0x10000            # never dereferenced: the checks come first
P = ctypes.c_void_p
INVALID, ALIGNMENT, WORKSPACE = 1, 2, 4


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return moe.load()


def test_route(lib):
    def f(logits=FAKE, bf16=0, T=4, E=16, K=2, renorm=1, mask=None, ids=FAKE, w=FAKE, cnt=FAKE, n=FAKE, loss=FAKE,
          ws=FAKE, wsb=1 << 20):
        return lib.moe_route(P(logits), bf16, T, E, K, renorm, 1.0, P(mask), P(ids), P(w), P(cnt),
                             P(n), P(loss), P(ws), wsb, None)
    for kw in (dict(T=-1), dict(E=0), dict(E=1025), dict(K=0), dict(K=17), dict(K=33, E=64),
               dict(bf16=2), dict(renorm=-1), dict(logits=0), dict(ids=0), dict(w=0), dict(cnt=0),
               dict(n=0), dict(loss=0), dict(T=2 ** 28, K=16)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(logits=FAKE + 2), dict(bf16=1, logits=FAKE + 1), dict(ids=FAKE + 2), dict(w=FAKE + 1),
               dict(cnt=FAKE + 2), dict(n=FAKE + 2), dict(loss=FAKE + 2), dict(ws=FAKE + 8)):
        assert f(**kw) == ALIGNMENT, kw
    need = moe.moe_route_workspace_bytes(4, 16)
    assert need > 0 and f(wsb=need - 1) == WORKSPACE and f(ws=0) == WORKSPACE
    assert moe.moe_route_workspace_bytes(4, 1025) == 0
    assert moe.moe_route_workspace_bytes(-1, 16) == 0


def test_route_backward(lib):
    def f(logits=FAKE, bf16=0, T=4, E=16, K=2, renorm=1, ids=FAKE, cnt=FAKE, n=FAKE, dw=FAKE, dl=FAKE, grad=FAKE):
        return lib.moe_route_backward(P(logits), bf16, T, E, K, renorm, 1.0, P(ids), P(cnt), P(n),
                                      P(dw), P(dl), P(grad), None)
    for kw in (dict(T=-1), dict(E=0), dict(E=1025), dict(K=0), dict(K=17), dict(bf16=3), dict(renorm=2),
               dict(logits=0), dict(ids=0), dict(cnt=0), dict(n=0), dict(grad=0)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(logits=FAKE + 2), dict(grad=FAKE + 2), dict(ids=FAKE + 2), dict(dw=FAKE + 2),
               dict(dl=FAKE + 1), dict(bf16=1, grad=FAKE + 1)):
        assert f(**kw) == ALIGNMENT, kw
    assert f(T=0, logits=0, grad=0) == 0                 # T == 0: no-op


def test_dispatch_int8(lib):
    def f(x=FAKE, T=4, H=32, K=2, dst=FAKE, q=FAKE, s=FAKE):
        return lib.moe_dispatch_int8(P(x), T, H, K, P(dst), P(q), P(s), None)
    for kw in (dict(T=-1), dict(H=0), dict(H=24), dict(H=8), dict(K=0), dict(K=33), dict(x=0), dict(dst=0),
               dict(q=0), dict(s=0), dict(T=2 ** 30, K=2)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(x=FAKE + 8), dict(q=FAKE + 8), dict(dst=FAKE + 2), dict(s=FAKE + 2)):
        assert f(**kw) == ALIGNMENT, kw
    assert f(T=0, x=0, q=0) == 0


def test_expert_matmul_int8(lib):
    def f(x=FAKE, xs=FAKE, w=FAKE, ws=FAKE, off=FAKE, rows=4, H=32, N=8, E=2, out=FAKE, err=0):
        return lib.moe_expert_matmul_int8(P(x), P(xs), P(w), P(ws), P(off), rows, H, N, E, P(out), P(err), None)
    for kw in (dict(rows=-1), dict(H=0), dict(H=24), dict(H=65552), dict(N=0), dict(E=0), dict(E=1025),
               dict(E=1024, N=2 ** 21), dict(x=0), dict(xs=0), dict(w=0), dict(ws=0), dict(off=0), dict(out=0)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(x=FAKE + 8), dict(w=FAKE + 8), dict(out=FAKE + 8), dict(xs=FAKE + 2), dict(ws=FAKE + 2),
               dict(off=FAKE + 2), dict(err=FAKE + 2)):
        assert f(**kw) == ALIGNMENT, kw
    assert f(rows=0, x=0, out=0) == 0


def _route_args(T=4, E=16, K=2):
    return [torch.zeros(T, E), torch.zeros(T, K, dtype=torch.int32), torch.zeros(T, K),
            torch.zeros(E, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(1)]


def test_binding_types_and_sizes(lib):
    a = _route_args()
    with pytest.raises(TypeError):
        moe.moe_route(a[0].half(), *a[1:])
    with pytest.raises(ValueError):
        moe.moe_route(*a)                                # host tensors
    with pytest.raises(ValueError):
        moe.moe_route(torch.zeros(16, 4).t(), *a[1:])    # strided
    x, w = torch.zeros(4, 32, dtype=torch.int8), torch.zeros(2, 8, 32, dtype=torch.int8)
    off, out = torch.zeros(3, dtype=torch.int32), torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        moe.moe_expert_matmul_int8(x.float(), torch.zeros(4), w, torch.zeros(2, 8), off, out)
    with pytest.raises(ValueError):
        moe.moe_expert_matmul_int8(x, torch.zeros(4), w, torch.zeros(2, 8), off, out)    # host tensors
    with pytest.raises(TypeError):
        moe.moe_dispatch_int8(torch.zeros(4, 32), off, x, torch.zeros(4))
    with pytest.raises(TypeError):
        moe.moe_route_backward(a[0].double(), a[1], a[3], a[4], None, None, a[0].double())


@pytest.mark.gpu
def test_binding_sizes_on_the_gpu(lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    a = [t.cuda() for t in _route_args()]
    ws = torch.empty(moe.moe_route_workspace_bytes(4, 16), dtype=torch.uint8, device="cuda")
    with pytest.raises(moe.MoeError):
        moe.moe_route(*a)                                # no workspace
    with pytest.raises(ValueError):
        moe.moe_route(a[0], a[1], a[2][:3], *a[3:], workspace=ws)
    with pytest.raises(ValueError):
        moe.moe_route(*a, token_mask=torch.ones(3, dtype=torch.bool, device="cuda"), workspace=ws)
    with pytest.raises(TypeError):
        moe.moe_route(*a, token_mask=torch.ones(4, dtype=torch.uint8, device="cuda"), workspace=ws)
    x = torch.zeros(4, 32, dtype=torch.int8, device="cuda")
    w = torch.zeros(2, 8, 32, dtype=torch.int8, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda")
    one, sc = torch.ones(4, device="cuda"), torch.ones(2, 8, device="cuda")
    with pytest.raises(TypeError):
        moe.moe_expert_matmul_int8(x, one, w, sc, off, out.float())
    with pytest.raises(ValueError):
        moe.moe_expert_matmul_int8(x, one, w[:, :, :16].contiguous(), sc, off, out)
    with pytest.raises(ValueError):
        moe.moe_expert_matmul_int8(x, one, w, sc, off[:2], out)
    with pytest.raises(ValueError):
        moe.moe_expert_matmul_int8(x, one, w, sc, off, out[:3])
