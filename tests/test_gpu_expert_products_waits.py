"""Each bounded wait of moe_expert_matmul and of its gradients made to run out, in
each of their forms: the call returns, the error word is the timeout bit, and the
next call is bit for bit what the call before was.  One barrier of the first
tiles' CTAs waits for an arrival that never comes, with a bound of some 2 ms on
every wait."""
import ctypes
import time

import numpy as np
import pytest
import torch

import combine_moe_layout_05_gb300 as moe

pytestmark = pytest.mark.gpu

WAIT_CYCLES = 4_000_000
KINDS = ["landed", "slot", "landed_in_both", "sums", "accumulator", "shared_sums"]
# pass, counts, H, N, activation: more steps than the rings have slots, and more tiles than accumulators
FORMS = {
    "narrow": ("forward", [5] * 40, 1040, 1300, 0),
    "narrow_gated": ("forward", [5] * 40, 1040, 1300, 3),
    "mid": ("forward", [100, 129, 150, 64] * 4, 1040, 2600, 1),
    "wide": ("forward", [2000], 1040, 20800, 3),
    "split": ("forward", [12, 8], 7168, 256, 2),
    "rows_narrow": ("rows", [5] * 40, 1304, 1040, 0),
    "rows_mid": ("rows", [100, 129, 150, 64] * 4, 2600, 1040, 0),
    "rows_wide": ("rows", [2000], 10400, 1040, 0),
    "weights": ("weights", [900, 0, 700, 33], 2600, 1040, 0),
}
PAIRS = [f for f in FORMS if "narrow" not in f and f != "split"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_moe_layout_05_gb300 import build
    build.build()
    moe.load()


def _hooks():
    P, i32 = ctypes.c_void_p, ctypes.c_int32
    f, g = moe.load().moe_testing_expert_matmul, moe.load().moe_testing_expert_matmul_backward
    f.argtypes = [P, P, P, i32, i32, i32, i32, i32, P, P, ctypes.c_int64, i32, P]
    g.argtypes = [P, P, P, i32, i32, i32, i32, i32, P, P, ctypes.c_int64, i32, P]
    f.restype = g.restype = i32
    return f, g


def _inputs(form):
    what, counts, H, N, act = FORMS[form]
    E, rows = len(counts), sum(counts)
    g = torch.Generator(device="cuda").manual_seed(len(form))
    rand = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    o = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    if what == "forward":
        a, b, shape = rand(rows, H), rand(E, N, H), (rows, N // 2 if act == 3 else N)
    elif what == "rows":
        a, b, shape = rand(rows, N), rand(E, N, H), (rows, H)
    else:
        a, b, shape = rand(rows, N), rand(rows, H), (E, N, H)
    return what, a, b, o, (rows, H, N, E), act, shape


def _call(inputs, stall, wait_cycles):
    what, a, b, o, sizes, act, shape = inputs
    out, err = torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), torch.full((1,), 77, dtype=torch.int32, device="cuda")
    f, g = _hooks()
    last = (out.data_ptr(), err.data_ptr(), wait_cycles, stall, torch.cuda.current_stream().cuda_stream)
    if what == "forward":
        status = f(a.data_ptr(), b.data_ptr(), o.data_ptr(), *sizes, act, *last)
    else:
        status = g(a.data_ptr(), b.data_ptr(), o.data_ptr(), *sizes, int(what == "weights"), *last)
    assert status == 0
    torch.cuda.synchronize()
    return out, err.item()


@pytest.mark.parametrize("form", list(FORMS))
def test_nothing_held_back(form):
    """The bound that the other tests set is never reached by itself."""
    inputs = _inputs(form)
    out, err = _call(inputs, -1, WAIT_CYCLES)
    again, _ = _call(inputs, -1, 0)
    assert err == 0 and torch.equal(out, again)


@pytest.mark.parametrize("form,kind", [(f, k) for f in FORMS for k in KINDS
                                       if (k != "shared_sums" or f == "split") and (k != "landed_in_both" or f in PAIRS)])
def test_an_expired_wait_is_reported(form, kind):
    inputs = _inputs(form)
    want, _ = _call(inputs, -1, 0)
    start = time.time()
    _, err = _call(inputs, KINDS.index(kind), WAIT_CYCLES)
    assert time.time() - start < 30
    assert err == moe.MOE_DEV_ERR_TIMEOUT
    for _ in range(2):                                   # the context and the multiprocessors are as before
        out, err = _call(inputs, -1, 0)
        assert err == 0 and torch.equal(out, want)


def test_the_error_word_is_cleared():
    """By both gradients in one call, which share it, and by one alone."""
    g, x, w = (torch.randn(s, device="cuda").to(torch.bfloat16) for s in ((40, 64), (40, 72), (2, 64, 72)))
    o = torch.tensor([0, 10, 40], dtype=torch.int32, device="cuda")
    err = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    moe.moe_expert_matmul_backward(g, x, w, o, torch.empty_like(x), torch.empty_like(w), dev_error=err)
    assert err.item() == 0
    err.fill_(77)
    moe.moe_expert_matmul_backward(g, x, None, o, None, torch.empty_like(w), dev_error=err)
    assert err.item() == 0
