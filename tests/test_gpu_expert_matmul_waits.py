"""Each bounded wait of moe_expert_matmul_int8 made to run out, in each of its
forms: the call returns, the error word is the timeout bit, and the next call is
right bit for bit.  One barrier of the first tiles' CTAs waits for an arrival
that never comes, with a bound of some 2 ms on every wait."""
import ctypes
import time

import numpy as np
import pytest
import torch

import combine_moe_layout_05_gb300 as moe

pytestmark = pytest.mark.gpu

WAIT_CYCLES = 4_000_000
# a tile's bytes, their slot, widened operands, their slot, sums ready, sums
# stored, and the sums of the other CTAs that share a contraction
KINDS = ["bytes", "byte_slot", "operands", "operand_slot", "sums", "accumulator", "shared_sums"]
# counts, H, N: more steps than the rings have slots, and more tiles than accumulators
FORMS = {
    "narrow": ([5] * 40, 1920, 1300),
    "mid": ([100, 129, 300, 64] * 4, 1920, 1300),
    "wide": ([2000], 2560, 2600),
    "split": ([12, 8], 7168, 256),
}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_moe_layout_05_gb300 import build
    build.build()
    moe.load()


def _hook():
    f = moe.load().moe_testing_expert_matmul_int8
    P, i32 = ctypes.c_void_p, ctypes.c_int32
    f.argtypes = [P, P, P, P, P, i32, i32, i32, i32, P, P, ctypes.c_int64, i32, P]
    f.restype = i32
    return f


def _inputs(form):
    counts, H, N = FORMS[form]
    E, rows = len(counts), sum(counts)
    lim = int((2 ** 24 / H) ** 0.5)                      # sums stay below 2^24, so they are the integers'
    g = torch.Generator(device="cuda").manual_seed(len(form))
    codes = lambda *shape: torch.randint(-lim, lim + 1, shape, generator=g, device="cuda", dtype=torch.int8)
    x, w = codes(rows, H), codes(E, N, H)
    xs, ws = (torch.rand(s, generator=g, device="cuda") + 0.1 for s in ((rows,), (E, N)))
    o = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    e = torch.repeat_interleave(torch.arange(E, device="cuda"), torch.tensor(counts, device="cuda"))
    want = torch.cat([(r.double() @ w[i].double().t()).float() for i, r in enumerate(torch.split(x, counts))])
    return x, xs, w, ws, o, (want * xs[:, None] * ws[e]).to(torch.bfloat16)


def _call(inputs, stall, wait_cycles):
    x, xs, w, ws, o, want = inputs
    out, err = torch.zeros_like(want), torch.full((1,), 77, dtype=torch.int32, device="cuda")
    status = _hook()(x.data_ptr(), xs.data_ptr(), w.data_ptr(), ws.data_ptr(), o.data_ptr(), x.shape[0], x.shape[1],
                     w.shape[1], w.shape[0], out.data_ptr(), err.data_ptr(), wait_cycles, stall,
                     torch.cuda.current_stream().cuda_stream)
    assert status == 0
    torch.cuda.synchronize()
    return out, err.item()


@pytest.mark.parametrize("form", list(FORMS))
def test_nothing_held_back(form):
    """The bound that the other tests set is never reached by itself."""
    inputs = _inputs(form)
    out, err = _call(inputs, -1, WAIT_CYCLES)
    assert err == 0 and torch.equal(out, inputs[-1])


@pytest.mark.parametrize("form,kind", [(f, k) for f in FORMS for k in KINDS if k != "shared_sums" or f == "split"])
def test_an_expired_wait_is_reported(form, kind):
    inputs = _inputs(form)
    start = time.time()
    _, err = _call(inputs, KINDS.index(kind), WAIT_CYCLES)
    assert time.time() - start < 30
    assert err == moe.MOE_DEV_ERR_TIMEOUT
    x, xs, w, ws, o, want = inputs
    out, word = torch.zeros_like(want), torch.full((1,), 77, dtype=torch.int32, device="cuda")
    for _ in range(3):                                   # the context and the multiprocessors are as before
        moe.moe_expert_matmul_int8(x, xs, w, ws, o, out, word)
        assert word.item() == 0 and torch.equal(out, want)
        out.zero_()
