"""moe_route_grouped, moe_expert_matmul and their gradients refuse memory of another
device than the current one, whichever argument it is.  The tensors here lie in host
memory and say that they are on a device; the library is a stand-in that counts its
calls."""
import pytest
import torch

from combine_moe_layout_05_gb300 import _binding, layer

HERE = 1                                                 # the current device


class OnDevice(torch.Tensor):
    is_cuda, at = True, HERE

    def get_device(self):
        return self.at


class Library:
    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(_binding, "_lib", lib)
    monkeypatch.setattr(_binding, "_current_stream", lambda: 0)
    monkeypatch.setattr(_binding, "_current_device", lambda: HERE)
    return lib


def on(t, at=HERE):
    t = t.as_subclass(OnDevice)
    t.at = at
    return t


def f(*shape):
    return torch.zeros(shape)


def h(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


T, E, K, ROWS, H, N = 4, 8, 2, 6, 16, 32
CALLS = {
    "moe_route_grouped": dict(logits=f(T, E), bias=f(E), topk_ids=i(T, K), topk_weights=f(T, K), expert_counts=i(E),
                              routed_tokens=i(1), loss=f(1), token_mask=torch.ones(T, dtype=torch.bool), workspace=f(1 << 14)),
    "moe_route_grouped_backward": dict(logits=f(T, E), topk_ids=i(T, K), expert_counts=i(E), routed_tokens=i(1),
                                       grad_weights=f(T, K), grad_loss=f(1), grad_logits=f(T, E)),
    "moe_expert_matmul": dict(x=h(ROWS, H), weights=h(E, N, H), expert_offsets=i(E + 1), out=h(ROWS, N), bias=f(E, N),
                              residual=h(ROWS, N), pre=h(ROWS, N), dev_error=i(1)),
    "moe_expert_activation_backward": dict(pre=h(ROWS, N), grad_out=h(ROWS, N), expert_offsets=i(E + 1), grad_pre=h(ROWS, N),
                                           grad_bias=f(E, N), workspace=f(1 << 14)),
    "moe_expert_matmul_backward": dict(grad_pre=h(ROWS, N), x=h(ROWS, H), weights=h(E, N, H), expert_offsets=i(E + 1),
                                       grad_x=h(ROWS, H), grad_weights=h(E, N, H), dev_error=i(1)),
}
SETTINGS = {"moe_expert_matmul": dict(activation="silu"), "moe_expert_activation_backward": dict(activation="silu")}


@pytest.mark.parametrize("name", CALLS)
def test_all_on_the_current_device(lib, name):
    args = {k: on(v) for k, v in CALLS[name].items()}
    getattr(_binding, name)(**args, **SETTINGS.get(name, {}))
    assert lib.calls == 1


@pytest.mark.parametrize("name,arg", [(n, a) for n in CALLS for a in CALLS[n]])
def test_one_on_another_device(lib, name, arg):
    args = {k: on(v, HERE - (k == arg)) for k, v in CALLS[name].items()}
    with pytest.raises(ValueError, match=f"{arg} is on device {HERE - 1}"):
        getattr(_binding, name)(**args, **SETTINGS.get(name, {}))
    assert lib.calls == 0


@pytest.mark.parametrize("name", CALLS)
def test_all_on_another_device(lib, name):
    args = {k: on(v, HERE - 1) for k, v in CALLS[name].items()}
    with pytest.raises(ValueError, match="is on device"):
        getattr(_binding, name)(**args, **SETTINGS.get(name, {}))
    assert lib.calls == 0


@pytest.mark.parametrize("name,arg", [(n, a) for n in CALLS for a in CALLS[n]])
def test_one_in_host_memory(lib, name, arg):
    args = {k: v if k == arg else on(v) for k, v in CALLS[name].items()}
    with pytest.raises(ValueError, match="CUDA tensor"):
        getattr(_binding, name)(**args, **SETTINGS.get(name, {}))
    assert lib.calls == 0


@pytest.mark.parametrize("arg", ["x", "topk_ids", "topk_weights"])
def test_experts(lib, arg):
    experts = layer.Experts(h(E, 2 * N, H), h(E, H, N))
    args = dict(x=h(T, H), topk_ids=i(T, K), topk_weights=f(T, K))
    with pytest.raises(ValueError, match=f"{arg} is on device"):
        experts(**{k: on(v, HERE - (k == arg)) for k, v in args.items()})
    assert lib.calls == 0
