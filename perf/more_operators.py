"""What the grouped router and the bf16 expert operators are measured on: their cases, their plain
forms in elementary torch operations, and their definitions in 64 bits.

Operators
  route                router logits -> ids, weights, counts and the balance loss: softmax or sigmoid scores,
                       a balance bias for the choice alone, groups of experts, renormalised and scaled weights
  route_backward       the gradient of the weights and of the loss with respect to the logits
  matmul               packed rows times their experts' bf16 weights, with bias, activation (gated or not)
                       and residual in the same pass, and the values before the activation for training
  activation_backward  the gradient at those values, and each expert's bias gradient
  matmul_backward      the gradients of the rows and of the weights

Sizes are those of the package's workloads (T, H, E, K and the routing's skew) with a generic number
of channels N, and ragged sizes beside them.
"""
from __future__ import annotations

import functools
import math

import torch

own = False

LOSS_COEF = 0.01
SCALE = 2.5
GATED = ("swiglu",)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one new token of a served sequence: latency only
        dict(name="route_one_token", op="route", T=1, E=256, K=8, dtype="f32", scoring="sigmoid", bias=True,
             groups=8, top_groups=4, group_top=2, renorm=True, padded=0.0, closed=0),
        # the largest prefill or training batch, the usual groups
        dict(name="route_prefill", op="route", T=16384, E=256, K=8, dtype="f32", scoring="sigmoid", bias=True,
             groups=8, top_groups=4, group_top=2, renorm=True, padded=0.0, closed=0),
        # training steps: the widest router without groups, and a long padded batch of softmax scores in bf16
        dict(name="route_backward_wide", op="route_backward", T=4096, E=384, K=8, dtype="f32", scoring="sigmoid",
             bias=True, groups=1, top_groups=1, group_top=1, renorm=True, padded=0.0, closed=0),
        dict(name="route_backward_bf16", op="route_backward", T=16384, E=128, K=6, dtype="bf16", scoring="softmax",
             bias=False, groups=8, top_groups=3, group_top=1, renorm=False, padded=0.1, closed=3),
        # one token's experts: eight rows, each with weights of its own
        dict(name="matmul_one_token", op="matmul", T=1, H=7168, N=4096, E=256, K=8, zipf=0.0, activation="swiglu",
             bias=False, residual=False, pre=False),
        # a decode step: a few rows for nearly every expert, bound by the weights' bytes
        dict(name="matmul_decode", op="matmul", T=128, H=7168, N=4096, E=256, K=8, zipf=0.0, activation="swiglu",
             bias=False, residual=False, pre=False),
        # odd everything: channels, row counts, a contraction that ends inside a tile, all of the epilogue
        dict(name="matmul_ragged", op="matmul", T=777, H=2056, N=1001, E=48, K=6, zipf=1.0, activation="gelu",
             bias=True, residual=True, pre=False),
        # the largest training batch's gate and up products, bound by the products
        dict(name="matmul_prefill_large", op="matmul", T=16384, H=4096, N=4096, E=128, K=8, zipf=1.0,
             activation="swiglu", bias=True, residual=False, pre=True),
        # the same batch on its way back, and a small one of odd sizes
        dict(name="activation_backward_large", op="activation_backward", T=16384, N=4096, E=128, K=8, zipf=1.0,
             activation="swiglu", bias=True),
        dict(name="activation_backward_ragged", op="activation_backward", T=777, N=1032, E=48, K=6, zipf=1.0,
             activation="gelu", bias=True),
        # a training step's two products: a skewed batch, and few rows of odd sizes into fp32 gradients
        dict(name="matmul_backward_large", op="matmul_backward", T=8192, H=4096, N=2048, E=128, K=8, zipf=1.0,
             f32=False),
        dict(name="matmul_backward_ragged", op="matmul_backward", T=500, H=1032, N=776, E=24, K=4, zipf=1.2,
             f32=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "matmul", "matmul", "activation_backward", "matmul_backward"])
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 1, 2, 4, 5, 8])
        E = groups * max(2, _log_int(rng, 8, 512) // groups)
        top_groups = rng.randint(1, groups)
        return dict(op=op, T=_log_int(rng, 1 if op == "route" else 16, max(16, min(16384, (1 << 22) // E))),
                    E=E, K=rng.randint(1, min(8, E // groups * top_groups)), dtype=rng.choice(["f32", "bf16"]),
                    scoring=rng.choice(["sigmoid", "softmax"]), bias=rng.random() < 0.6, groups=groups,
                    top_groups=top_groups, group_top=rng.choice([1, 2]), renorm=rng.random() < 0.5,
                    padded=rng.choice([0.0, 0.0, 0.25]), closed=rng.choice([0, 0, 2]) if E >= 16 else 0)
    K = rng.randint(1, 8)
    E = _log_int(rng, 1, 384)
    K = min(K, E)
    T = _log_int(rng, 1, 16384)
    zipf = rng.choice([0.0, 0.7, 1.2])
    activation = rng.choice(["none", "silu", "gelu", "swiglu", "swiglu"])
    H = 8 * _log_int(rng, 8, 896)
    if op == "matmul":
        N = _log_int(rng, 64, 4096)
        if rng.random() < 0.5:
            N = -(-N // 8) * 8
        if activation in GATED:
            N = -(-N // 2) * 2
        E = max(K, min(E, 256 * 4096 * 7168 // (N * H)))
        T = max(1, min(T, 131072 * 4096 * 4096 // (N * H * K)))
        return dict(op=op, T=T, H=H, N=N, E=E, K=K, zipf=zipf, activation=activation, bias=rng.random() < 0.5,
                    residual=rng.random() < 0.3, pre=rng.random() < 0.3)
    N = 8 * _log_int(rng, 8, 512)
    if op == "activation_backward":
        if activation in GATED:
            N = -(-N // 16) * 16
        return dict(op=op, T=T, N=N, E=E, K=K, zipf=zipf, activation=activation, bias=rng.random() < 0.7)
    E = max(K, min(E, 128 * 2048 * 4096 // (N * H)))
    T = max(1, min(T, 65536 * 2048 * 4096 // (N * H * K)))
    return dict(op=op, T=T, H=H, N=N, E=E, K=K, zipf=zipf, f32=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _routing(T, E, K, zipf, gen, device):
    """[T, K] distinct expert ids a token: uniform, or drawn one after another in proportion to
    rank^-zipf over a random order of the experts (the K largest of log weight + Gumbel noise)."""
    logw = -zipf * torch.log(torch.arange(1, E + 1, device=device, dtype=torch.float32))
    order = torch.randperm(E, generator=gen, device=device)
    u = torch.rand((T, E), generator=gen, device=device).clamp_(1e-30, 1 - 2.0 ** -24)
    pick = torch.sort(logw - torch.log(-torch.log(u)), dim=1, descending=True, stable=True)[1][:, :K]
    return order[pick]


def _offsets(c, gen):
    """First packed row of each expert, [E + 1]."""
    ids = _routing(c["T"], c["E"], c["K"], c["zipf"], gen, "cuda").reshape(-1)
    counts = torch.zeros(c["E"], dtype=torch.long, device="cuda").index_add_(0, ids, torch.ones_like(ids))
    offsets = torch.zeros(c["E"] + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    return dict(expert_offsets=offsets, offsets_host=offsets.tolist())


def _normal(shape, gen, std=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=gen)


def _rows(shape, gen):
    """Activations: rows of different size."""
    return _normal(shape, gen) * torch.exp(0.5 * _normal((shape[0], 1), gen))


def _prepare_route(c, seed):
    g, T, E, K = _gen(seed), c["T"], c["E"], c["K"]
    # a shared lean of the experts plus each token's own preference
    x = torch.randn((T, E), generator=g, device="cuda") * 1.5
    x += torch.randn((1, E), generator=g, device="cuda") * 0.5
    if c["closed"]:
        x[:, torch.randperm(E, generator=g, device="cuda")[: c["closed"]]] = -math.inf
    mask = torch.rand((T,), generator=g, device="cuda") >= c["padded"] if c["padded"] > 0 else None
    # a balance bias as training leaves it: a number of equal steps up or down
    bias = torch.randint(-60, 61, (E,), generator=g, device="cuda").float() * 0.001 if c["bias"] else None
    i32 = dict(dtype=torch.int32, device="cuda")
    s = dict(case=c, logits=x.to(torch.bfloat16 if c["dtype"] == "bf16" else torch.float32), mask=mask, bias=bias)
    if c["op"] == "route":
        s.update(topk_ids=torch.empty((T, K), **i32), topk_weights=torch.empty((T, K), device="cuda"),
                 expert_counts=torch.empty(E, **i32), routed_tokens=torch.empty(1, **i32),
                 loss=torch.empty(1, device="cuda"),
                 # room for each block's partial counts and score sums
                 workspace=torch.empty(8 << 20, dtype=torch.uint8, device="cuda"))
        return s
    f = _plain_route(s)
    s.update(topk_ids=f["topk_ids"], expert_counts=f["expert_counts"], routed_tokens=f["routed_tokens"],
             grad_weights=torch.randn((T, K), generator=g, device="cuda"),
             grad_loss=torch.ones(1, device="cuda"), grad_logits=torch.empty_like(s["logits"]))
    return s


def _prepare_matmul(c, seed):
    g, rows, H, N, E = _gen(seed), c["T"] * c["K"], c["H"], c["N"], c["E"]
    C = N // 2 if c["activation"] in GATED else N
    s = dict(case=c, **_offsets(c, g), x=_rows((rows, H), g), weights=_normal((E, N, H), g, H ** -0.5),
             bias=torch.randn((E, N), generator=g, device="cuda") * 0.3 if c["bias"] else None,
             residual=_normal((rows, C), g) if c["residual"] else None)
    s.update(out=torch.empty((rows, C), dtype=torch.bfloat16, device="cuda"),
             pre=torch.empty((rows, N), dtype=torch.bfloat16, device="cuda") if c["pre"] else None)
    return s


def _prepare_activation_backward(c, seed):
    g, rows, N, E = _gen(seed), c["T"] * c["K"], c["N"], c["E"]
    C = N // 2 if c["activation"] in GATED else N
    s = dict(case=c, **_offsets(c, g), pre=_rows((rows, N), g), grad_out=_normal((rows, C), g))
    s.update(grad_pre=torch.empty_like(s["pre"]), grad_bias=torch.empty((E, N), device="cuda") if c["bias"] else None,
             # room for the bias gradient's partial sums
             workspace=torch.empty((min(rows, E) + rows // 32 + 1) * N * 4 + 4096, dtype=torch.uint8, device="cuda"))
    return s


def _prepare_matmul_backward(c, seed):
    g, rows, H, N, E = _gen(seed), c["T"] * c["K"], c["H"], c["N"], c["E"]
    s = dict(case=c, **_offsets(c, g), grad_pre=_rows((rows, N), g), x=_rows((rows, H), g),
             weights=_normal((E, N, H), g, H ** -0.5))
    s.update(grad_x=torch.empty_like(s["x"]),
             grad_weights=torch.empty((E, N, H), dtype=torch.float32 if c["f32"] else torch.bfloat16, device="cuda"))
    return s


def prepare(case, seed):
    return {"route": _prepare_route, "route_backward": _prepare_route, "matmul": _prepare_matmul,
            "activation_backward": _prepare_activation_backward,
            "matmul_backward": _prepare_matmul_backward}[case["op"]](case, seed)


# ---------------------------------------------------------------- plain forms

def _open(x, mask):
    live = x > -math.inf
    return live if mask is None else live & mask[:, None]


def _scores(x, live, scoring):
    """Scores in the type of x; 0 where an expert is not open."""
    if scoring == "sigmoid":
        return torch.where(live, 1 / (1 + torch.exp(-x)), torch.zeros_like(x))
    m = torch.where(live, x, -math.inf).amax(1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.where(live, torch.exp(x - m), torch.zeros_like(x))
    return e / _nonzero(e.sum(1, keepdim=True))


def _nonzero(s):
    return torch.where(s == 0, torch.ones_like(s), s)


def _choose(c, x, live, bias):
    """ids [T, K], -1 where fewer are open.  In 64 bits: two experts may be nearer than fp32's rounding."""
    key = _scores(x.double(), live, c["scoring"])
    if bias is not None:
        key = key + bias.double()
    key = torch.where(live, key, -math.inf)
    G = c["groups"]
    if c["top_groups"] < G:
        parts = torch.sort(key.view(key.shape[0], G, -1), dim=2, descending=True)[0]
        score = parts[:, :, 0]
        if c["group_top"] == 2:
            score = score + torch.where(parts[:, :, 1] > -math.inf, parts[:, :, 1], 0.0)
        kept = torch.sort(score, dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
        keep = torch.zeros_like(score).scatter_(1, kept, 1.0) > 0
        key = torch.where(keep.repeat_interleave(key.shape[1] // G, 1), key, -math.inf)
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    ids = ids[:, :c["K"]]
    return torch.where(top[:, :c["K"]] > -math.inf, ids, torch.full_like(ids, -1))


def _plain_route(s):
    c, x = s["case"], s["logits"].float()
    E, K = c["E"], c["K"]
    live = _open(x, s["mask"])
    score = _scores(x, live, c["scoring"])
    ids = _choose(c, x, live, s["bias"])
    taken = ids >= 0
    w = torch.where(taken, score.gather(1, ids.clamp(min=0)), torch.zeros_like(score[:, :K]))
    if c["renorm"]:
        w = w / _nonzero(w.sum(1, keepdim=True))
    counts = torch.zeros(E, dtype=torch.int32, device=x.device).index_add_(
        0, ids.clamp(min=0).reshape(-1), taken.reshape(-1).to(torch.int32))
    routed = live.any(1).sum().to(torch.int32).view(1)
    n = routed.clamp(min=1).float()
    p = score / _nonzero(score.sum(1, keepdim=True))
    loss = LOSS_COEF * E * ((counts.float() / (K * n)) * (p.sum(0) / n)).sum().view(1)
    return dict(topk_ids=ids.to(torch.int32), topk_weights=w * SCALE, expert_counts=counts,
                routed_tokens=routed, loss=loss)


def _plain_route_backward(s):
    c, x, ids = s["case"], s["logits"].float(), s["topk_ids"].long()
    E, K = c["E"], c["K"]
    live = _open(x, s["mask"])
    score = _scores(x, live, c["scoring"])
    total = _nonzero(score.sum(1, keepdim=True))
    p = score / total
    n = s["routed_tokens"].clamp(min=1).float()
    a = s["grad_loss"] * LOSS_COEF * E * s["expert_counts"].float() / (K * n * n)
    grad = (a - (p * a).sum(1, keepdim=True)) / total                 # at the scores
    taken = ids >= 0
    at = ids.clamp(min=0)
    w = torch.where(taken, score.gather(1, at), torch.zeros_like(p[:, :K]))
    dw = torch.where(taken, s["grad_weights"] * SCALE, torch.zeros_like(w))
    if c["renorm"]:
        sum_w = _nonzero(w.sum(1, keepdim=True))
        dw = torch.where(taken, (dw - (w / sum_w * dw).sum(1, keepdim=True)) / sum_w, torch.zeros_like(w))
    grad = grad.scatter_add(1, at, dw)
    if c["scoring"] == "sigmoid":
        slope = torch.where(live, score / (1 + torch.exp(x)), torch.zeros_like(x))
        return dict(grad_logits=(slope * grad).to(s["logits"].dtype))
    return dict(grad_logits=(score * (grad - (score * grad).sum(1, keepdim=True))).to(s["logits"].dtype))


def _gelu_argument(z):
    """gelu(z) = z * sigmoid of this."""
    return 1.5957691216057308 * (z + 0.044715 * z * z * z)


def _activate(z, activation):
    if activation == "none":
        return z
    if activation == "swiglu":
        gate, up = z.chunk(2, dim=1)
        return gate / (1 + torch.exp(-gate)) * up
    return z / (1 + torch.exp(-(z if activation == "silu" else _gelu_argument(z))))


def _experts(s):
    """(expert, its rows) of the experts that have rows."""
    o = s["offsets_host"]
    return [(e, slice(o[e], o[e + 1])) for e in range(s["case"]["E"]) if o[e + 1] > o[e]]


def _plain_matmul(s):
    c = s["case"]
    out = torch.empty_like(s["out"])
    pre = torch.empty_like(s["pre"]) if c["pre"] else None
    for e, r in _experts(s):                       # one matrix product an expert that has rows
        z = s["x"][r].float() @ s["weights"][e].float().t()
        if c["bias"]:
            z = z + s["bias"][e]
        if c["pre"]:
            pre[r] = z.to(torch.bfloat16)
        y = _activate(z, c["activation"])
        if c["residual"]:
            y = y + s["residual"][r].float()
        out[r] = y.to(torch.bfloat16)
    return dict(out=out, pre=pre) if c["pre"] else dict(out=out)


def _plain_activation_backward(s):
    c, z, dy = s["case"], s["pre"].float(), s["grad_out"].float()
    a = c["activation"]
    if a == "none":
        dz = dy
    elif a == "gelu":
        u = _gelu_argument(z)
        sig = 1 / (1 + torch.exp(-u))
        dz = dy * (sig + z * sig / (1 + torch.exp(u)) * 1.5957691216057308 * (1 + 3 * 0.044715 * z * z))
    else:
        gate = z.chunk(2, dim=1)[0] if a == "swiglu" else z
        sig = 1 / (1 + torch.exp(-gate))
        slope = sig + gate * sig / (1 + torch.exp(gate))
        dz = dy * slope if a == "silu" else torch.cat([dy * z.chunk(2, dim=1)[1] * slope, dy * gate * sig], 1)
    out = dict(grad_pre=dz.to(torch.bfloat16))
    if c["bias"]:
        bias = torch.zeros_like(s["grad_bias"])
        for e, r in _experts(s):
            bias[e] = dz[r].sum(0)
        out["grad_bias"] = bias
    return out


def _plain_matmul_backward(s):
    grad_x, grad_w = torch.empty_like(s["grad_x"]), torch.zeros_like(s["grad_weights"])
    for e, r in _experts(s):
        dz = s["grad_pre"][r].float()
        grad_x[r] = (dz @ s["weights"][e].float()).to(grad_x.dtype)
        grad_w[e] = (dz.t() @ s["x"][r].float()).to(grad_w.dtype)
    return dict(grad_x=grad_x, grad_weights=grad_w)


# ---------------------------------------------------------------- one pass

def _own(s):
    import combine_moe_layout_05_gb300 as moe
    c = s["case"]
    if c["op"] == "route":
        moe.moe_route_grouped(s["logits"], s["bias"], s["topk_ids"], s["topk_weights"], s["expert_counts"],
                              s["routed_tokens"], s["loss"], scoring=c["scoring"], groups=c["groups"],
                              top_groups=c["top_groups"], group_top=c["group_top"], renormalize=c["renorm"],
                              scale=SCALE, loss_coef=LOSS_COEF, token_mask=s["mask"], workspace=s["workspace"])
        return {k: s[k] for k in ("topk_ids", "topk_weights", "expert_counts", "routed_tokens", "loss")}
    if c["op"] == "route_backward":
        moe.moe_route_grouped_backward(s["logits"], s["topk_ids"], s["expert_counts"], s["routed_tokens"],
                                       s["grad_weights"], s["grad_loss"], s["grad_logits"], scoring=c["scoring"],
                                       renormalize=c["renorm"], scale=SCALE, loss_coef=LOSS_COEF)
        return dict(grad_logits=s["grad_logits"])
    if c["op"] == "matmul":
        moe.moe_expert_matmul(s["x"], s["weights"], s["expert_offsets"], s["out"], bias=s["bias"],
                              activation=c["activation"], residual=s["residual"], pre=s["pre"])
        return dict(out=s["out"], pre=s["pre"]) if c["pre"] else dict(out=s["out"])
    if c["op"] == "activation_backward":
        moe.moe_expert_activation_backward(s["pre"], s["grad_out"], s["expert_offsets"], s["grad_pre"],
                                           activation=c["activation"], grad_bias=s["grad_bias"],
                                           workspace=s["workspace"])
        out = dict(grad_pre=s["grad_pre"])
        return dict(out, grad_bias=s["grad_bias"]) if c["bias"] else out
    moe.moe_expert_matmul_backward(s["grad_pre"], s["x"], s["weights"], s["expert_offsets"], grad_x=s["grad_x"],
                                   grad_weights=s["grad_weights"])
    return dict(grad_x=s["grad_x"], grad_weights=s["grad_weights"])


def run(state):
    if own:
        return _own(state)
    return {"route": _plain_route, "route_backward": _plain_route_backward, "matmul": _plain_matmul,
            "activation_backward": _plain_activation_backward,
            "matmul_backward": _plain_matmul_backward}[state["case"]["op"]](state)


# ---------------------------------------------------------------- work

@functools.lru_cache(maxsize=None)
def _active_experts(T, E, K, zipf):
    """Experts that have a row, as one seeded draw of the routing has it (on the CPU)."""
    g = torch.Generator().manual_seed(0)
    return int(torch.unique(_routing(T, E, K, zipf, g, "cpu")).numel())


def work(case):
    T, K, E = case["T"], case["K"], case["E"]
    if case["op"] in ("route", "route_backward"):
        size = 2 if case["dtype"] == "bf16" else 4
        if case["op"] == "route":
            mask = T if case["padded"] > 0 else 0
            return dict(bytes=T * E * size + mask + T * K * 8 + E * (8 if case["bias"] else 4), flops=T * E * 8)
        return dict(bytes=2 * T * E * size + T * K * 8 + E * 4, flops=T * E * 12)
    N, rows = case["N"], T * K
    C = N // 2 if case.get("activation") in GATED else N
    if case["op"] == "activation_backward":
        return dict(bytes=rows * (2 * N + C) * 2 + (E * N * 4 if case["bias"] else 0), flops=rows * N * 10)
    H, active = case["H"], _active_experts(T, E, K, case["zipf"])
    if case["op"] == "matmul":
        out = C * (2 if case["residual"] else 1) + (N if case["pre"] else 0)
        return dict(bytes=rows * (H + out) * 2 + active * N * (2 * H + (4 if case["bias"] else 0)) + 4 * (E + 1),
                    flops=2 * rows * N * H)
    return dict(bytes=rows * (N + 2 * H) * 2 + active * N * H * 2 + E * N * H * (4 if case["f32"] else 2) + 4 * (E + 1),
                flops=4 * rows * N * H)


# ---------------------------------------------------------------- 64 bits

def _shut(s):
    x = s["logits"].double()
    return x if s["mask"] is None else x.masked_fill(~s["mask"][:, None], -math.inf)


def _score64(x, scoring):
    return torch.sigmoid(x) if scoring == "sigmoid" else torch.softmax(x, dim=1).nan_to_num(nan=0.0)


def _exact_route(s):
    c, (T, E), K, G = s["case"], s["logits"].shape, s["case"]["K"], s["case"]["groups"]
    x = _shut(s)
    shut = torch.isneginf(x)
    score = _score64(x, c["scoring"])
    key = score if s["bias"] is None else score + s["bias"].double()
    key = key.masked_fill(shut, -math.inf)
    if c["top_groups"] < G:
        best = key.reshape(T, G, E // G).topk(min(c["group_top"], E // G), dim=2).values
        # a group with one open expert counts that one
        value = torch.where(torch.isneginf(best), torch.zeros_like(best), best).sum(2)
        value = value.masked_fill(torch.isneginf(best[..., 0]), -math.inf)
        rank = torch.argsort(torch.argsort(-value, dim=1, stable=True), dim=1)
        drop = (rank >= c["top_groups"])[:, :, None].expand(T, G, E // G).reshape(T, E)
        key = key.masked_fill(drop, -math.inf)
    ids = torch.argsort(-key, dim=1, stable=True)[:, :K]
    none = torch.isneginf(key.gather(1, ids))
    w = score.gather(1, ids).masked_fill(none, 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=torch.finfo(torch.float64).tiny)
    ids = ids.masked_fill(none, -1)
    counts = torch.bincount((ids + 1).reshape(-1), minlength=E + 1)[1:]
    routed = T - int(shut.all(1).sum())
    p = score / score.sum(1, keepdim=True).clamp(min=torch.finfo(torch.float64).tiny)
    loss = LOSS_COEF * E * torch.dot(counts.double(), p.sum(0)) / (K * max(routed, 1) ** 2)
    return dict(topk_ids=ids.to(torch.int32), topk_weights=w * SCALE, expert_counts=counts.to(torch.int32),
                routed_tokens=torch.tensor([routed], dtype=torch.int32, device=x.device), loss=loss.view(1))


def _exact_route_backward(s):
    """By differentiating the forward's definition."""
    c, E, K = s["case"], s["case"]["E"], s["case"]["K"]
    x = _shut(s)
    rows = (x > -math.inf).any(1)
    z = x[rows].requires_grad_(True)
    score = torch.sigmoid(z) if c["scoring"] == "sigmoid" else torch.softmax(z, dim=1)
    ids = s["topk_ids"][rows].long()
    w = torch.where(ids >= 0, score.gather(1, ids.clamp(min=0)), torch.zeros((), dtype=z.dtype, device=z.device))
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    n = max(int(rows.sum()), 1)
    p = score / score.sum(1, keepdim=True)
    loss = LOSS_COEF * E * torch.dot(s["expert_counts"].double() / (K * n), p.sum(0) / n)
    total = (w * SCALE * s["grad_weights"][rows].double()).sum() + loss * s["grad_loss"].double().sum()
    grad = torch.zeros_like(x)
    if z.numel():
        grad[rows] = torch.autograd.grad(total, z)[0]
    return dict(grad_logits=grad)


def _activation64(z, activation):
    if activation == "none":
        return z
    if activation == "silu":
        return z * torch.sigmoid(z)
    if activation == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    half = z.shape[1] // 2
    return z[:, :half] * torch.sigmoid(z[:, :half]) * z[:, half:]


def _exact_matmul(s):
    c, o = s["case"], s["offsets_host"]
    outs, pres = [], []
    for e, (a, b) in enumerate(zip(o[:-1], o[1:])):
        if b <= a:
            continue
        z = torch.mm(s["x"][a:b].double(), s["weights"][e].double().T)
        if s["bias"] is not None:
            z += s["bias"][e].double()
        y = _activation64(z, c["activation"])
        outs.append(y + s["residual"][a:b].double() if c["residual"] else y)
        if c["pre"]:
            pres.append(z)
    return dict(out=torch.cat(outs), pre=torch.cat(pres)) if c["pre"] else dict(out=torch.cat(outs))


def _exact_activation_backward(s):
    """By differentiating the activation."""
    c, o = s["case"], s["offsets_host"]
    bias = torch.zeros((c["E"], c["N"]), dtype=torch.float64, device="cuda")
    parts = []
    for e, (a, b) in enumerate(zip(o[:-1], o[1:])):
        if b <= a:
            continue
        z = s["pre"][a:b].double().requires_grad_(True)
        y = _activation64(z, c["activation"])
        parts.append(torch.autograd.grad(y, z, s["grad_out"][a:b].double())[0])
        bias[e] = parts[-1].sum(0)
    out = dict(grad_pre=torch.cat(parts))
    return dict(out, grad_bias=bias) if c["bias"] else out


def _exact_matmul_backward(s):
    c, o = s["case"], s["offsets_host"]
    grad_w = torch.zeros((c["E"], c["N"], c["H"]), dtype=torch.float64, device="cuda")
    parts = []
    for e, (a, b) in enumerate(zip(o[:-1], o[1:])):
        if b > a:
            dz, x = s["grad_pre"][a:b].double(), s["x"][a:b].double()
            parts.append(torch.mm(dz, s["weights"][e].double()))
            torch.mm(dz.T, x, out=grad_w[e])
    return dict(grad_x=torch.cat(parts), grad_weights=grad_w)


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "route_backward": _exact_route_backward, "matmul": _exact_matmul,
            "activation_backward": _exact_activation_backward,
            "matmul_backward": _exact_matmul_backward}[case["op"]](s)
