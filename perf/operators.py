"""The gated block and the cross entropy head: their cases, plain forms and calls.

Two operators beside the dense product C = A . B of this library, both with
their gradients:

* the gated block  h = act(x Wg^T + bg) * (x Wu^T + bu)  over one merged weight
  W = [Wg; Wu] of 2 F rows, and its backward pass (dx, dW and, with a bias,
  dbias) from dh;
* the cross entropy of the projection  l = x W^T  over a large vocabulary,
  its per-token loss and log-sum-exp, and the gradients dx and dW, without
  keeping the logits.

x, W, dh and the gradients are bfloat16 (a bias, its gradient, losses and their
gradients float32), weights are stored [out, in] as usual.
"""

import math

import torch

own = False

_GATES = ("silu", "gelu", "gelu_tanh", "relu", "sigmoid")
_IGNORE = -100
_handle = None


def _gemm():
    """The program's one handle of the library."""
    global _handle
    if _handle is None:
        import tile_partitioned_dense_amd as tg
        _handle = tg.TileGemm(torch.cuda.current_device())
    return _handle


# --------------------------------------------------------------------- cases

def _glu(name, op, T, K, F, gate, bias, out="bf16"):
    return {"name": name, "op": op, "T": T, "K": K, "F": F, "gate": gate, "bias": bias, "out": out}


def _xent(name, op, T, K, V, ignored=0.0, smoothing=0.0, z_loss=0.0, weighted=False, index="int64"):
    return {"name": name, "op": op, "T": T, "K": K, "V": V, "ignored": ignored, "smoothing": smoothing,
            "z_loss": z_loss, "weighted": weighted, "index": index}


def listed():
    return [
        # one token of one sequence through the decode workload's merged projection
        _glu("glu_decode_1", "glu", 1, 8192, 14336, "silu", False),
        # a batch of sequences decoding together, a float32 result and a bias, an odd width
        _glu("glu_decode_45", "glu", 45, 4096, 5464, "gelu_tanh", True, "fp32"),
        # a long prompt through one shard of the merged projection
        _glu("glu_prompt_8192", "glu", 8192, 8192, 3584, "gelu_tanh", False),
        # the backward pass of a small adapter-sized block: few tokens, latency counts
        _glu("glu_grad_40", "glu_grad", 40, 1024, 1368, "relu", True),
        # a packed batch of no round length, a width that fills no tile
        _glu("glu_grad_1501", "glu_grad", 1501, 4104, 2744, "gelu", True),
        # a training step's shard at full length
        _glu("glu_grad_8192", "glu_grad", 8192, 8192, 3584, "silu", False),
        # the score of one answered token against the whole vocabulary
        _xent("xent_score_1", "xent", 1, 4096, 131072),
        # the likelihood of an evaluation batch, padded rows left out
        _xent("xent_eval_1999", "xent", 1999, 2056, 50257, ignored=0.2, index="int32"),
        # fine-tuning on a handful of tokens with a small vocabulary
        _xent("xent_train_24", "xent_train", 24, 1024, 8191),
        # an ordinary step: one sequence
        _xent("xent_train_1024", "xent_train", 1024, 4096, 32000, ignored=0.1),
        # everything at once: odd sizes, padding, weights for each token, smoothing and the z term
        _xent("xent_train_3001", "xent_train", 3001, 2048, 50257, ignored=0.3, smoothing=0.1, z_loss=1e-4,
              weighted=True, index="int32"),
        # the largest: a full batch over a large vocabulary
        _xent("xent_train_8192", "xent_train", 8192, 4096, 131072, ignored=0.05),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["glu", "glu_grad", "xent", "xent_train"])
    T = _log_int(rng, 1, 8192)
    K = _log_int(rng, 128, 8192, 8)
    if op in ("glu", "glu_grad"):
        F = _log_int(rng, 64, 14336, 8)
        T = max(1, min(T, int(8192 * 8192 * 3584 / (K * F))))
        return _glu(None, op, T, K, F, rng.choice(_GATES), rng.random() < 0.5,
                    rng.choice(["bf16", "fp32"]) if op == "glu" else "bf16")
    V = _log_int(rng, 500, 131072)
    T = max(1, min(T, int(8192 * 4096 * 131072 / (K * V))))
    return _xent(None, op, T, K, V, ignored=rng.choice([0.0, 0.1, 0.5]), smoothing=rng.choice([0.0, 0.0, 0.1]),
                 z_loss=rng.choice([0.0, 0.0, 1e-3]), weighted=rng.random() < 0.4,
                 index=rng.choice(["int64", "int32"]))


def work(case):
    T, K = case["T"], case["K"]
    if case["op"] in ("glu", "glu_grad"):
        F = case["F"]
        bias = 8 * F if case["bias"] else 0
        product = 4 * T * F * K  # both projections
        if case["op"] == "glu":
            return {"bytes": 2 * T * K + 4 * F * K + bias + T * F * (4 if case["out"] == "fp32" else 2),
                    "flops": product}
        # x, W, dh read; dx, dW, dbias written; the projections once and a product for each gradient
        return {"bytes": 4 * T * K + 8 * F * K + 2 * T * F + 2 * bias, "flops": 3 * product}
    V = case["V"]
    rows = T * ((8 if case["index"] == "int64" else 4) + 8)  # target, loss, log-sum-exp
    if case["op"] == "xent":
        return {"bytes": 2 * T * K + 2 * V * K + rows, "flops": 2 * T * V * K}
    return {"bytes": 4 * T * K + 4 * V * K + rows + 4 * T, "flops": 6 * T * V * K}


# -------------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(rows, cols, scale):
        return torch.randn(rows, cols, generator=gen, device="cuda").mul_(scale).to(torch.bfloat16)

    T, K = case["T"], case["K"]
    state = {"case": case, "x": normal(T, K, 1.0)}  # normalised activations
    if case["op"] in ("glu", "glu_grad"):
        F = case["F"]
        state["w"] = normal(2 * F, K, K ** -0.5)
        state["bias"] = torch.randn(2 * F, generator=gen, device="cuda") * 0.2 if case["bias"] else None
        if case["op"] == "glu_grad":
            state["dh"] = normal(T, F, 1.0 / T)
        return state
    V = case["V"]
    state["w"] = normal(V, K, 2.0 * K ** -0.5)  # logits of standard deviation 2
    target = torch.randint(0, V, (T,), generator=gen, device="cuda")
    keep = torch.rand(T, generator=gen, device="cuda") >= case["ignored"]
    target = torch.where(keep, target, _IGNORE)
    state["target"] = target.to(torch.int32) if case["index"] == "int32" else target
    # the loss is the mean over the rows that count, with a weight for each token or without
    weight = torch.rand(T, generator=gen, device="cuda") + 0.5 if case["weighted"] else torch.ones(T, device="cuda")
    weight = torch.where(keep, weight, 0.0)
    state["dloss"] = weight / weight.sum().clamp(min=1e-6)
    return state


# --------------------------------------------------------------- plain forms

def _gate(z, gate):
    """act(z) and its derivative."""
    if gate == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return z * s, s * (1.0 + z * (1.0 - s))
    if gate == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s, s * (1.0 - s)
    if gate == "relu":
        on = (z > 0).to(z.dtype)
        return z * on, on
    if gate == "gelu":
        p = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return z * p, p + z * torch.exp(-0.5 * z * z) * (0.5 * math.sqrt(2.0 / math.pi))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)


def _plain_glu(s, case):
    z = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"]
    g, u = z[:, :case["F"]], z[:, case["F"]:]
    act, slope = _gate(g, case["gate"])
    if case["op"] == "glu":
        return {"h": (act * u).to(torch.float32 if case["out"] == "fp32" else torch.bfloat16)}
    dh = s["dh"].float()
    dz = torch.cat([dh * u * slope, dh * act], dim=1)
    out = {"dx": (dz @ s["w"].float()).to(torch.bfloat16), "dw": (dz.t() @ s["x"].float()).to(torch.bfloat16)}
    if s["bias"] is not None:
        out["dbias"] = dz.sum(0, dtype=torch.float64).float()
    return out


def _plain_xent(s, case):
    x, w, target = s["x"].float(), s["w"].float(), s["target"].long()
    logits = x @ w.t()
    top = logits.max(dim=1, keepdim=True).values
    lse = top[:, 0] + torch.log(torch.exp(logits - top).sum(dim=1))
    keep = target != _IGNORE
    at = target.clamp(min=0)
    eps, z = case["smoothing"], case["z_loss"]
    loss = lse - (1.0 - eps) * logits.gather(1, at[:, None])[:, 0] + z * lse * lse
    if eps:
        loss = loss - eps * logits.mean(dim=1)
    out = {"loss": torch.where(keep, loss, 0.0), "lse": lse}
    if case["op"] == "xent":
        return out
    scale = torch.where(keep, s["dloss"], 0.0)[:, None]
    d = torch.exp(logits - lse[:, None]) * (scale * (1.0 + 2.0 * z * lse[:, None])) - scale * (eps / case["V"])
    d.scatter_add_(1, at[:, None], -(1.0 - eps) * scale)
    return out | {"dx": (d @ w).to(torch.bfloat16), "dw": (d.t() @ x).to(torch.bfloat16)}


# ----------------------------------------------------------------- the calls

def _own_glu(s, case):
    import tile_partitioned_dense_amd as tg
    gemm, x, w = _gemm(), s["x"], s["w"]
    gate = tg.Gate[case["gate"].upper()]
    if case["op"] == "glu":
        h = torch.empty(case["T"], case["F"], device="cuda",
                        dtype=torch.float32 if case["out"] == "fp32" else torch.bfloat16)
        gemm.glu(x, w.t(), h, gate=gate, bias=s["bias"])
        return {"h": h}
    out = {"dx": torch.empty_like(x), "dw": torch.empty_like(w)}
    if s["bias"] is not None:
        out["dbias"] = torch.empty_like(s["bias"])
    gemm.glu_backward(x, w.t(), s["dh"], dA=out["dx"], dB=out["dw"].t(), gate=gate, bias=s["bias"],
                      dbias=out.get("dbias"))
    return out


def _own_xent(s, case):
    gemm, x, w = _gemm(), s["x"], s["w"]
    out = {"loss": torch.empty(case["T"], device="cuda"), "lse": torch.empty(case["T"], device="cuda")}
    options = {"ignore_index": _IGNORE, "label_smoothing": case["smoothing"], "z_loss": case["z_loss"]}
    gemm.xent(x, w.t(), s["target"], out["loss"], out["lse"], **options)
    if case["op"] == "xent":
        return out
    out |= {"dx": torch.empty_like(x), "dw": torch.empty_like(w)}
    gemm.xent_backward(x, w.t(), s["target"], out["lse"], s["dloss"], dA=out["dx"], dB=out["dw"].t(), **options)
    return out


def run(state):
    case = state["case"]
    if case["op"] in ("glu", "glu_grad"):
        return _own_glu(state, case) if own else _plain_glu(state, case)
    return _own_xent(state, case) if own else _plain_xent(state, case)


# ---------------------------------------------------------------- in 64 bits

def _slope64(z, gate, act):
    """The derivative of act at z in 64 bits, as autograd finds it."""
    z = z.detach().requires_grad_(True)
    with torch.enable_grad():
        return torch.autograd.grad(act(z).sum(), z)[0]


def exact(case, seed):
    s = prepare(case, seed)
    x, w = s["x"].double(), s["w"].double()
    if case["op"] in ("glu", "glu_grad"):
        F = case["F"]
        act = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "relu": torch.relu,
               "sigmoid": torch.sigmoid,
               "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[case["gate"]]
        b = s["bias"].double() if s["bias"] is not None else torch.zeros(2 * F, device="cuda", dtype=torch.float64)
        gate = torch.mm(x, w[:F].t()) + b[:F]
        up = torch.mm(x, w[F:].t()) + b[F:]
        if case["op"] == "glu":
            return {"h": act(gate) * up}
        dh = s["dh"].double()
        dgate, dup = dh * up * _slope64(gate, case["gate"], act), dh * act(gate)
        out = {"dx": dgate @ w[:F] + dup @ w[F:], "dw": torch.cat([dgate.t() @ x, dup.t() @ x])}
        if s["bias"] is not None:
            out["dbias"] = torch.cat([dgate.sum(0), dup.sum(0)])
        return out
    V, eps, z = case["V"], case["smoothing"], case["z_loss"]
    target = s["target"].long()
    keep = (target != _IGNORE).double()
    at = target.clamp(min=0)
    pieces = [(a, min(V, a + 16384)) for a in range(0, V, 16384)]
    lse = torch.full((case["T"],), -math.inf, device="cuda", dtype=torch.float64)
    total = torch.zeros_like(lse)
    for a, b in pieces:
        l = x @ w[a:b].t()
        lse = torch.logaddexp(lse, torch.logsumexp(l, dim=1))
        total += l.sum(dim=1)
    hit = (x * w[at]).sum(dim=1)
    out = {"loss": keep * (lse - (1 - eps) * hit - eps * total / V + z * lse ** 2), "lse": lse}
    if case["op"] == "xent":
        return out
    scale = keep * s["dloss"].double()
    dx, dw = torch.zeros_like(x), torch.empty_like(w)
    rows = torch.arange(case["T"], device="cuda")
    for a, b in pieces:
        p = torch.exp(x @ w[a:b].t() - lse[:, None]) * (1 + 2 * z * lse)[:, None] - eps / V
        inside = (at >= a) & (at < b)
        p[rows[inside], at[inside] - a] -= 1 - eps
        p *= scale[:, None]
        dx += p @ w[a:b]
        dw[a:b] = p.t() @ x
    return out | {"dx": dx, "dw": dw}
