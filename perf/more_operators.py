"""8-bit products with block scales, routing to experts and the experts' products: cases, plain forms and calls.

Operators around the dense product C = A . B^T of this library with E4M3
operands and float32 scales (one for 128 consecutive values of a row of A, one
for each 128 x 128 block of B):

* quantize: bfloat16 values to E4M3 and scales, by rows or by blocks; rows may
  be gathered, and a gated block's act(gate) * up formed on the way;
* the product itself, with a bias and an activation;
* routing: from a router's logits to each token's experts and their weights,
  and to the order of the tokens by expert; and the gradient of the weights;
* the experts' products over rows sorted by expert;
* combine: each token's weighted sum of its experts' rows.

A scale of a row is kept with the rows next to each other (the scales of one
128-value block of all rows are consecutive), weights are stored [out, in].
"""

import math

import torch

own = False

_GATES = ("silu", "gelu", "gelu_tanh", "relu", "sigmoid")
_FP8 = torch.float8_e4m3fn
_TOP = 448.0           # largest E4M3 value
_LEAST = 2.0 ** -100   # largest magnitude of a block below which it is taken as that
_handle = None


def _gemm():
    """The program's one handle of the library."""
    global _handle
    if _handle is None:
        import tile_partitioned_dense_amd as tg
        _handle = tg.TileGemm(torch.cuda.current_device())
    return _handle


# --------------------------------------------------------------------- cases

def _quant(name, M, K, form="rows", gate="", rows=0):
    """rows: gathered from that many (0: not gathered)."""
    return {"name": name, "op": "quantize", "M": M, "K": K, "form": form, "gate": gate, "rows": rows}


def _fp8(name, M, N, K, out="bf16", bias=False, act=""):
    return {"name": name, "op": "fp8", "M": M, "N": N, "K": K, "out": out, "bias": bias, "act": act}


def _route(name, op, T, E, k, score, bias=False, groups=1, top_groups=1, group_top=2, renorm=True, scale=1.0,
           logits="fp32", absent=0.0):
    """absent: share of the places that hold no expert of this device."""
    return {"name": name, "op": op, "T": T, "E": E, "k": k, "score": score, "bias": bias, "groups": groups,
            "top_groups": top_groups, "group_top": group_top, "renorm": renorm, "scale": scale, "logits": logits,
            "absent": absent}


def _experts(name, T, k, E, N, K, out="bf16"):
    return {"name": name, "op": "experts", "T": T, "k": k, "E": E, "N": N, "K": K, "out": out}


def _combine(name, T, k, N, absent=0.0, out="bf16"):
    return {"name": name, "op": "combine", "T": T, "k": k, "N": N, "absent": absent, "out": out}


def listed():
    return [
        # one token of one sequence on its way into a projection: latency
        _quant("quant_token_1", 1, 8192),
        # a prompt's merged gate+up projection on its way into the down projection
        _quant("quant_gated_8192", 8192, 3584, gate="silu"),
        # the decode workload's batch through the merged projection: the weights' stream
        _fp8("fp8_decode_16", 16, 28672, 8192),
        # a packed batch of no round length, a width that fills no tile, a K that ends inside a block
        _fp8("fp8_batch_1999", 1999, 5464, 4112, out="fp32", bias=True, act="silu"),
        # a long prompt through one shard of the merged projection
        _fp8("fp8_prompt_8192", 8192, 7168, 8192),
        # a few sequences decoding together, softmax scores
        _route("route_decode_8", "route", 8, 64, 4, "softmax"),
        # a long prompt: sigmoid scores, a bias for balance, groups, renormalised and scaled weights
        _route("route_prompt_8191", "route", 8191, 256, 8, "sigmoid", bias=True, groups=8, top_groups=4, scale=2.5,
               absent=0.25),
        # a training step's gradient of the router's logits
        _route("route_grad_4096", "route_grad", 4096, 160, 6, "softmax", renorm=False, scale=16.0, logits="bf16"),
        # a batch of sequences decoding together: most experts see a token or two, some none
        _experts("experts_decode_24", 24, 8, 64, 4096, 2048),
        # a prompt of no round length over few experts: from one full tile to many
        _experts("experts_prompt_4099", 4099, 4, 16, 7168, 2048),
        # the decoding batch's rows back to its tokens
        _combine("combine_decode_24", 24, 8, 2048),
        # a long prompt's, some of whose experts are on other devices
        _combine("combine_prompt_8191", 8191, 8, 4096, absent=0.25),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["quantize", "fp8", "fp8", "route", "route", "route_grad", "experts", "experts", "combine"])
    most = 8192 * 7168 * 8192  # products of the largest listed case
    if op == "quantize":
        form = rng.choice(["rows", "rows", "blocks"])
        M, K = _log_int(rng, 1, 16384), _log_int(rng, 16, 8192, 16)
        gate = rng.choice(["", *_GATES]) if form == "rows" else ""
        return _quant(None, M, K, form, gate, _log_int(rng, 1, 16384) if form == "rows" and rng.random() < 0.4 else 0)
    if op == "fp8":
        N, K = _log_int(rng, 1, 28672), _log_int(rng, 16, 8192, 16)
        M = max(1, min(_log_int(rng, 1, 8192), most // (N * K)))
        return _fp8(None, M, N, K, rng.choice(["bf16", "fp32"]), rng.random() < 0.4,
                    rng.choice(["", "", "relu", "sigmoid", "tanh", "silu"]))
    if op == "combine":
        return _combine(None, _log_int(rng, 1, 8192), rng.randint(1, 8), _log_int(rng, 8, 4096, 8),
                        rng.choice([0.0, 0.3]), rng.choice(["bf16", "fp32"]))
    if op == "experts":
        E = _log_int(rng, 1, 128)
        k = rng.randint(1, min(8, E))
        N, K = _log_int(rng, 16, 7168), _log_int(rng, 16, 4096, 16)
        # the experts' weights, and each token's products, within the largest listed case's
        E = max(k, min(E, 64 * 4096 * 2048 // (N * K)))
        T = max(1, min(_log_int(rng, 1, 8192), most // (4 * N * K * k)))
        return _experts(None, T, k, E, N, K, rng.choice(["bf16", "fp32"]))
    groups = rng.choice([1, 1, 2, 4, 8])
    E = groups * _log_int(rng, 2, 512 // groups)
    top_groups = rng.randint(1, groups)
    k = rng.randint(1, min(16, top_groups * (E // groups)))
    return _route(None, op, _log_int(rng, 1, 8192), E, k, rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5, groups,
                  top_groups, rng.choice([1, 2]), rng.random() < 0.6, rng.choice([1.0, 2.5]),
                  rng.choice(["fp32", "bf16"]), rng.choice([0.0, 0.25]) if op == "route" else 0.0)


def _blocks(n):
    return -(-n // 128)


def work(case):
    op = case["op"]
    if op == "quantize":
        M, K = case["M"], case["K"]
        scales = M * _blocks(K) if case["form"] == "rows" else _blocks(M) * _blocks(K)
        return {"bytes": M * K * (5 if case["gate"] else 3) + 4 * scales + (4 * M if case["rows"] else 0), "flops": 0}
    if op in ("fp8", "experts"):
        N, K = case["N"], case["K"]
        M = case["M"] if op == "fp8" else case["T"] * case["k"]
        # experts that have rows: at least as many as a token has, at most all
        weights = 1 if op == "fp8" else min(case["E"], M)
        return {"bytes": M * K + 4 * M * _blocks(K) + weights * (N * K + 4 * _blocks(N) * _blocks(K))
                + M * N * (4 if case["out"] == "fp32" else 2) + (4 * N if op == "fp8" and case["bias"] else 0),
                "flops": 2 * M * N * K}
    T, k = case["T"], case["k"]
    if op == "combine":
        live = int(T * k * (1 - case["absent"]))
        return {"bytes": live * case["N"] * 2 + 8 * T * k + T * case["N"] * (4 if case["out"] == "fp32" else 2),
                "flops": 2 * live * case["N"]}
    E, size = case["E"], 4 if case["logits"] == "fp32" else 2
    if op == "route":  # logits; ids, weights, rows, places, offsets
        return {"bytes": T * E * size + 16 * T * k + 4 * (E + 1), "flops": 0}
    return {"bytes": 2 * T * E * size + 8 * T * k, "flops": 0}


# -------------------------------------------------------------------- inputs

def _popular(gen, T, E, k):
    """k different experts for each of T tokens, some asked for more often than others."""
    want = torch.rand(T, E, generator=gen, device="cuda").log().neg().log().neg()
    want += torch.randn(E, generator=gen, device="cuda")
    return want.topk(k, dim=1).indices.to(torch.int32)


def _codes(gen, scale_shape, *shape):
    """E4M3 codes of normal values and scales, as quantize leaves them."""
    q = torch.randn(*shape, generator=gen, device="cuda").mul_(100.0).clamp_(-_TOP, _TOP).to(_FP8)
    return q, torch.rand(*scale_shape, generator=gen, device="cuda").add_(0.5).mul_(0.01)


def _row_scales(M, K, make=torch.empty):
    """[M, blocks of K], rows next to each other, a block's first one at a multiple of 4."""
    return make(_blocks(K), (M + 3) // 4 * 4, device="cuda").t()[:M]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, state = case["op"], {"case": case}
    if op == "quantize":
        M, K = case["M"], case["K"]
        have = case["rows"] or M
        # activations have rows and columns that are larger than others
        x = torch.randn(have, K * (2 if case["gate"] else 1), generator=gen, device="cuda")
        x *= torch.randn(have, 1, generator=gen, device="cuda").exp_()
        state["x"] = x.to(torch.bfloat16)
        if case["rows"]:
            state["rows"] = torch.randint(0, have, (M,), generator=gen, device="cuda", dtype=torch.int32)
        return state
    if op == "fp8":
        M, N, K = case["M"], case["N"], case["K"]
        state["a"], scale = _codes(gen, (_blocks(K), M), M, K)
        state["a_scale"] = _row_scales(M, K)
        state["a_scale"].copy_(scale.t())
        state["b"], state["b_scale"] = _codes(gen, (_blocks(N), _blocks(K)), N, K)
        state["bias"] = torch.randn(N, generator=gen, device="cuda") if case["bias"] else None
        return state
    if op == "experts":
        T, k, E, N, K = (case[n] for n in ("T", "k", "E", "N", "K"))
        count = torch.bincount(_popular(gen, T, E, k).reshape(-1), minlength=E)
        state["offsets"] = torch.cat([count.new_zeros(1), count.cumsum(0)]).to(torch.int32)
        state["most"] = int(count.max())  # rows of the largest expert
        state["a"], scale = _codes(gen, (_blocks(K), T * k), T * k, K)
        state["a_scale"] = _row_scales(T * k, K)
        state["a_scale"].copy_(scale.t())
        state["b"], state["b_scale"] = _codes(gen, (E, _blocks(N), _blocks(K)), E, N, K)
        return state
    T, k = case["T"], case["k"]
    if op == "combine":
        here = torch.rand(T * k, generator=gen, device="cuda") >= case["absent"]
        order = torch.rand(T * k, generator=gen, device="cuda").argsort()
        rank = torch.where(here[order], here[order].cumsum(0) - 1, -1)
        state["places"] = torch.empty_like(order).scatter_(0, order, rank).to(torch.int32).view(T, k)
        state["z"] = torch.randn(T * k, case["N"], generator=gen, device="cuda").to(torch.bfloat16)
        state["weights"] = torch.rand(T, k, generator=gen, device="cuda").add_(0.1).div_(k)
        return state
    E = case["E"]
    logits = torch.randn(T, E, generator=gen, device="cuda") * 2.0
    state["logits"] = logits.to(torch.bfloat16 if case["logits"] == "bf16" else torch.float32)
    state["bias"] = torch.randn(E, generator=gen, device="cuda") * 0.05 if case["bias"] else None
    if op == "route_grad":
        state["ids"] = _popular(gen, T, E, k)
        state["dweights"] = torch.randn(T, k, generator=gen, device="cuda")
        return state
    # the experts of this device: ids below `first` are of another one
    state["first"] = int(E * case["absent"])
    return state


# --------------------------------------------------------------- plain forms

def _act(z, name):
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-z))
    if name == "relu":
        return torch.where(z > 0, z, 0.0)
    if name == "tanh":
        return torch.tanh(z)
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _padded(x, rows, cols):
    """x with zeros up to whole blocks of rows x cols."""
    M, K = x.shape
    out = x.new_zeros(-(-M // rows) * rows, -(-K // cols) * cols)
    out[:M, :K] = x
    return out


def _plain_quantize(s, case):
    M, K = case["M"], case["K"]
    x = s["x"]
    if case["rows"]:
        x = x[s["rows"].long()]
    x = x.float()
    if case["gate"]:
        x = _act(x[:, :K], case["gate"]) * x[:, K:]
    high = 1 if case["form"] == "rows" else 128
    x = _padded(x, high, 128)
    b = x.view(x.shape[0] // high, high, x.shape[1] // 128, 128)
    top = b.abs().amax(dim=(1, 3)).clamp(min=_LEAST)
    q = (b * (_TOP / top)[:, None, :, None]).clamp(-_TOP, _TOP).to(_FP8).view(x.shape)[:M, :K]
    return {"q": q.contiguous(), "scale": top / _TOP}


def _wide(q, scale, rows):
    """The float32 values of codes [.., M, K] with a scale for `rows` x 128 of them."""
    M, K = q.shape[-2:]
    scale = scale.repeat_interleave(128, dim=-1)[..., :K]
    if rows > 1:
        scale = scale.repeat_interleave(rows, dim=-2)[..., :M, :]
    return q.float() * scale


def _plain_fp8(s, case):
    c = _wide(s["a"], s["a_scale"], 1) @ _wide(s["b"], s["b_scale"], 128).t()
    if s["bias"] is not None:
        c = c + s["bias"]
    return {"c": _act(c, case["act"]).to(torch.float32 if case["out"] == "fp32" else torch.bfloat16)}


def _plain_experts(s, case):
    M, offsets = case["T"] * case["k"], s["offsets"].long()
    # each expert's rows, as many for all as the largest has
    at = (offsets[:-1, None] + torch.arange(s["most"], device="cuda")).clamp(max=M - 1)
    c = torch.bmm(_wide(s["a"], s["a_scale"], 1)[at], _wide(s["b"], s["b_scale"], 128).transpose(1, 2))
    row = torch.arange(M, device="cuda")
    expert = torch.searchsorted(offsets, row, right=True) - 1
    return {"c": c[expert, row - offsets[expert]].to(torch.float32 if case["out"] == "fp32" else torch.bfloat16)}


def _scores(logits, kind):
    """Scores in 64 bits: which expert is chosen hangs on their order."""
    l = logits.double()
    if kind == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _weights(scores, case):
    if case["renorm"]:
        scores = scores / scores.sum(dim=1, keepdim=True)
    return scores * case["scale"]


def _plain_route(s, case):
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    scores = _scores(s["logits"], case["score"])
    value = scores if s["bias"] is None else scores + s["bias"].double()
    if G > 1:
        by_group = value.view(T, G, E // G)
        best = by_group.sort(dim=2, descending=True).values[:, :, :case["group_top"]].sum(dim=2)
        groups = best.sort(dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        open_ = torch.zeros(T, G, dtype=torch.bool, device="cuda").scatter_(1, groups, True)
        value = torch.where(open_[:, :, None], by_group, -math.inf).view(T, E)
    ids = value.sort(dim=1, descending=True, stable=True).indices[:, :k]
    weights = _weights(scores.gather(1, ids), case).float()
    # the tokens in the order of their experts, those of this device
    flat = ids.reshape(-1) - s["first"]
    here = E - s["first"]
    key = torch.where(flat >= 0, flat, here)
    order = key.sort(stable=True).indices
    offsets = torch.cat([key.new_zeros(1), torch.bincount(key, minlength=here + 1)[:here].cumsum(0)])
    at = torch.arange(T * k, device="cuda")
    live = at < offsets[-1]
    places = torch.empty_like(order).scatter_(0, order, torch.where(live, at, -1))
    i32 = torch.int32
    return {"ids": ids.to(i32), "weights": weights, "offsets": offsets.to(i32),
            "rows": torch.where(live, order // k, -1).to(i32), "places": places.to(i32).view(T, k)}


def _plain_route_grad(s, case):
    scores, ids = _scores(s["logits"], case["score"]), s["ids"].long()
    chosen, d = scores.gather(1, ids), s["dweights"].double() * case["scale"]
    if case["renorm"]:
        total = chosen.sum(dim=1, keepdim=True)
        d = (d - (d * chosen).sum(dim=1, keepdim=True) / total) / total
    if case["score"] == "sigmoid":
        dl = torch.zeros_like(scores).scatter_(1, ids, d * chosen * (1.0 - chosen))
    else:
        dl = torch.zeros_like(scores).scatter_(1, ids, d * chosen) - scores * (d * chosen).sum(dim=1, keepdim=True)
    return {"dlogits": dl.to(s["logits"].dtype)}


def _plain_combine(s, case):
    places = s["places"].long()
    z = s["z"][places.clamp(min=0)].float()
    w = torch.where(places >= 0, s["weights"], 0.0)
    return {"y": (z * w[:, :, None]).sum(dim=1).to(torch.float32 if case["out"] == "fp32" else torch.bfloat16)}


_PLAIN = {"quantize": _plain_quantize, "fp8": _plain_fp8, "experts": _plain_experts, "route": _plain_route,
          "route_grad": _plain_route_grad, "combine": _plain_combine}


# ----------------------------------------------------------------- the calls

def _out(case, M, N):
    """Rows a whole number of 16 bytes apart, as the library's products take them."""
    out = torch.empty(M, (N + 7) // 8 * 8, device="cuda",
                      dtype=torch.float32 if case["out"] == "fp32" else torch.bfloat16)
    return out[:, :N]


def _own_quantize(s, case):
    import tile_partitioned_dense_amd as tg
    M, K = case["M"], case["K"]
    q = torch.empty(M, K, device="cuda", dtype=_FP8)
    if case["form"] == "blocks":
        scale = torch.empty(_blocks(M), _blocks(K), device="cuda")
        _gemm().quantize(s["x"], q, scale, form=tg.Quant.BLOCKS)
    else:
        scale = _row_scales(M, K)
        _gemm().quantize(s["x"], q, scale, gate=tg.Gate[case["gate"].upper()] if case["gate"] else None,
                         rows=s.get("rows"))
    return {"q": q, "scale": scale}


def _own_fp8(s, case):
    import tile_partitioned_dense_amd as tg
    c = _out(case, case["M"], case["N"])
    _gemm().fp8(s["a"], s["b"], c, s["a_scale"], s["b_scale"], bias=s["bias"],
                act=tg.Act[case["act"].upper()] if case["act"] else None)
    return {"c": c}


def _own_experts(s, case):
    c = _out(case, case["T"] * case["k"], case["N"])
    _gemm().fp8_experts(s["a"], s["b"], c, s["a_scale"], s["b_scale"], s["offsets"])
    return {"c": c}


def _own_route(s, case):
    import tile_partitioned_dense_amd as tg
    T, E, k = case["T"], case["E"], case["k"]
    ids, weights, rows, places = torch.empty(4, T, k, device="cuda", dtype=torch.int32).unbind()
    weights, rows = weights.view(torch.float32), rows.view(-1)
    offsets = torch.empty(E - s["first"] + 1, device="cuda", dtype=torch.int32)
    _gemm().route(s["logits"], ids, weights, score=tg.Score[case["score"].upper()], bias=s["bias"],
                  groups=case["groups"], top_groups=case["top_groups"], group_top=case["group_top"],
                  renormalize=case["renorm"], scale=case["scale"])
    _gemm().place(ids, offsets, rows, places, first=s["first"])
    return {"ids": ids, "weights": weights, "offsets": offsets, "rows": rows, "places": places}


def _own_route_grad(s, case):
    import tile_partitioned_dense_amd as tg
    dlogits = torch.empty_like(s["logits"])
    _gemm().route_backward(s["logits"], s["ids"], s["dweights"], dlogits, score=tg.Score[case["score"].upper()],
                           renormalize=case["renorm"], scale=case["scale"])
    return {"dlogits": dlogits}


def _own_combine(s, case):
    y = _out(case, case["T"], case["N"])
    _gemm().combine(s["z"], s["places"], s["weights"], y)
    return {"y": y}


_OWN = {"quantize": _own_quantize, "fp8": _own_fp8, "experts": _own_experts, "route": _own_route,
        "route_grad": _own_route_grad, "combine": _own_combine}


def run(state):
    case = state["case"]
    if own:
        return _OWN[case["op"]](state, case)
    return _PLAIN[case["op"]](state, case)


# ---------------------------------------------------------------- in 64 bits

def _exact_act(z, name):
    f = torch.nn.functional
    return {"": lambda v: v, "silu": f.silu, "sigmoid": torch.sigmoid, "relu": torch.relu, "tanh": torch.tanh,
            "gelu": f.gelu, "gelu_tanh": lambda v: f.gelu(v, approximate="tanh")}[name](z)


def _exact_scales(scale, high, M, K):
    return scale.double().repeat_interleave(high, 0)[:M].repeat_interleave(128, 1)[:, :K]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        M, K = case["M"], case["K"]
        x = s["x"].double()
        if case["rows"]:
            x = torch.index_select(x, 0, s["rows"].long())
        if case["gate"]:
            x = _exact_act(x[:, :K], case["gate"]) * x[:, K:]
        high = 1 if case["form"] == "rows" else 128
        size = torch.nn.functional.pad(x.abs(), (0, -K % 128, 0, -M % high))
        top = torch.nn.functional.max_pool2d(size[None], (high, 128), (high, 128))[0].clamp(min=_LEAST)
        return {"q": x / _exact_scales(top / _TOP, high, M, K), "scale": top / _TOP}
    if op == "fp8":
        M, N, K = case["M"], case["N"], case["K"]
        a = s["a"].double() * _exact_scales(s["a_scale"], 1, M, K)
        b = s["b"].double() * _exact_scales(s["b_scale"], 128, N, K)
        c = torch.mm(a, b.t())
        if s["bias"] is not None:
            c += s["bias"].double()
        return {"c": _exact_act(c, case["act"])}
    if op == "experts":
        M, N, K = case["T"] * case["k"], case["N"], case["K"]
        a = s["a"].double() * _exact_scales(s["a_scale"], 1, M, K)
        parts, ends = [], s["offsets"].tolist()
        for e in range(case["E"]):
            if ends[e + 1] > ends[e]:
                b = s["b"][e].double() * _exact_scales(s["b_scale"][e], 128, N, K)
                parts.append(torch.mm(a[ends[e]:ends[e + 1]], b.t()))
        return {"c": torch.cat(parts)}
    if op == "combine":
        y = torch.zeros(case["T"], case["N"], device="cuda", dtype=torch.float64)
        for j in range(case["k"]):
            at = s["places"][:, j].long()
            on = (at >= 0).nonzero()[:, 0]
            y[on] += s["weights"][on, j, None].double() * s["z"][at[on]].double()
        return {"y": y}
    logits = s["logits"].double()
    p = torch.softmax(logits, 1) if case["score"] == "softmax" else torch.sigmoid(logits)
    if op == "route_grad":
        leaf = logits.clone().requires_grad_(True)
        with torch.enable_grad():
            q = torch.softmax(leaf, 1) if case["score"] == "softmax" else torch.sigmoid(leaf)
            w = q.gather(1, s["ids"].long())
            w = (w / w.sum(1, keepdim=True) if case["renorm"] else w) * case["scale"]
            return {"dlogits": torch.autograd.grad((w * s["dweights"].double()).sum(), leaf)[0]}
    G, E = case["groups"], case["E"]
    v = p if s["bias"] is None else p + s["bias"].double()
    if G > 1:
        best = v.view(-1, G, E // G).topk(min(case["group_top"], E // G), dim=2).values.sum(2)
        worst = best.topk(case["top_groups"], dim=1).values[:, -1:]
        v = v.masked_fill((best < worst).repeat_interleave(E // G, 1), -math.inf)
    w = p.gather(1, v.topk(case["k"], dim=1).indices)
    w = w / w.sum(1, keepdim=True) if case["renorm"] else w
    return {"ids": None, "weights": w * case["scale"], "offsets": None, "rows": None, "places": None}
