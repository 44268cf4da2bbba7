"""Plain 64-bit references and error bounds of the E4M3 products with block
scales, of the quantization and of the routing to experts. They share no code
with the library; everything runs on the CPU in float64.

Bounds. The E4M3 matrix instruction adds products in runs of 8 consecutive
values of K, each run cut below 2^-13 of its largest product's binade (the
device model of oracle/mx.py): at most 7 * 2^(E - 13) a run, times the block's
scales. What is added in fp32 beside that is within TAU = 1e-5 of
D = sum |a| |b|. fp32 results use the bf16 instruction: TAU alone. A rounding to
bf16 is off by at most HALF of the value, one to E4M3 by 2^-4 of it or by half
of the smallest subnormal, 2^-10; fp32 elementwise evaluation by EVAL."""

from __future__ import annotations

import torch

TAU, HALF, EVAL = 1e-5, 2.0 ** -8, 2.0 ** -18
FP8 = torch.float8_e4m3fn
ACTS = {"NONE": lambda v: v, "RELU": lambda v: v.clamp(min=0), "SIGMOID": torch.sigmoid, "TANH": torch.tanh,
        "SILU": torch.nn.functional.silu}
LIP = {"NONE": 1.0, "RELU": 1.0, "SIGMOID": 0.25, "TANH": 1.0, "SILU": 1.1}


def blocks(n):
    return -(-n // 128)


def codes(gen, *shape):
    """E4M3 codes as quantization leaves them: normal values, some blocks at full range."""
    return (torch.randn(*shape, generator=gen) * 100).clamp(-448, 448).to(FP8)


def row_scales(M, K, device="cpu", pad=0):
    """[M, blocks of K], rows next to each other, `pad` values behind them."""
    return torch.full((blocks(K), M + pad), float("nan"), device=device).t()[:M]


def widen(q, s, high):
    """Codes [M, K] times their scales, in 64 bits."""
    M, K = q.shape
    s = s.double().repeat_interleave(128, 1)[:, :K]
    return q.double() * (s.repeat_interleave(high, 0)[:M] if high > 1 else s)


def product(a, sa, b, sb, bias=None, act="NONE", fp32=False):
    """The result and its error bound."""
    x, y = widen(a, sa, 1), widen(b, sb, 128)
    c = x @ y.T
    err = TAU * (x.abs() @ y.abs().T)
    if not fp32:
        K = x.shape[1]
        pad = (0, -K % 8)
        xa = torch.nn.functional.pad(x.abs(), pad).view(x.shape[0], 1, -1, 8)
        ya = torch.nn.functional.pad(y.abs(), pad).view(1, y.shape[0], -1, 8)
        for i in range(0, x.shape[0], 16):
            top = (xa[i:i + 16] * ya).amax(3)
            # (the binade of the scaled product may be one above the codes' own)
            err[i:i + 16] += 7 * 2.0 ** -13 * top.sum(2)
    if bias is not None:
        c = c + bias.double()
        err = err + 2.0 ** -23 * c.abs()
    y = ACTS[act](c)
    if act != "NONE":
        err = LIP[act] * err + EVAL * y.abs() + 2.0 ** -22
    return y, err


def close(got, want, err, bf16, what):
    got = got.double().cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if bf16:
        err = err + HALF * (want.abs() + err) + 2.0 ** -133
    bad = ~((got - want).abs() <= err) & ~(got.isnan() & want.isnan())
    n = int(bad.sum())
    if n:
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {n} of {bad.numel()} off, first at {i}: got {got[i]}, want {want[i]}, "
                             f"bound {err[i] if err.dim() else err}")


def quantize(x, high):
    """fp32 x to codes and scales by the documented fp32 formula."""
    M, K = x.shape
    p = torch.nn.functional.pad(x, (0, -K % 128, 0, -M % high))
    b = p.view(p.shape[0] // high, high, -1, 128)
    top = b.abs().amax((1, 3)).clamp(min=2.0 ** -100)
    q = (b * (torch.tensor(448.0) / top)[:, None, :, None]).view(p.shape)[:M, :K]
    return q.to(FP8), top / 448.0


def scores(logits, kind):
    l = logits.double()
    l = torch.where(l.isnan(), float("-inf"), l)
    if kind == "SIGMOID":
        return torch.sigmoid(l)
    m = l.amax(1, keepdim=True)
    e = torch.where(l == m, 1.0, torch.exp(l - m))
    e = torch.where(m == float("-inf"), 0.0, e)
    e = torch.where((m == float("inf")) & (l != m), 0.0, e)
    total = e.sum(1, keepdim=True)
    return torch.where(total > 0, e / total, 0.0)


def route(logits, k, kind, bias=None, groups=1, top_groups=1, group_top=2, renorm=True, scale=1.0):
    """ids and weights, one token at a time."""
    s = scores(logits, kind)
    T, E = s.shape
    v = s if bias is None else s + bias.double()
    v = torch.where(v.isnan(), float("-inf"), v)
    ids, size = torch.empty(T, k, dtype=torch.int64), E // groups
    for t in range(T):
        row = v[t].tolist()
        best = []
        for g in range(groups):
            top = sorted(row[g * size:(g + 1) * size], reverse=True)[:group_top]
            value = sum(top)
            best.append(value if value == value else float("-inf"))
        chosen = sorted(range(groups), key=lambda g: (-best[g], g))[:top_groups]
        pool = [e for e in range(E) if groups == 1 or e // size in chosen]
        ids[t] = torch.tensor(sorted(pool, key=lambda e: (-row[e], e))[:k])
    w = s.gather(1, ids)
    if renorm:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return ids, w * scale


def route_grad(logits, ids, dw, kind, renorm, scale):
    """The formula, in 64 bits; ids outside the experts count for nothing."""
    s = scores(logits, kind)
    T, E = s.shape
    ids = ids.long()
    on = (ids >= 0) & (ids < E)
    at = torch.where(on, ids, 0)
    p = torch.where(on, s.gather(1, at), 0.0)
    d = torch.where(on, dw.double() * scale, 0.0)
    if renorm:
        total = p.sum(1, keepdim=True)
        d = torch.where(on & (total > 0), (d - (d * p).sum(1, keepdim=True) / total) / total, 0.0)
    g = torch.zeros_like(s).scatter_add_(1, at, d)
    if kind == "SIGMOID":
        return g * s * (1 - s)
    return s * (g - (g * s).sum(1, keepdim=True))


def place(ids, first, E):
    """offsets, rows, places."""
    T, k = ids.shape
    flat = ids.reshape(-1).tolist()
    live = sorted((e - first, n) for n, e in enumerate(flat) if first <= e < first + E)
    offsets, rows, places = [0] * (E + 1), [-1] * (T * k), [-1] * (T * k)
    for p, (e, n) in enumerate(live):
        rows[p], places[n] = n // k, p
        offsets[e + 1] += 1
    for e in range(E):
        offsets[e + 1] += offsets[e]
    i32 = torch.int32
    return (torch.tensor(offsets, dtype=i32), torch.tensor(rows, dtype=i32),
            torch.tensor(places, dtype=i32).view(T, k))
