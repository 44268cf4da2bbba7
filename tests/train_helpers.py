"""Plain 64-bit references and derived error bounds of the gated block and of
the cross entropy head (and their gradients), for the GPU tests. They share no
code with the library; everything runs on the CPU in float64.

Bounds. A product of K terms accumulated in fp32 is within TAU = 1e-5 of
D = sum |a| |b| (the library's rule for its products). A rounding to bf16 is off by
at most HALF = 2^-8 of the value, fp32 elementwise evaluation by EVAL = 2^-18 of
the value (a few roundings and hardware exponentials with arguments up to about
30, each 2^-24 of the argument)."""

from __future__ import annotations

import math

import torch

TAU, HALF, EVAL = 1e-5, 2.0 ** -8, 2.0 ** -18
GATES = ("SILU", "GELU", "GELU_TANH", "RELU", "SIGMOID")
# largest |act'| and |act''| of each gate (of gelu and gelu_tanh at about 1.41 and 0)
LIP = {"SILU": 1.1, "GELU": 1.13, "GELU_TANH": 1.13, "RELU": 1.0, "SIGMOID": 0.25}
LIP2 = {"SILU": 0.5, "GELU": 0.8, "GELU_TANH": 0.8, "RELU": 0.0, "SIGMOID": 0.1}


def act_slope(z, gate):
    if gate == "SILU":
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    if gate == "SIGMOID":
        s = torch.sigmoid(z)
        return s, s * (1 - s)
    if gate == "RELU":
        return torch.where(z > 0, z, 0.0), (z > 0).double()
    if gate == "GELU":
        P = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * P, P + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


class Glu:
    """x [T, K], w [2 F, K], dh [T, F] bf16, bias [2 F] fp32 or None (CPU)."""

    def __init__(self, x, w, bias, gate, dh=None):
        self.gate, self.F = gate, w.shape[0] // 2
        x, w = x.double(), w.double()
        z = x @ w.T
        ez = TAU * (x.abs() @ w.abs().T)
        if bias is not None:
            z = z + bias.double()
            ez = ez + 2.0 ** -23 * z.abs()
        F = self.F
        g, u, eg, eu = z[:, :F], z[:, F:], ez[:, :F], ez[:, F:]
        act, slope = act_slope(g, gate)
        ea = LIP[gate] * eg + EVAL * act.abs() + 2.0 ** -22
        self.h = act * u
        self.h_err = ea * (u.abs() + eu) + act.abs() * eu + EVAL * self.h.abs()
        if dh is None:
            return
        dh = dh.double()
        es = LIP2[gate] * eg + EVAL * slope.abs() + 2.0 ** -20
        if gate == "RELU":  # the step may fall on either side of 0
            es = es + (g.abs() <= eg).double()
        dz = torch.cat([dh * u * slope, dh * act], 1)
        e = torch.cat([dh.abs() * (es * (u.abs() + eu) + slope.abs() * eu), dh.abs() * ea], 1)
        self.dbias = dz.sum(0)
        self.dbias_err = e.sum(0) + 2.0 ** -20 * dz.abs().sum(0)
        e = e + HALF * (dz.abs() + e)  # held in bf16
        self.dx = dz @ w
        self.dx_err = e @ w.abs() + TAU * ((dz.abs() + e) @ w.abs())
        self.dw = dz.T @ x
        self.dw_err = e.T @ x.abs() + TAU * ((dz.abs() + e).T @ x.abs())


class Xent:
    """x [T, K], w [V, K] bf16, target [T], dloss [T] or None (CPU)."""

    def __init__(self, x, w, target, ignore=-100, smoothing=0.0, z_loss=0.0, dloss=None):
        V = w.shape[0]
        x, w, target = x.double(), w.double(), target.long()
        l = x @ w.T
        el = TAU * (x.abs() @ w.abs().T)
        self.lse = torch.logsumexp(l, 1)
        worst = el.max(1).values
        self.lse_err = worst + EVAL * (1 + self.lse.abs()) + 2.0 ** -22 * l.abs().max(1).values
        keep = target != ignore
        known = keep & (target >= 0) & (target < V)
        at = torch.where(known, target, 0)
        hit = l.gather(1, at[:, None])[:, 0]
        loss = self.lse - (1 - smoothing) * hit - smoothing * l.mean(1) + z_loss * self.lse ** 2
        loss = torch.where(known, loss, math.nan)
        self.loss = torch.where(keep, loss, 0.0)
        self.loss_err = torch.where(keep, self.lse_err * (1 + 2 * z_loss * self.lse.abs()) + 2 * worst
                                    + EVAL * (hit.abs() + z_loss * self.lse ** 2), 0.0)
        if dloss is None:
            return
        s = torch.where(keep, dloss.double(), 0.0)[:, None]
        p = torch.exp(l - self.lse[:, None]) * (1 + 2 * z_loss * self.lse[:, None])
        G = p - smoothing / V
        G.scatter_add_(1, at[:, None], -(1 - smoothing) * torch.ones_like(s))
        G = G * s
        # e^(l - lse) takes the error of both exponents; its rounding and that
        # of the terms follow
        e = s.abs() * (p * (el + self.lse_err[:, None] + EVAL * (1 + l.abs() + self.lse[:, None].abs()))
                       + EVAL * 1.0 / V)
        e = e + HALF * (G.abs() + e) + EVAL * G.abs()
        self.dx = G @ w
        self.dx_err = e @ w.abs() + TAU * ((G.abs() + e) @ w.abs())
        self.dw = G.T @ x
        self.dw_err = e.T @ x.abs() + TAU * ((G.abs() + e).T @ x.abs())


def close(got, want, err, bf16, what):
    """Every element within its bound (and a bf16 result's rounding), and, where
    there are enough of them, the whole result within 1.5 * HALF in the 2-norm:
    its roundings (of G or dz, and of the result) are independent, each of at
    most HALF and so of about HALF / sqrt(3), together 0.82 HALF."""
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
    if bf16 and want.numel() >= 4096 and bool(want.isfinite().all()) and float(want.norm()) > 0:
        rel = float((got - want).norm() / want.norm())
        assert rel <= 1.5 * HALF, f"{what}: {rel} in the 2-norm"
