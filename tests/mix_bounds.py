"""The gated mix and its gradients in fp64, with bounds on a kernel's error
that are a few percent of the results or less: independent roundings are
added as such (in quadrature), and only what may be systematic is added up.

What a kernel rounds, and by how much (half a step of a type: HALF):
  * bf16 MMA operands -- P in the forward pass, W and dS in the backward pass --
    and every bf16 output: independent, at most HALF = 2^-8 of the value, uniform
    within its step, so of standard deviation at most HALF / sqrt(3); in sequences of
    up to 128 tokens dS is the sum of two such operands: HALF^2;
  * a score: fp32 sums of d products ((4 + sqrt(d)) half-steps of the terms'
    size) and, under a cap, a tanh within 8e-6 of the score (fp32: 4 half-steps).
    The tanh's error is a function of the score: systematic;
  * a weight's exponential: 2^-21 of it; in the forward pass without the bounded
    cap, where one exponential in four is a polynomial's: 7.5e-5;
  * log-sums, D_c and D_s: fp32 sums, from weights with the errors above.
With E the relative error of a weight from its score and exponential, a row's
normalised weights are off by E + sum(P E) at most, D by
sum P (E + sum(P E)) |dP - D|, dS by those times its terms.
"""

from __future__ import annotations

import math

import numpy as np

from tests.rotary_and_cap import HALF, capped

H32 = HALF["fp32"]
SIGMAS = 6.0            # of sums of many independent roundings, over at most 10^7 entries


class Bound:
    """An error's standard deviation (independent parts) and its systematic part, elementwise."""

    def __init__(self, var, lin):
        self.sigma, self.lin = np.sqrt(var), lin


def mix_bounds(q, k, v, do, alpha, cap, sink, recent, dtype, tc, stored_d=False):
    """q, do [B, N, Hq, d], k, v [B, N, Hkv, d] fp64 -> (results, bounds) by name (out, dq, dk, dv, dalpha).
    tc: the tensor-core path (bf16, d 128, window at most 128) -- MMA operands in bf16; else fp32 on the CUDA cores.
    stored_d: a wrong kernel, for the bounds' own test, that takes D from the attentions rounded to bf16."""
    B, N, hq, d = q.shape
    hkv = k.shape[2]
    G, scale = hq // hkv, 1.0 / math.sqrt(d)
    i = np.arange(N)
    causal = i[:, None] >= i[None, :]
    lam = causal & ((i[None, :] < sink) | (i[:, None] - i[None, :] < recent))
    r, store = (HALF["bf16"] / math.sqrt(3) if tc else 0.0), HALF[dtype] / math.sqrt(3)
    r_g = r * HALF["bf16"] if N <= 128 else r
    acc = (8 + math.sqrt(N)) * H32                                       # of an fp32 sum's terms
    res = {"out": np.zeros_like(q), "dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v), "dalpha": np.zeros(hkv)}
    var, lin = ({n: np.zeros_like(x) for n, x in res.items()} for _ in range(2))
    for b in range(B):
        for h in range(hq):
            j = h // G
            qq, kk, vv, oo, a = q[b, :, h], k[b, :, j], v[b, :, j], do[b, :, h], alpha[j]
            raw = qq @ kk.T * scale
            s = capped(raw, cap)
            t = np.tanh(raw / cap) if cap else np.zeros_like(raw)
            terms = np.abs(qq) @ np.abs(kk).T * scale
            E = (4 + math.sqrt(d)) * H32 * terms + 8 * H32 * np.abs(s) + 2.0 ** -21
            if cap:
                E = E + (8e-6 if dtype == "bf16" and tc else 4 * H32) * np.abs(s)
            E_fwd = E + (7.5e-5 if tc and not 0 < cap <= 60 else 0.0)
            dp = oo @ vv.T
            dp_err = (4 + math.sqrt(d)) * H32 * (np.abs(oo) @ np.abs(vv).T)
            slope = 1.0 - t * t
            W, W_lin, g, g_lin = (np.zeros((N, N)) for _ in range(4))
            row_da = np.zeros(N)
            for seen, share, sign in ((causal, a, 1.0), (lam, 1.0 - a, -1.0)):
                p = np.where(seen, np.exp(s - np.where(seen, s, -np.inf).max(1, keepdims=True)), 0.0)
                p /= p.sum(1, keepdims=True)
                o = p @ vv
                res["out"][b, :, h] += share * o
                # forward: each weight's rounding moves the row towards or away from its value
                var["out"][b, :, h] += share ** 2 * r * r * ((p * p) @ (vv * vv) - 2 * ((p * p) @ vv) * o + (p * p).sum(1, keepdims=True) * o * o)
                norm_f = E_fwd + (p * E_fwd).sum(1, keepdims=True)
                lin["out"][b, :, h] += abs(share) * ((p * norm_f) @ np.abs(vv) + acc * (p @ np.abs(vv)))
                if tc and seen is lam and not 0 < cap <= 60:
                    var["out"][b, :, h] += (share * store * o) ** 2      # A_s waits in bf16
                o_d = _to_bf16(o) if stored_d else o
                D = (oo * o_d).sum(1, keepdims=True)
                norm = E + (p * E).sum(1, keepdims=True)
                D_lin = (p * norm * np.abs(dp - D)).sum(1, keepdims=True) + (p * dp_err).sum(1, keepdims=True) + \
                    acc * (p * np.abs(dp)).sum(1, keepdims=True)
                row_da += D_lin[:, 0]
                res["dalpha"][j] += sign * float(D.sum())
                W += share * p
                W_lin += abs(share) * p * norm
                g += share * p * (dp - D)
                g_lin += abs(share) * p * (norm * np.abs(dp - D) + D_lin + dp_err)
            var["dalpha"][j] += float((row_da ** 2).sum())                # rows are independent
            g_lin = scale * (slope * g_lin + ((2 * 8e-6 if tc else 4 * H32) * t * t + 2 * H32) * np.abs(g) * bool(cap)) + \
                4 * H32 * np.abs(g) * scale
            g = g * slope * scale
            res["dv"][b, :, j] += W.T @ oo
            var["dv"][b, :, j] += r * r * (W * W).T @ (oo * oo)
            lin["dv"][b, :, j] += W_lin.T @ np.abs(oo) + acc * (np.abs(W).T @ np.abs(oo))
            res["dq"][b, :, h] = g @ kk
            var["dq"][b, :, h] = r_g * r_g * (g * g) @ (kk * kk)
            lin["dq"][b, :, h] = g_lin @ np.abs(kk) + acc * (np.abs(g) @ np.abs(kk))
            res["dk"][b, :, j] += g.T @ qq
            var["dk"][b, :, j] += r_g * r_g * (g * g).T @ (qq * qq)
            lin["dk"][b, :, j] += g_lin.T @ np.abs(qq) + acc * (np.abs(g).T @ np.abs(qq))
    for n in ("out", "dq", "dk", "dv"):
        var[n] += (store * res[n]) ** 2
    lin["dalpha"] += 4 * H32 * np.abs(res["dalpha"])
    return res, {n: Bound(var[n], lin[n] + 1e-30) for n in res}


def _to_bf16(x):
    bits = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((bits + 0x7FFF + ((bits >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32).astype(np.float64)


def excess(name, got, want, bound):
    """None, or a text that says where `got` leaves its bounds: each entry, and the norm over each (sequence, head)."""
    err = np.abs(got - want)
    if not np.all(np.isfinite(got)):
        return f"{name}: not finite"
    tol = SIGMAS * bound.sigma + bound.lin
    if not np.all(err <= tol):
        at = np.unravel_index(np.argmax(err - tol), err.shape)
        return f"{name}{list(at)}: off by {err[at]:.3e}, bound {tol[at]:.3e}"
    if err.ndim == 4:
        norm = lambda x: np.sqrt((x ** 2).sum((1, 3)))  # noqa: E731
        # a norm over 10^3 entries and more is within 1.25 of its expectation; fewer count as one
        many = err.shape[1] * err.shape[3] >= 1000
        limit = (1.25 if many else SIGMAS) * norm(bound.sigma) + norm(bound.lin)
        if not np.all(norm(err) <= limit):
            at = np.unravel_index(np.argmax(norm(err) / limit), limit.shape)
            return f"{name} of sequence {at[0]}, head {at[1]}: norm of the error {norm(err)[at]:.3e}, bound {limit[at]:.3e}"
    return None
