"""Plain fp64 forms of the rotary embedding and of capped attention, for the
tests of those operators, and the tolerances that go with them.

A rounding to a type is off by at most half a step: HALF[dtype] of the value.
"""

from __future__ import annotations

import math

import numpy as np

HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def rope_ref(x, pos, inv_freq, rot, sections, layout, factor, sign=1.0):
    """x [B, T, H, d] fp64, pos [axes, B, T]: each channel pair as a complex
    number times factor * exp(i * angle)."""
    axis = np.repeat(np.arange(len(sections)), sections)
    ang = sign * pos[axis].transpose(1, 2, 0).astype(np.float64) * np.asarray(inv_freq, dtype=np.float64)   # [B, T, rot/2]
    turn = factor * np.exp(1j * ang)[:, :, None]
    y = np.array(x, dtype=np.float64)
    if layout == "halves":
        z = (x[..., : rot // 2] + 1j * x[..., rot // 2: rot]) * turn
        y[..., : rot // 2], y[..., rot // 2: rot] = z.real, z.imag
    else:
        z = (x[..., 0:rot:2] + 1j * x[..., 1:rot:2]) * turn
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    return y


def rope_tolerance(x, rot, layout, factor, dtype):
    """Elementwise: the sine and cosine (fp32 of an angle reduced in fp64, and
    a multiply by the factor) are within 6 fp32 half-steps of 1, the two
    products and their sum add 3 more of the pair's size, and the store rounds
    once to dtype."""
    size = np.abs(np.array(x, dtype=np.float64))
    a, b = (size[..., : rot // 2], size[..., rot // 2: rot]) if layout == "halves" else (size[..., 0:rot:2], size[..., 1:rot:2])
    pair = (a + b) * abs(factor)
    tol = np.zeros_like(size)
    if layout == "halves":
        tol[..., : rot // 2] = tol[..., rot // 2: rot] = pair
    else:
        tol[..., 0:rot:2] = tol[..., 1:rot:2] = pair
    tol = tol * 9 * HALF["fp32"]
    rotated = np.zeros_like(size)
    rotated[..., :rot] = 1.0
    # half a step of the result, whose size is at most the pair's; channels that pass through are exact
    size_of_result = np.where(rotated > 0, tol / (9 * HALF["fp32"]), 0.0)
    return tol + HALF[dtype] * size_of_result


def capped(s, cap):
    return cap * np.tanh(s / cap) if cap else s


def attend_ref(q, k, v, seen, cap, scale):
    """q [n, d], k, v [m, d] fp64, seen [n, m] bool -> [n, d]; a row that sees nothing is 0."""
    s = np.where(seen, capped(q @ k.T * scale, cap), -np.inf)
    top = np.max(s, axis=1, initial=-np.inf, keepdims=True)
    p = np.exp(s - np.where(np.isfinite(top), top, 0.0)) * seen
    total = p.sum(1, keepdims=True)
    return (p / np.where(total > 0, total, 1.0)) @ v


def attend_tolerance(q, k, v, cap, scale, dtype):
    """How far an output may be from attend_ref on the same inputs, one number
    for a head: the weights' relative error, twice (numerator and row sum),
    and the store's rounding, each times the largest |v|.

    Weights, bf16: each is rounded to 8 bits (half a step, 2^-8 of the value at most
    of its binade's lower end) and computed from a score that is off by at most
    (d + 16) fp32 half-steps of its terms plus the cap's own
    8e-6 of the score; the exponential on the FMA pipe adds 7.5e-5.
    Weights, fp32: the score's error and four half-steps of the score; the sums over
    m keys add their error, (8 + sqrt(m)) half-steps of a convex combination."""
    if not len(k):
        return 0.0
    vmax, m, d = float(np.abs(v).max()), len(k), q.shape[1]
    terms = float((np.abs(q) @ np.abs(k).T * scale).max())
    score = (d + 16) * HALF["fp32"] * terms
    s = min(terms, cap) if cap else terms
    if dtype == "bf16":
        w = 2.0 ** -8 + score + 8e-6 * s + 7.5e-5
        return (2 * w + 2.0 ** -8) * vmax
    w = score + 4 * s * HALF["fp32"] + 4 * HALF["fp32"]
    return (2 * w + 2 * (8 + math.sqrt(m)) * HALF["fp32"]) * vmax


def mix_ref(q, k, v, do, alpha, cap, sink, recent, dtype):
    """The gated mix and its gradients in fp64, and how far a kernel may be
    from each: ((out, dq, dk, dv, dalpha), (their elementwise bounds)).

    Bounds.  e is the relative error of a weight P_c or P_s: its score's error
    ((d + 16) fp32 half-steps of the score's terms, and the cap's own) and the
    error of the row's log-sum and exponentials (1e-4 where the forward pass
    uses the FMA-pipe exponential, else 16 half-steps); r is the rounding of a
    value to the MMA operand's type (bf16; none in fp32); f is m fp32
    half-steps for a sum of m terms.  Then, with |.| sums of the terms' sizes:
      out:  (2 (e + r) + f) of sum P |v|, once per attention, and the roundings
            of A_s and of the store;
      D_c, D_s: f of |dout| . |A|, and |dout| . (error of A);
      dS:   (e + r + f) of its terms sizes P (|dP| + |D|) plus P (error of dP and D);
      dv, dq, dk: the errors of W or dS times the other operand, and the store."""
    B, N, hq, d = q.shape
    hkv = k.shape[2]
    G, scale = hq // hkv, 1.0 / math.sqrt(d)
    i = np.arange(N)
    causal = i[:, None] >= i[None, :]
    lam = causal & ((i[None, :] < sink) | (i[:, None] - i[None, :] < recent))
    bf = dtype == "bf16"
    h32, r, store = HALF["fp32"], (HALF["bf16"] if bf else 0.0), HALF[dtype]
    f = (N + d) ** 0.5 * 4 * h32 + 16 * h32
    out, dq = np.zeros_like(q), np.zeros_like(q)
    dk, dv = np.zeros_like(k), np.zeros_like(v)
    da = np.zeros(hkv)
    t_out, t_dq, t_dk, t_dv, t_da = (np.zeros_like(x) for x in (out, dq, dk, dv, da))
    for b in range(B):
        for h in range(hq):
            j = h // G
            qq, kk, vv, oo, a = q[b, :, h], k[b, :, j], v[b, :, j], do[b, :, h], alpha[j]
            raw = qq @ kk.T * scale
            s = capped(raw, cap)
            slope = 1.0 - np.tanh(raw / cap) ** 2 if cap else np.ones_like(raw)
            terms = np.abs(qq) @ np.abs(kk).T * scale
            es = (d + 16) * h32 * terms + (8e-6 if bf else 4 * h32) * np.abs(s)
            e = 2 * es.max(1, initial=0.0, where=causal)[:, None] + (1e-4 if bf else 16 * h32)   # weight and log-sum
            dp = oo @ vv.T
            dp_size = np.abs(oo) @ np.abs(vv).T
            W, dW, g, dg = (np.zeros((N, N)) for _ in range(4))
            for seen, share, sign in ((causal, a, 1.0), (lam, 1.0 - a, -1.0)):
                top = np.where(seen, s, -np.inf).max(1, keepdims=True)
                p = np.where(seen, np.exp(s - top), 0.0)
                p /= p.sum(1, keepdims=True)
                o = p @ vv
                do_err = (2 * (e + r) + f) * (p @ np.abs(vv)) + store * np.abs(o) * 2      # of the stored attention
                D = (oo * o).sum(1, keepdims=True)
                D_err = (np.abs(oo) * do_err).sum(1, keepdims=True) + f * (np.abs(oo) * np.abs(o)).sum(1, keepdims=True)
                out[b, :, h] += share * o
                t_out[b, :, h] += abs(share) * do_err
                da[j] += sign * float(D.sum())
                t_da[j] += float(D_err.sum())
                W += share * p
                dW += abs(share) * (e + r) * p
                g += share * p * (dp - D)
                # slope (of size at most 1) is off by twice the score's error over the cap, at most 3 e
                dg += abs(share) * p * ((4 * e + 2 * r) * (np.abs(dp) + np.abs(D)) + f * dp_size + D_err)
            t_out[b, :, h] += store * (np.abs(out[b, :, h]) + t_out[b, :, h])
            g, dg = g * slope * scale, (dg * np.maximum(slope, 0) + 2e-6 * np.abs(g) * bool(cap) + r * np.abs(g * slope)) * scale
            dv[b, :, j] += W.T @ oo
            t_dv[b, :, j] += dW.T @ np.abs(oo) + f * (np.abs(W).T @ np.abs(oo))
            dq[b, :, h] = g @ kk
            t_dq[b, :, h] = dg @ np.abs(kk) + f * (np.abs(g) @ np.abs(kk))
            dk[b, :, j] += g.T @ qq
            t_dk[b, :, j] += dg.T @ np.abs(qq) + f * (np.abs(g).T @ np.abs(qq))
    t_dq += store * (np.abs(dq) + t_dq)
    t_dk += store * (np.abs(dk) + t_dk)
    t_dv += store * (np.abs(dv) + t_dv)
    t_da += h32 * np.abs(da)
    tiny = 1e-30
    return (out, dq, dk, dv, da), tuple(x + tiny for x in (t_out, t_dq, t_dk, t_dv, t_da))
