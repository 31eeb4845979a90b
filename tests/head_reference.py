"""Plain fp64 numpy definitions of the head operators (log-probs, clipped
policy loss, preference loss), their gradients, and error bounds counted from
the roundings the operators make.  No code of the library is used."""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

# half a step of each type, relative to the value
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "f32": 2.0 ** -24}
# smallest positive subnormal / 2: the absolute part of a rounding
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "f32": 2.0 ** -150}


@dataclass
class Problem:
    n_groups: int
    G: int
    L: int
    h: np.ndarray        # [N x d] fp64 (exact values of the 16-bit inputs)
    W: np.ndarray        # [V x d]
    tokens: np.ndarray   # [N]
    mask: np.ndarray     # [N] bool
    T: float = 1.0

    @property
    def rows(self):
        return np.flatnonzero(self.mask)


def logits(P):
    return P.h @ P.W.T / P.T


def logp_entropy(P):
    """q and entropy [N], 0 on masked rows, and log softmax of every row."""
    z = logits(P)
    m = z.max(1, keepdims=True)
    lse = (m + np.log(np.exp(z - m).sum(1, keepdims=True)))
    lp = z - lse
    N = len(P.tokens)
    q = lp[np.arange(N), P.tokens]
    ent = -(np.exp(lp) * lp).sum(1)
    return np.where(P.mask, q, 0.0), np.where(P.mask, ent, 0.0), lp


def gradients(P, g, lp):
    """dH, dW of sum_t g_t q_t, and the sums of absolute products that roundings scale with."""
    g = np.where(P.mask, g, 0.0)
    N = len(P.tokens)
    dz = -np.exp(lp)
    one = np.zeros_like(dz)
    one[np.arange(N), P.tokens] = 1.0
    dz = (dz + one) * (g / P.T)[:, None]
    return dz @ P.W, dz.T @ P.h, np.abs(dz) @ np.abs(P.W), np.abs(dz).T @ np.abs(P.h)


def clip_loss(P, adv, old, ref, beta, lo, hi, seq_mean):
    """loss, row stats [N x 3], d loss / d q [N]."""
    q, _, lp = logp_entropy(P)
    seq = np.arange(len(q)) // P.L
    A = np.asarray(adv, np.float64)[seq]
    r = np.where(P.mask, np.exp(np.where(P.mask, q - old, 0.0)), 0.0)
    rc = np.clip(r, 1 - lo, 1 + hi)
    ell = -np.minimum(r * A, rc * A)
    g = np.where(r * A <= rc * A, -A * r, 0.0)
    pen = np.zeros_like(q)
    if beta:
        x = np.where(P.mask, ref - q, 0.0)
        pen = np.expm1(x) - x
        ell = ell + beta * pen
        g = g - beta * np.expm1(x)
    n = P.n_groups * P.G
    length = np.bincount(seq, P.mask, n)
    if seq_mean:
        act = max(1, int((length > 0).sum()))
        w = np.where(P.mask, 1.0 / (np.maximum(length, 1)[seq] * act), 0.0)
    else:
        w = P.mask / max(1, int(P.mask.sum()))
    stats = np.where(P.mask[:, None], np.stack([q, r, pen], 1), 0.0)
    return float((ell * w).sum()), stats, g * w, lp


def pair_loss(P, ref, beta, kind="sigmoid", smoothing=0.0, length_mean=False):
    """loss, pair stats [n x 4], d loss / d q [N], log softmax."""
    q, _, lp = logp_entropy(P)
    x = np.where(P.mask, q - ref, 0.0).reshape(-1, P.L)
    length = P.mask.reshape(-1, P.L).sum(1)
    div = np.maximum(length, 1) if length_mean else np.ones_like(length)
    S = (x.sum(1) / div).reshape(-1, 2)
    m = beta * (S[:, 0] - S[:, 1])
    live = length.reshape(-1, 2).sum(1) > 0
    if kind == "sigmoid":
        sp = lambda a: np.logaddexp(0.0, a)  # noqa: E731  log(1 + e^a)
        ell = (1 - smoothing) * sp(-m) + smoothing * sp(m)
        dm = smoothing - 1 / (1 + np.exp(m))
    elif kind == "hinge":
        ell, dm = np.maximum(0, 1 - m), np.where(m < 1, -1.0, 0.0)
    else:
        t = m / beta - 1 / (2 * beta)
        ell, dm = t * t, 2 * t / beta
    n = max(1, int(live.sum()))
    ell, dm = np.where(live, ell, 0.0), np.where(live, dm, 0.0) / n
    g = (np.stack([beta * dm, -beta * dm], 1).reshape(-1) / div)[np.arange(len(q)) // P.L]
    stats = np.stack([beta * S[:, 0], beta * S[:, 1], m, ell], 1)
    return float(ell.sum() / n), stats, np.where(P.mask, g, 0.0), lp


# ---------------------------------------------------------------- error bounds

def logp_bound(P):
    """|q error| per row: the logits' sums (16 additions of 16 products in the tensor core, rounded towards zero, a
    whole step of fp32 each, then d / 256 additions in registers) against sum |h W|; exp2, log2 and the sums over V, a few
    steps each (1e-6 of a number of order one); and the rounding of q itself."""
    d = P.h.shape[1]
    B = (np.abs(P.h) @ np.abs(P.W).T).max(1) / P.T
    q = np.abs(logp_entropy(P)[0])
    return (18 + d / 256) * 2.0 ** -23 * B + 2e-6 + 2 * HALF_STEP["f32"] * q


def grad_bound(ref, absprod, dtype, out, q_err, scale):
    """|error| per element of a gradient: two roundings of the dlogits (the kept exponential is bf16 for both types),
    the coefficient's own error (from q), the fp32 sums, and the output's rounding."""
    rel = HALF_STEP["bf16"] + HALF_STEP[dtype] + 4 * q_err + 1e-4
    return HALF_STEP[out] * np.abs(ref) * (1 + rel) + rel * absprod + scale * 1e-9 + TINY[out]
