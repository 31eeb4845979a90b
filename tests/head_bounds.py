"""Error bounds of the head operators' gradients, counted from the roundings that each path makes.

The dlogits of a row are g (onehot - p).  Three paths make them:
  fp16            p from exponentials kept in fp16, the dlogits rounded to fp16
  bf16            p from exponentials kept in fp16, the dlogits rounded to bf16
  bf16 relative   the given token's entry is exact, by the choice of the row's factor, which carries that entry's rounding
                  to bf16 to the other entries; those, p_v / p_tok, are rounded to bf16 themselves; for dW the row of h
                  times the factor is rounded to bf16 too
All else is in fp32: sums over K in the tensor cores, which round towards zero (at most a step of the sum of absolute
products for each 16 of K), the functions (a few steps), and the coefficient, whose error is that of q."""
import numpy as np

import head_reference as R

STEP32 = 2.0 ** -23
KEPT = 2.0 ** -11          # the kept exponential, fp16


def grad_bounds(P, g, lp, dtype, relative, out, q_err, scale):
    """(dH, its bound, dW, its bound), scaled.  The absolute part: entries of the dlogits below the smallest normal
    number.  fp16 holds max |g| at 2^13 or more, so its half step there, 2^-25, is 2^-38 of max |g|; the kept exponentials'
    is below that.  bf16 has fp32's range."""
    rH, rW, aH, aW = R.gradients(P, g, lp)
    g = np.where(P.mask, g, 0.0) / P.T
    N, V = lp.shape
    h, more = R.HALF_STEP[dtype], 1 + 2.0 ** -7
    fH, fW = (2 * q_err + (K / 16 + 16) * STEP32 for K in (V, N))     # fp32: relative to the sum of absolute products
    if relative:
        t = np.abs(g * np.expm1(lp[np.arange(N), P.tokens]))[:, None]   # the given tokens' entries
        tH, tW = t * np.abs(P.W[P.tokens]), np.zeros_like(aW)
        np.add.at(tW, P.tokens, t * np.abs(P.h))
        bH = fH * aH + 2 * h * more * np.maximum(aH - tH, 0.0)
        bW = fW * aW + h * more * tW + 3 * h * more * np.maximum(aW - tW, 0.0)
    else:
        bH, bW = (fH + (KEPT + h) * more) * aH, (fW + (KEPT + h) * more) * aW
        tiny = 2.0 ** -36 * np.abs(g).max()
        bH, bW = bH + tiny * np.abs(P.W).sum(0)[None, :], bW + tiny * np.abs(P.h[P.mask]).sum(0)[None, :]
    rH, rW, bH, bW = scale * rH, scale * rW, scale * bH, scale * bW
    bH = bH + R.HALF_STEP[dtype] * (np.abs(rH) + bH) + R.TINY[dtype]
    bW = bW + R.HALF_STEP[out] * (np.abs(rW) + bW) + R.TINY[out]
    return rH, bH, rW, bW


def shows_loss(ref, bound):
    """Whether an all-zero result would be far outside the bound: most of the gradient lies well above it."""
    return bool((np.abs(ref) > 4 * bound).mean() > 0.5)
