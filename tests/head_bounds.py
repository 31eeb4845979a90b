"""Error bounds of the head operators' gradients, counted from the roundings that each path makes.

The dlogits of a row are g (onehot - p).  Three paths make them:
  fp16            p from exponentials kept in fp16, the dlogits rounded to fp16
  bf16            p from exponentials kept in fp16, the dlogits rounded to bf16
  bf16 relative   p_v / p_tok rounded to bf16; for dW the row of h, times the row's factor, rounded to bf16 too
All else is in fp32: sums over K in the tensor cores, which round towards zero (at most a step of the sum of absolute
products for each 16 of K), the functions (a few steps), and the coefficient, whose error is that of q."""
import numpy as np

import head_reference as R

STEP32 = 2.0 ** -23
KEPT = 2.0 ** -11          # the kept exponential, fp16


def rel_bound(dtype, relative, dw, K, q_err):
    """Relative to the sum of absolute products; K is the length of the gradient's sum."""
    h = R.HALF_STEP[dtype]
    rounds = (2 * h if dw else h) if relative else KEPT + h
    return rounds * (1 + 2.0 ** -7) + 2 * q_err + (K / 16 + 16) * STEP32


def grad_bounds(P, g, lp, dtype, relative, out, q_err, scale):
    """(dH, its bound, dW, its bound), scaled.  The absolute part: entries of the dlogits below the smallest normal
    number.  fp16 holds max |g| at 2^13 or more, so its half step there, 2^-25, is 2^-38 of max |g|; the kept exponentials'
    is below that.  bf16 has fp32's range."""
    rH, rW, aH, aW = R.gradients(P, g, lp)
    gmax = np.abs(np.where(P.mask, g, 0.0)).max() / P.T
    tiny = 2.0 ** -36 * gmax * (dtype == "fp16" or not relative)
    N, V = lp.shape
    bH = scale * (rel_bound(dtype, relative, False, V, q_err) * aH + tiny * np.abs(P.W).sum(0)[None, :])
    bW = scale * (rel_bound(dtype, relative, True, N, q_err) * aW + tiny * np.abs(P.h[P.mask]).sum(0)[None, :])
    rH, rW = scale * rH, scale * rW
    bH = bH + R.HALF_STEP[dtype] * (np.abs(rH) + bH) + R.TINY[dtype]
    bW = bW + R.HALF_STEP[out] * (np.abs(rW) + bW) + R.TINY[out]
    return rH, bH, rW, bW


def shows_loss(ref, bound):
    """Whether an all-zero result would be far outside the bound: most of the gradient lies well above it."""
    return bool((np.abs(ref) > 4 * bound).mean() > 0.5)
