"""Plain fp64 definitions of the norm before the head, its gradient and the 8-bit checkpoints, in numpy, with error bounds
counted from the roundings the operators make.  No code of the library is used."""
from __future__ import annotations

import numpy as np
import torch

TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn,
         "e5m2": torch.float8_e5m2}
# half a step of each type, relative to the value, and half of its smallest positive number
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "f32": 2.0 ** -24, "e4m3": 2.0 ** -4, "e5m2": 2.0 ** -3}
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "f32": 2.0 ** -150, "e4m3": 2.0 ** -10, "e5m2": 2.0 ** -17}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
LEAST = 2.0 ** -126
BLOCK = 64
STEP32 = 2.0 ** -23


def rounded(x, dtype):
    """fp64 values rounded to a type's, as fp64."""
    return torch.from_numpy(np.asarray(x, np.float64)).to(TORCH[dtype]).double().numpy()


def stream(x, residual, dtype):
    """s: the residual stream after the addition."""
    return x if residual is None else rounded(x + residual, dtype)


def norm(s, w, eps):
    """y and 1 / sqrt(mean s^2 + eps) of every row."""
    rstd = 1.0 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    return s * rstd * w, rstd


def rel32(d):
    """How far 1 / sqrt(...) in fp32 may be off, relatively: the squares and their sum, each thread d / 32 in turn at most,
    and ten operations more."""
    return (d / 32 + 16) * STEP32


def y_bound(y, d, dtype):
    return rel32(d) * np.abs(y) + HALF_STEP[dtype] * np.abs(y) * (1 + rel32(d)) + TINY[dtype]


def row_scale(y, dtype):
    return np.maximum(np.abs(y).max(1) / LARGEST[dtype], LEAST)


def code_bound(y, scale, d, dtype):
    """How far code * scale may be off y, where nothing saturates."""
    e = rel32(d) + 4 * STEP32
    return e * np.abs(y) + HALF_STEP[dtype] * np.abs(y) * (1 + e) + TINY[dtype] * scale * (1 + e)


def norm_grad(s, w, dy, eps):
    """dx (without dsum), dw, and their bounds in fp32 before the outputs' rounding."""
    d, n = s.shape[1], s.shape[0]
    _, rstd = norm(s, w, eps)
    g = dy * w
    dx = rstd * (g - s * rstd ** 2 * (g * s).mean(1, keepdims=True))
    each = dy * s * rstd
    size = rstd * (np.abs(g) + np.abs(s) * rstd ** 2 * np.abs(g * s).mean(1, keepdims=True))
    e = 4 * rel32(d)
    return dx, each.sum(0), e * size, (e + (n + 16) * STEP32) * np.abs(each).sum(0)


def rounding(x, bound, dtype):
    """A bound in fp32 and the rounding to an output's type."""
    return bound + HALF_STEP[dtype] * (np.abs(x) + bound) + TINY[dtype]


def pack(x):
    """Codes and scales as the definition has them, scales in fp64 rounded to bf16 once: where a scale or a code lies next to
    a rounding's border, fp32 may take the other side."""
    b = x.reshape(x.shape[0], -1, BLOCK)
    scale = rounded(np.maximum(np.abs(b).max(2) / 127.0, LEAST), "bf16")
    codes = np.rint(b / scale[:, :, None])
    return codes.reshape(x.shape), scale


def unpack(codes, scales):
    return (codes.reshape(codes.shape[0], -1, BLOCK) * scales[:, :, None]).reshape(codes.shape)


def ckpt_bound(x, scales, dtype):
    """How far a checkpoint's value may be off x."""
    each = np.repeat(scales, BLOCK, axis=1)
    return 0.501 * each + HALF_STEP[dtype] * (np.abs(x) + each) + TINY[dtype]
