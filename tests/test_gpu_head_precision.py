"""The head operators' gradients against bounds counted from each path's own roundings (head_bounds.py), tight enough that
a path with fewer bits than its own, or a gradient that is lost, would not pass."""
import numpy as np
import pytest

import head_bounds as B
import head_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import rl_fine_tuning_gb300 as rg  # noqa: E402
from test_gpu_head_ops import Case, clean, far_case, host  # noqa: E402


def in_bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().double().numpy()


def check(c, dH, dW, g, lp, scale, dw_f32, relative):
    assert int(c.status) == 0 and int(c.inf) == 0
    q_err = R.logp_bound(c.P)[c.P.mask].max(initial=0)
    rH, bH, rW, bW = B.grad_bounds(c.P, g, lp, c.dtype, relative, "f32" if dw_f32 else c.dtype, q_err, scale)
    eH, eW = np.abs(host(dH) - rH), np.abs(host(dW) - rW)
    assert np.all(eH <= bH), ("dH", np.max(eH / bH))
    assert np.all(eW <= bW), ("dW", np.max(eW / bW))
    return rH, bH, rW, bW


# (n_groups, G, L, d, V, dtype, mask, chunk_rows): 4M logits a chunk and more are relative in bf16
PATHS = [
    (2, 4, 37, 320, 1000, "fp16", "ragged", 0),
    (1, 3, 211, 128, 515, "fp16", "holes", 128),       # five chunks
    (1, 1, 250, 64, 70001, "fp16", "ragged", 0),       # K pieces
    (2, 4, 37, 320, 1000, "bf16", "ragged", 0),        # merge and dlogits in one
    (1, 3, 211, 128, 515, "bf16", "holes", 128),
    (1, 1, 250, 64, 70001, "bf16", "ragged", 0),       # relative
    (1, 1, 300, 128, 40000, "bf16", "all", 128),       # relative, three chunks
]


@pytest.mark.parametrize("s", PATHS, ids=str)
@pytest.mark.parametrize("dw_f32", [False, True])
def test_gradients_within_their_paths_roundings(s, dw_f32):
    n, G, L, d, V, dt, mask, cr = s
    c = Case(n, G, L, d, V, dt, mask, seed=60, chunk_rows=cr)
    rows = min(cr, n * G * L) if cr else n * G * L
    relative = dt == "bf16" and (rows + 127) // 128 * 128 * V >= 1 << 22
    dq = c.rng.normal(size=len(c.tok)).astype(np.float32)
    dH, dW = c.logp_bwd(torch.from_numpy(dq).cuda(), 8.0, dw_f32)
    g, lp = clean(dq, c.P.mask), R.logp_entropy(c.P)[2]
    rH, bH, rW, bW = check(c, dH, dW, g, lp, 8.0, dw_f32, relative)
    assert B.shows_loss(rH[c.P.rows], bH[c.P.rows])
    if dt == "fp16":       # dlogits rounded to bf16, planted in the reference, are found
        dz = -np.exp(lp)
        dz[np.arange(len(g)), c.P.tokens] += 1.0
        dz = in_bf16(dz * g[:, None])
        assert np.any(np.abs(8.0 * dz @ c.P.W - rH) > bH) and np.any(np.abs(8.0 * dz.T @ c.P.h - rW) > bW)


@pytest.mark.parametrize("size", [1e-18, 1e-12, 1.0, 1e6])
def test_relative_gradients_of_improbable_tokens_keep_their_size(size):
    """Rows with q down to -38, whose factor is g e^q, and d loss / d q of any size, brought back by the loss scale.  Only
    the improbable rows have a gradient, so a lost one shows in dH and in dW."""
    c = far_case(1, 1, 250, 70001, 0, 0, 61)
    W = c.W.float().cpu()
    rows = c.P.rows[::10]
    for n, t in enumerate(rows):
        o = (int(c.tok[t]) + 29) % 70001
        c.h[t] = ((24.0 + 0.35 * n) * W[o] / float(W[o] @ W[o])).to(torch.bfloat16).cuda()
    c.P.h = host(c.h)
    q, _, lp = R.logp_entropy(c.P)
    low = rows[q[rows] < -20]
    assert -40 < q.min() < -30 and len(low) > 5
    dq = np.zeros(250, np.float32)
    dq[low] = size * (1 + c.rng.random(len(low)))
    scale = float(np.float32(1.0 / size))
    dH, dW = c.logp_bwd(torch.from_numpy(dq).cuda(), scale)
    rH, bH, rW, bW = check(c, dH, dW, dq.astype(np.float64), lp, scale, False, True)
    assert B.shows_loss(rH[low], bH[low])
    big = np.abs(rW) > 1e-3 * np.abs(rW).max()
    assert B.shows_loss(rW[big], bW[big])
