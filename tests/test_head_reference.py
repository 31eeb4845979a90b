"""The fp64 definitions the GPU tests compare with: gradients against central differences, closed forms, and empty inputs."""
import numpy as np
import pytest

import head_reference as R


def problem(seed=0, n_groups=2, G=2, L=5, d=6, V=9, T=1.3, lens=None):
    rng = np.random.default_rng(seed)
    N = n_groups * G * L
    mask = rng.random(N) < 0.7 if lens is None else (np.arange(L)[None] < np.asarray(lens)[:, None]).reshape(-1)
    return R.Problem(n_groups, G, L, rng.normal(size=(N, d)), rng.normal(size=(V, d)), rng.integers(0, V, N), mask, T)


def losses(P, rng):
    N, n = len(P.tokens), P.n_groups * P.G
    q = R.logp_entropy(P)[0]
    adv, old, ref = rng.normal(size=n), q - 0.3 * rng.normal(size=N), q + 0.3 * rng.normal(size=N)
    dq = rng.normal(size=N)
    out = [("given", lambda p: (float((dq * R.logp_entropy(p)[0]).sum()), None, np.where(p.mask, dq, 0), R.logp_entropy(p)[2]))]
    for seq_mean in (False, True):
        for beta in (0.0, 0.04):
            out.append((f"clip {seq_mean} {beta}", lambda p, s=seq_mean, b=beta: R.clip_loss(p, adv, old, ref, b, 0.2, 0.3, s)))
    for kind, e, mean in (("sigmoid", 0.0, False), ("sigmoid", 0.2, True), ("hinge", 0.0, False), ("square", 0.0, True)):
        out.append((f"pair {kind} {mean}", lambda p, k=kind, s=e, m=mean: R.pair_loss(p, ref, 0.4, k, s, m)))
    return out


@pytest.mark.parametrize("lens", [None, [5, 0, 3, 1], [0, 0, 2, 5], [0, 0, 0, 0]])
def test_gradients_match_central_differences(lens):
    P = problem(1, lens=lens)
    rng = np.random.default_rng(2)
    for name, f in losses(P, rng):
        _, _, g, lp = f(P)
        dH, dW, _, _ = R.gradients(P, g, lp)
        for arr, grad in ((P.h, dH), (P.W, dW)):
            for _ in range(12):
                i = tuple(rng.integers(0, s) for s in arr.shape)
                keep, eps = arr[i], 1e-5
                arr[i] = keep + eps
                up = f(P)[0]
                arr[i] = keep - eps
                dn = f(P)[0]
                arr[i] = keep
                assert abs((up - dn) / (2 * eps) - grad[i]) <= 1e-6 * (1 + abs(grad[i])), (name, i)


def test_closed_forms():
    P = problem(3, T=1.0)
    P.W[:] = 0                                   # uniform softmax: q = -log V, entropy = log V
    q, ent, _ = R.logp_entropy(P)
    assert np.allclose(q[P.mask], -np.log(9)) and np.allclose(ent[P.mask], np.log(9)) and not q[~P.mask].any()
    P = problem(4)
    q = R.logp_entropy(P)[0]
    # on-policy, no reference: loss is the mean of -A, and nothing is clipped
    adv = np.array([1.0, -2.0, 0.5, 3.0])
    loss, stats, _, _ = R.clip_loss(P, adv, q, None, 0.0, 0.2, 0.2, False)
    assert np.isclose(loss, -(adv[np.arange(20) // 5] * P.mask).sum() / P.mask.sum())
    assert np.allclose(stats[P.mask, 1], 1)
    # policy equal to the reference: margin 0, loss log 2
    loss, stats, _, _ = R.pair_loss(P, q, 0.3)
    assert np.isclose(loss, np.log(2)) and np.allclose(stats[:, :3], 0)
