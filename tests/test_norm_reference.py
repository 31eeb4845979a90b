"""The fp64 definitions that the norm's and the checkpoints' tests use, against differences and by hand."""
import numpy as np
import pytest

import norm_reference as R


@pytest.mark.parametrize("d,eps", [(64, 1e-6), (128, 0.3)])
def test_the_gradient_is_the_differences(d, eps):
    rng = np.random.default_rng(d)
    s, w, dy = rng.normal(size=(5, d)), rng.normal(size=d), rng.normal(size=(5, d))
    dx, dw, _, _ = R.norm_grad(s, w, dy, eps)

    def loss(s, w):
        return (R.norm(s, w, eps)[0] * dy).sum()

    h = 1e-5
    for _ in range(8):
        u, v = rng.normal(size=s.shape), rng.normal(size=d)
        got = (loss(s + h * u, w + h * v) - loss(s - h * u, w - h * v)) / (2 * h)
        want = (dx * u).sum() + (dw * v).sum()
        assert abs(got - want) <= 1e-8 * (1 + np.abs(dx * u).sum() + np.abs(dw * v).sum())


def test_norm_by_hand():
    s = np.zeros((2, 64))
    s[0, :4] = [4.0, -4.0, 4.0, 4.0]                      # mean square 1
    y, _ = R.norm(s, np.full(64, 0.5), 0.0 + 3.0)         # 1 / sqrt(1 + 3) = 1/2
    assert y[0, :4].tolist() == [1.0, -1.0, 1.0, 1.0] and not y[1].any()
    assert R.row_scale(y, "e4m3").tolist() == [1 / 448, R.LEAST]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_checkpoint_values_within_half_a_step(dt):
    rng = np.random.default_rng(3)
    x = R.rounded(rng.normal(size=(40, 192)) * np.exp(3 * rng.normal(size=(40, 1))), dt)
    x[3] = 0.0
    codes, scales = R.pack(x)
    assert np.abs(codes).max() == 127 and not codes[3].any()
    assert np.all(np.abs(R.rounded(R.unpack(codes, scales), dt) - x) <= R.ckpt_bound(x, scales, dt))
    top = np.maximum(np.abs(x).reshape(40, 3, 64).max(2) / 127, R.LEAST)
    assert np.all(np.abs(scales - top) <= 2.0 ** -8 * scales)
