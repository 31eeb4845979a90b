"""The head operators where they can go wrong, beyond their ordinary range."""
import numpy as np
import pytest

import head_bounds as B
import head_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import rl_fine_tuning_gb300 as rg  # noqa: E402
from test_gpu_head_ops import Case, clean, host  # noqa: E402


def check(c, dH, dW, g, lp, scale, dw_f32=False, relative=False):
    assert int(c.status) == 0 and int(c.inf) == 0
    q_err = R.logp_bound(c.P)[c.P.mask].max()
    rH, bH, rW, bW = B.grad_bounds(c.P, g, lp, c.dtype, relative, "f32" if dw_f32 else c.dtype, q_err, scale)
    eH, eW = np.abs(host(dH) - rH), np.abs(host(dW) - rW)
    assert np.all(eH <= bH), ("dH", np.max(eH / bH))
    assert np.all(eW <= bW), ("dW", np.max(eW / bW))
    assert not host(dH)[~c.P.mask].any()
    return rH, bH, rW, bW


# ---------------------------------------------------------------- gradients near the end of fp32's range

@pytest.mark.parametrize("dt,size", [("fp16", 1e-30), ("fp16", 1e-36), ("fp16", 2e-38), ("bf16", 1e-30)])
def test_tiny_gradients_of_given_size(dt, size):
    """d loss / d q near the smallest fp32 numbers, brought back by the loss scale: as exact as any other."""
    c = Case(1, 2, 60, 128, 500, dt, "ragged", seed=40)
    dq = (size * c.rng.normal(size=len(c.tok))).astype(np.float32)
    scale = float(np.float32(0.25 / size))
    dH, dW = c.logp_bwd(torch.from_numpy(dq).cuda(), scale, True)
    rH, bH, rW, bW = check(c, dH, dW, clean(dq, c.P.mask), R.logp_entropy(c.P)[2], scale, True)
    assert B.shows_loss(rH[c.P.rows], bH[c.P.rows])
    dH, dW = c.logp_bwd(torch.from_numpy(dq).cuda(), 1.0)          # unscaled: far below fp16, no overflow on the way
    assert int(c.inf) == 0 and (dt == "bf16" or not (dH.any() or dW.any()))


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("margin", [70.0, 78.0, 84.0, 88.0, 95.0])
@pytest.mark.parametrize("cr", [0, 128])
def test_saturated_pairs(dt, margin, cr):
    """A preferred completion far ahead: sigmoid(-m) down to the end of fp32, gradients near 0 and finite."""
    L = 80
    c = Case(2, 2, L, 128, 300, dt, "all", seed=41, chunk_rows=cr, beta=1.0)
    q = R.logp_entropy(c.P)[0]
    sign = np.where(np.arange(4 * L) // L % 2 == 0, 1.0, -1.0)
    ref = (q - sign * margin / (2 * L)).astype(np.float32)         # each completion's S is +- margin / 2
    loss, _, st, dH, dW = c.pair(torch.from_numpy(ref).cuda(), rg.pair_opts(dw_f32=True))
    assert int(c.status) == 0 and int(c.inf) == 0
    rl, rs, g, lp = R.pair_loss(c.P, ref.astype(np.float64), c.beta)
    # S: fp32 numbers of q, each off by logp_bound; d sigmoid(-m) / dm is at most itself
    rel = 2 * L * R.logp_bound(c.P).max()
    assert np.all(np.abs(host(st)[:, 2] - rs[:, 2]) <= rel + 1e-5)
    assert abs(float(loss) - rl) <= (np.expm1(rel + 1e-5) + 1e-5) * rl + 1e-44
    rH, rW, aH, aW = R.gradients(c.P, g, lp)
    f = np.expm1(rel + 1e-5) + (2.0 ** -6 if dt == "bf16" else 2.0 ** -9)
    # expf(m) is infinite from m = 88.7 on: 0 where sigmoid(-m) is below 3e-39.  bf16 dlogits carry no scale of their own:
    # entries and products below the smallest normal number may become 0.
    low = 3e-39 if dt == "fp16" else 2.0 ** -125
    assert np.all(np.abs(host(dW) - rW) <= f * aW + low * (1 + np.abs(c.P.h)).sum(0))
    assert np.all(np.abs(host(dH) - rH) <= f * aH + R.TINY[dt] + low * (1 + np.abs(c.P.W)).sum(0))


# ---------------------------------------------------------------- rows with a bad token

def with_bad_tokens(c, rows):
    """Tokens out of range in `rows` on the device; the reference problem keeps good ones."""
    c.tok = c.tok.clone()
    for i, t in enumerate(rows):
        c.tok[t] = -1 if i % 2 else c.P.W.shape[0]
    bad = np.zeros(len(c.P.tokens), bool)
    bad[list(rows)] = True
    return bad & c.P.mask


@pytest.mark.parametrize("dt,V,cr,far", [("fp16", 300, 0, 0), ("bf16", 300, 0, 0), ("fp16", 300, 128, 0),
                                         ("bf16", 70001, 0, 0), ("bf16", 70001, 0, 1)])
def test_a_bad_token_beside_large_logits(dt, V, cr, far):
    """Logits of 150 and more in the row with the bad token: it contributes nothing, and nothing overflows."""
    c = Case(1, 2, 100, 64, V, dt, "all", seed=42, chunk_rows=cr)
    t = 7
    o = int(c.tok[t])
    W = c.W[o].float()
    c.h[t] = (160.0 * W / float(W @ W)).to(c.h.dtype)
    if far:                # another row's token is improbable: the chunk takes its dlogits relative to the maximum
        W = c.W[(int(c.tok[20]) + 9) % V].float()
        c.h[20] = (70.0 * W / float(W @ W)).to(c.h.dtype)
    c.P.h = host(c.h)
    assert R.logits(c.P)[t].max() > 150 and (R.logp_entropy(c.P)[0].min() < -45) == bool(far)
    bad = with_bad_tokens(c, [t])
    dq = np.ones(200, np.float32)
    dH, dW = c.logp_bwd(torch.from_numpy(dq).cuda(), 1.0, True)
    assert int(c.status) == 2 and int(c.inf) == 0 and not dH[t].any()
    g = np.where(bad, 0.0, 1.0)
    q_err = np.delete(R.logp_bound(c.P), t).max()
    rH, bH, rW, bW = B.grad_bounds(c.P, g, R.logp_entropy(c.P)[2], dt, V > 1000 and not far, "f32", q_err, 1.0)
    assert np.all(np.abs(host(dH) - rH) <= bH) and np.all(np.abs(host(dW) - rW) <= bW)
    if dt == "bf16":       # the same through the clipped loss
        old = torch.from_numpy(R.logp_entropy(c.P)[0].astype(np.float32)).cuda()
        loss, st, dH, dW = c.clip(torch.ones(2, device="cuda"), old, old, rg.clip_opts())
        assert int(c.status) == 2 and int(c.inf) == 0 and not dH[t].any() and not st[t].any()
        assert bool(torch.isfinite(dW.float()).all()) and bool(torch.isfinite(loss))


@pytest.mark.parametrize("dt,V,cr", [("bf16", 300, 0), ("bf16", 300, 128), ("fp16", 300, 0), ("bf16", 70001, 0)])
@pytest.mark.parametrize("mean", [False, True])
def test_bad_tokens_in_a_pair_contribute_nothing(dt, V, cr, mean):
    """S counts 0 for such a row (not minus its reference log-prob); with length_mean it stays in the divisor."""
    c = Case(3, 2, 70, 64, V, dt, "all", seed=43, chunk_rows=cr, beta=2.0 if mean else 0.05)
    bad = with_bad_tokens(c, [3, 69, 150, 151, 152, 153])
    bad[280:350] = True                                  # a completion of bad tokens alone
    c.tok[280:350] = V + 5
    q = R.logp_entropy(c.P)[0]
    ref = (q - 0.3 * c.rng.normal(size=len(q))).astype(np.float32)
    rref = np.where(bad, q, ref)                         # the reference: q - logp_ref = 0 there
    ref[bad] = -25.0
    opts = rg.pair_opts(length_mean=mean, dw_f32=True)
    loss, qq, st, dH, dW = c.pair(torch.from_numpy(ref).cuda(), opts)
    rl, rs, g, lp = R.pair_loss(c.P, rref, c.beta, length_mean=mean)
    assert int(c.status) == 2 and int(c.inf) == 0
    assert not host(qq)[bad].any() and not host(dH)[bad].any()
    S_err = (1 if mean else 70) * (R.logp_bound(c.P).max() + 2e-6)
    m_err = 2 * c.beta * S_err + 1e-6 * max(1.0, np.abs(rs).max())
    assert np.all(np.abs(host(st)[:, :3] - rs[:, :3]) <= m_err)
    assert np.all(np.abs(host(st)[:, 3] - rs[:, 3]) <= m_err + 1e-6) and abs(float(loss) - rl) <= m_err + 1e-6
    g = np.where(bad, 0.0, g)
    rH, bH, rW, bW = B.grad_bounds(c.P, g, lp, dt, V > 1000, "f32", m_err, 1.0)
    assert np.all(np.abs(host(dH) - rH) <= bH) and np.all(np.abs(host(dW) - rW) <= bW)
    l2, q2, s2 = c.pair(torch.from_numpy(ref).cuda(), opts, bwd=False)
    assert torch.equal(l2, loss) and torch.equal(q2, qq) and torch.equal(s2, st)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_bad_tokens_in_the_clipped_loss_contribute_nothing(dt):
    """Their term is 0; they stay in the number of rows that the mean divides by."""
    c = Case(2, 2, 60, 64, 200, dt, "ragged", seed=44)
    old, ref = c.old_ref()
    bad = with_bad_tokens(c, c.P.rows[::9])
    adv = c.rng.normal(size=4).astype(np.float32)
    t = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    loss, st, dH, dW = c.clip(t(adv), t(old), t(ref), rg.clip_opts(clip_high=0.28, dw_f32=True))
    assert int(c.status) == 2 and int(c.inf) == 0
    keep = c.P.mask & ~bad
    n_all, n_good = c.P.mask.sum(), keep.sum()
    mask, c.P.mask = c.P.mask, keep
    rl, rs, g, lp = R.clip_loss(c.P, adv, clean(old, mask), clean(ref, mask), c.beta, 0.2, 0.28, False)
    share = n_good / n_all
    qb = R.logp_bound(c.P)
    per = (np.abs(adv).max() * rs[:, 1].max() + c.beta * 6) * qb.max() + 2e-6
    assert abs(float(loss) - share * rl) <= per
    assert not host(st)[~keep].any() and np.all(np.abs(host(st)[:, 0] - rs[:, 0]) <= qb)
    check_q = qb[keep].max()
    rH, bH, rW, bW = B.grad_bounds(c.P, share * g, lp, dt, False, "f32", check_q, 1.0)
    assert np.all(np.abs(host(dH) - rH) <= bH) and np.all(np.abs(host(dW) - rW) <= bW)
    assert not host(dH)[~keep].any()


# ---------------------------------------------------------------- extreme temperatures

@pytest.mark.parametrize("rows", [4, 60])
@pytest.mark.parametrize("T", [1e-4, 1e4, 1e20])
def test_extreme_temperatures(rows, T):
    """Nearly argmax at one end, uniform at the other: the columns that do not count stay out of the sums."""
    c = Case(1, 1, rows, 128, 257, "bf16", "all", T=T, seed=45)
    q, e = c.logp()
    assert int(c.status) == 0
    rq, re, _ = R.logp_entropy(c.P)
    qb = R.logp_bound(c.P) + 4e-7 * np.abs(R.logits(c.P)).max(1)      # the scale of the logits is an fp32 number
    assert np.all(np.abs(host(q) - rq) <= qb)
    if T > 1:
        assert np.all(np.abs(host(e) - re) <= qb * (2 + np.log(257)) + 1e-6 * (1 + np.log(257)))
        dq = np.ones(rows, np.float32)
        dH, dW = c.logp_bwd(torch.from_numpy(dq).cuda(), T, True)
        check(c, dH, dW, dq, R.logp_entropy(c.P)[2], T, True)


@pytest.mark.parametrize("dt,V", [("fp16", 257), ("bf16", 257), ("bf16", 70001)])
@pytest.mark.parametrize("T", [1e-6, 1e-5])
def test_gradients_at_the_lowest_temperatures(dt, V, T):
    """Logits of 1e6 to 1e8: every probability is 0 or 1, in the statistics and in the dlogits alike.  Rows whose two
    largest logits are too close for fp32 to order get no weight."""
    c = Case(1, 2, 100, 64, V, dt, "all", T=T, seed=46)
    order = c.rng.permutation(200)[:100]                 # half of the rows: some other row's token, an improbable one
    c.tok = c.tok.clone()
    c.tok[torch.from_numpy(order).cuda()] = (c.tok[torch.from_numpy(order).cuda()] + 11) % V
    c.P.tokens = c.tok.cpu().numpy()
    rq, _, lp = R.logp_entropy(c.P)
    two = np.partition(lp, -2, axis=1)[:, -2:]
    sure = (two[:, 1] - two[:, 0]) > 100 + 2 * R.logp_bound(c.P)
    assert sure.mean() > 0.8 and (rq[sure] < -1000).any() and (rq[sure] > -1e-9).any()
    q, _ = c.logp()
    assert np.all(np.abs(host(q) - rq) <= R.logp_bound(c.P) + 4e-7 * np.abs(R.logits(c.P)).max(1))
    dq = sure.astype(np.float32)
    scale = float(np.float32(T))
    dH, dW = c.logp_bwd(torch.from_numpy(dq).cuda(), scale, True)
    assert int(c.status) == 0 and int(c.inf) == 0
    # a sure row's dlogits are +-1 or 0 exactly; the functions and the scale are a few steps of fp32 off
    rH, bH, rW, bW = B.grad_bounds(c.P, dq.astype(np.float64), lp, dt, False, "f32", 8 * B.STEP32, scale)
    assert np.all(np.abs(host(dH) - rH) <= bH), np.max(np.abs(host(dH) - rH) / bH)
    assert np.all(np.abs(host(dW) - rW) <= bW), np.max(np.abs(host(dW) - rW) / bW)


# ---------------------------------------------------------------- the tensor cores' rounding towards zero

@pytest.mark.parametrize("place", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("N", [9728, 1024])
def test_dh_is_not_too_small_by_the_place_of_the_token(N, dt, place):
    """dH against 64 bits along dH itself, where element-wise roundings average out: given tokens at the start of the
    vocabulary, whose terms all later additions round down, in its middle and at its end.  9728 rows: whole sums over the
    vocabulary; 1024: sums in pieces.  The loss is 3.2e-8 to 3.4e-8 for each of up to 6272 additions (0.2e-8 of it left:
    1.3e-5); the roundings of 1024 rows' largest dlogits, 1.4e-4 each on average, leave 0.5e-5 (three times that)."""
    d, V, span = 512, 100352, 4096
    g = torch.Generator(device="cuda").manual_seed(47)
    dtype = {"bf16": torch.bfloat16, "fp16": torch.float16}[dt]

    def randn(*s):
        return torch.randn(*s, device="cuda", generator=g)
    W = (randn(V, d) * d ** -0.5).to(dtype)
    lo = int(place * (V - span))
    tok = torch.randint(lo, lo + span, (N,), device="cuda", generator=g, dtype=torch.int32)
    h = (randn(N, d) + (2 + 10 * torch.rand(N, 1, device="cuda", generator=g)) * W[tok.long()].float()).to(dtype)
    dq = randn(N)
    shape = rg.make_shape(1, 1, N, d, V, rg.BF16 if dt == "bf16" else rg.FP16)
    ws = torch.empty(rg.grpo_policy_workspace_bytes(shape, "logp_grad"), dtype=torch.uint8, device="cuda")
    mask = torch.ones(N, dtype=torch.uint8, device="cuda")
    dH, dW = torch.empty_like(h), torch.empty_like(W)
    status, inf = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    rg.grpo_logprobs_bwd(h, W, tok, mask, dq, shape, 1.0, 64.0, ws, dH, dW, inf, status)
    assert int(status) == 0 and int(inf) == 0
    W64, dot, square = W.double(), 0.0, 0.0
    for r in torch.arange(N, device="cuda").split(1024):
        p = torch.softmax(h[r].double() @ W64.t(), 1).neg_()
        p[torch.arange(len(r), device="cuda"), tok[r].long()] += 1
        want = (64.0 * dq[r].double()[:, None] * p) @ W64
        dot += float((dH[r].double() * want).sum())
        square += float((want * want).sum())
    assert abs(dot / square - 1) < 3e-5
