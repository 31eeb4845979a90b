"""Log-probs, clipped policy loss and preference loss on the GPU against their fp64 definitions, element by element,
within bounds counted from the roundings the operators make (head_reference.py)."""
import ctypes

import numpy as np
import pytest

import head_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import rl_fine_tuning_gb300 as rg  # noqa: E402

TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16}
CODE = {"bf16": rg.BF16, "fp16": rg.FP16}


def host(x):
    return x.double().cpu().numpy()


class Case:
    """Random inputs on the device, and their exact values as a reference problem."""

    def __init__(self, n_groups, G, L, d, V, dtype="bf16", mask="ragged", T=1.0, seed=0, chunk_rows=0, likely=True,
                 beta=0.04, loss_mode=0, hscale=1.0):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        N, n = n_groups * G * L, n_groups * G
        W = (torch.randn(V, d, generator=g) * d ** -0.5).to(TORCH[dtype])
        tok = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
        h = hscale * torch.randn(N, d, generator=g)
        if likely:
            h = h + (2 + 10 * torch.rand(N, 1, generator=g)) * W[tok.long()].float()
        h = h.to(TORCH[dtype])
        if mask == "ragged":
            lens = rng.integers(0, L + 1, n)
            lens[rng.integers(0, n)] = L
            m = (np.arange(L)[None] < lens[:, None]).reshape(-1)
        elif mask == "holes":
            m = rng.random(N) < 0.5
        elif mask == "none":
            m = np.zeros(N, bool)
        elif mask == "one":
            m = np.zeros(N, bool)
            m[N // 2] = True
        else:
            m = np.ones(N, bool)
        self.P = R.Problem(n_groups, G, L, h.double().numpy(), W.double().numpy(), tok.numpy(), m, float(np.float32(T)))
        self.dtype, self.T, self.n = dtype, T, n
        self.shape = rg.make_shape(n_groups, G, L, d, V, CODE[dtype], beta=beta, chunk_rows=chunk_rows, loss_mode=loss_mode)
        self.beta = float(np.float32(beta))
        self.seq_mean = bool(loss_mode)
        self.h, self.W, self.tok = h.cuda(), W.cuda(), tok.cuda()
        self.mask = torch.from_numpy(m.astype(np.uint8)).cuda()
        self.status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
        self.inf = torch.full((1,), 9, dtype=torch.int32, device="cuda")
        self.rng = rng

    def ws(self, op, dw_f32=False):
        # 0xFF everywhere: what the operators read of it, they have to write first
        return torch.full((rg.grpo_policy_workspace_bytes(self.shape, op, dw_f32),), 255, dtype=torch.uint8, device="cuda")

    def f32(self, *n):
        return torch.full(n, 7.0, dtype=torch.float32, device="cuda")

    def grads(self, dw_f32=False):
        return (torch.full_like(self.h, 7.0), torch.full_like(self.W, 7.0, dtype=torch.float32 if dw_f32 else self.W.dtype))

    def logp(self, entropy=True, mask=True):
        q, e = self.f32(len(self.tok)), self.f32(len(self.tok)) if entropy else None
        rg.grpo_logprobs(self.h, self.W, self.tok, self.mask if mask else None, self.shape, self.T, self.ws("logp"), q, e,
                         self.status)
        torch.cuda.synchronize()
        return q, e

    def logp_bwd(self, dq, scale=1.0, dw_f32=False):
        dH, dW = self.grads(dw_f32)
        rg.grpo_logprobs_bwd(self.h, self.W, self.tok, self.mask, dq, self.shape, self.T, scale,
                             self.ws("logp_grad", dw_f32), dH, dW, self.inf, self.status, dw_f32=dw_f32)
        torch.cuda.synchronize()
        return dH, dW

    def clip(self, adv, old, ref, opts, scale=1.0, bwd=True):
        loss, st = self.f32(1), self.f32(len(self.tok), 3)
        ws = self.ws("clip", opts.dw_f32)
        if not bwd:
            rg.grpo_clip_loss_fwd(self.h, self.W, self.tok, self.mask, adv, old, ref, self.shape, opts, ws, loss, st,
                                  self.status)
            torch.cuda.synchronize()
            return loss, st
        dH, dW = self.grads(opts.dw_f32)
        rg.grpo_clip_loss_fwd_bwd(self.h, self.W, self.tok, self.mask, adv, old, ref, self.shape, opts, scale, ws, loss, dH,
                                  dW, self.inf, st, self.status)
        torch.cuda.synchronize()
        return loss, st, dH, dW

    def pair(self, ref, opts, scale=1.0, bwd=True):
        loss, q, st = self.f32(1), self.f32(len(self.tok)), self.f32(self.shape.n_groups, 4)
        ws = self.ws("pair", opts.dw_f32)
        if not bwd:
            rg.grpo_pair_loss_fwd(self.h, self.W, self.tok, self.mask, ref, self.shape, opts, ws, loss, q, st, self.status)
            torch.cuda.synchronize()
            return loss, q, st
        dH, dW = self.grads(opts.dw_f32)
        rg.grpo_pair_loss_fwd_bwd(self.h, self.W, self.tok, self.mask, ref, self.shape, opts, scale, ws, loss, dH, dW,
                                  self.inf, q, st, self.status)
        torch.cuda.synchronize()
        return loss, q, st, dH, dW

    def old_ref(self, spread=0.15, away=1e-3, lo=0.2, hi=0.28):
        """Stored log-probs whose ratios stay `away` from the clip borders (fp32 values, exact in the reference)."""
        q = R.logp_entropy(self.P)[0]
        lr = spread * self.rng.normal(size=len(q))
        near = (np.abs(np.exp(lr) - (1 - lo)) < away) | (np.abs(np.exp(lr) - (1 + hi)) < away)
        old = (q - np.where(near, lr + 5 * away, lr)).astype(np.float32)
        ref = (q + 0.3 * self.rng.normal(size=len(q))).astype(np.float32)
        # masked rows are never read: not even a NaN there may show
        old[~self.P.mask] = np.nan
        ref[~self.P.mask] = np.inf
        return old, ref


def clean(x, mask):
    return np.where(mask, np.nan_to_num(x.astype(np.float64), posinf=0, neginf=0), 0.0)


def check_logp(c, q, ent):
    rq, re, _ = R.logp_entropy(c.P)
    bound = R.logp_bound(c.P)
    assert int(c.status) == 0
    assert np.all(np.abs(host(q) - rq) <= bound), np.max(np.abs(host(q) - rq) / bound)
    assert not host(q)[~c.P.mask].any()
    if ent is not None:
        V = c.P.W.shape[0]
        eb = bound * (2 + np.log(V)) + 1e-6 * (1 + np.abs(R.logits(c.P)).max(1))
        assert np.all(np.abs(host(ent) - re) <= eb), np.max(np.abs(host(ent) - re) / eb)
        assert not host(ent)[~c.P.mask].any()


def check_grads(c, dH, dW, g, lp, scale=1.0, dw_f32=False):
    rH, rW, aH, aW = R.gradients(c.P, g, lp)
    q_err = R.logp_bound(c.P).max()
    assert int(c.status) == 0 and int(c.inf) == 0
    bH = R.grad_bound(scale * rH, scale * aH, c.dtype, c.dtype, q_err, scale)
    bW = R.grad_bound(scale * rW, scale * aW, c.dtype, "f32" if dw_f32 else c.dtype, q_err, scale)
    eH, eW = np.abs(host(dH) - scale * rH), np.abs(host(dW) - scale * rW)
    assert np.all(eH <= bH), ("dH", np.max(eH / bH))
    assert np.all(eW <= bW), ("dW", np.max(eW / bW))
    assert not host(dH)[~c.P.mask].any()


# (n_groups, G, L, d, V, dtype, mask, chunk_rows)
SHAPES = [
    (1, 1, 1, 64, 1, "bf16", "all", 0),            # one token, a vocabulary of one: q = 0, no gradient
    (1, 1, 1, 64, 7, "fp16", "all", 0),
    (1, 2, 3, 128, 257, "bf16", "holes", 0),       # the few-row kernel, masked rows among them
    (1, 8, 2, 192, 1000, "fp16", "all", 0),
    (1, 17, 1, 320, 389, "bf16", "all", 0),        # 17 rows: the wider few-row kernel
    (1, 32, 1, 64, 130, "bf16", "ragged", 0),
    (1, 33, 1, 64, 130, "bf16", "ragged", 0),      # one row more: the chunked path
    (2, 4, 37, 320, 1000, "bf16", "ragged", 0),
    (1, 3, 211, 128, 515, "fp16", "holes", 128),   # five chunks
    (1, 2, 300, 576, 333, "bf16", "all", 256),
    (1, 1, 700, 64, 2049, "bf16", "ragged", 384),
    (3, 2, 41, 1088, 64, "fp16", "ragged", 0),
    (1, 4, 50, 128, 700, "bf16", "none", 0),       # no row counts
    (1, 4, 50, 128, 700, "bf16", "one", 128),
]


@pytest.mark.parametrize("s", SHAPES, ids=str)
@pytest.mark.parametrize("T", [1.0, 0.7])
def test_logprobs(s, T):
    n, G, L, d, V, dt, mask, cr = s
    c = Case(n, G, L, d, V, dt, mask, T, seed=1, chunk_rows=cr)
    check_logp(c, *c.logp())
    q, _ = c.logp(entropy=False)
    check_logp(c, q, None)
    if mask == "all":
        assert torch.equal(c.logp(mask=False)[0], c.logp()[0])


def test_logprobs_are_exact_enough_to_sum():
    """Sums of q over a completion: the tensor cores' rounding towards zero, left in, makes every logit of about 11 at
    d = 4096 some 4e-5 too small; here the sum over 512 rows stays within 512 times 2e-6, the other roundings' size."""
    c = Case(1, 1, 512, 4096, 1031, "bf16", "all", seed=5)
    q, e = c.logp()
    check_logp(c, q, e)
    assert abs((host(q) - R.logp_entropy(c.P)[0]).sum()) <= 512 * 2e-6


@pytest.mark.parametrize("s", SHAPES, ids=str)
@pytest.mark.parametrize("dw_f32", [False, True])
def test_logprobs_bwd(s, dw_f32):
    n, G, L, d, V, dt, mask, cr = s
    c = Case(n, G, L, d, V, dt, mask, 1.3, seed=2, chunk_rows=cr)
    dq = c.rng.normal(size=len(c.tok)).astype(np.float32)
    dq[~c.P.mask] = np.nan
    dH, dW = c.logp_bwd(torch.from_numpy(dq).cuda(), 64.0, dw_f32)
    check_grads(c, dH, dW, clean(dq, c.P.mask), R.logp_entropy(c.P)[2], 64.0, dw_f32)


@pytest.mark.parametrize("size", [1e-7, 1.0, 1e4])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_logprobs_bwd_scales_with_its_input(size, dt):
    """d loss / d q of any size: the fp16 dlogits keep their precision, the loss scale only places the outputs."""
    c = Case(1, 2, 60, 128, 500, dt, "ragged", seed=3)
    dq = (size * c.rng.normal(size=len(c.tok))).astype(np.float32)
    dH, dW = c.logp_bwd(torch.from_numpy(dq).cuda(), 1.0 / size)
    check_grads(c, dH, dW, clean(dq, c.P.mask), R.logp_entropy(c.P)[2], 1.0 / size)


@pytest.mark.parametrize("s", SHAPES, ids=str)
@pytest.mark.parametrize("beta,loss_mode,T", [(0.04, 0, 1.0), (0.0, 1, 1.5)])
def test_clip_loss(s, beta, loss_mode, T):
    n, G, L, d, V, dt, mask, cr = s
    c = Case(n, G, L, d, V, dt, mask, T, seed=4, chunk_rows=cr, beta=beta, loss_mode=loss_mode)
    old, ref = c.old_ref()
    adv = c.rng.normal(size=c.n).astype(np.float32)
    adv[::3] = 0.0
    opts = rg.clip_opts(temperature=T, clip_low=0.2, clip_high=0.28)
    scale = 256.0 if dt == "fp16" else 1.0
    t = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    loss, st, dH, dW = c.clip(t(adv), t(old), t(ref) if beta else None, opts, scale)
    rl, rs, g, lp = R.clip_loss(c.P, adv, clean(old, c.P.mask), clean(ref, c.P.mask), c.beta, 0.2, 0.28, c.seq_mean)
    qb = R.logp_bound(c.P)
    sb = np.stack([qb, (qb + 4e-7) * rs[:, 1], qb * np.abs(np.expm1(0.3 * 6)) + 1e-6], 1)
    assert np.all(np.abs(host(st) - rs) <= sb * c.P.mask[:, None]), np.max(np.abs(host(st) - rs) / (sb + 1e-30))
    per = (np.abs(adv).max(initial=0) * rs[:, 1].max(initial=0) + c.beta * 6) * qb.max() + 2e-6
    assert abs(float(loss) - rl) <= per
    check_grads(c, dH, dW, g, lp, scale)
    l2, s2 = c.clip(t(adv), t(old), t(ref) if beta else None, opts, bwd=False)
    assert torch.equal(l2, loss) and torch.equal(s2, st)


@pytest.mark.parametrize("A,r,kept", [(1.0, 2.0, False), (1.0, 0.5, True), (-1.0, 2.0, True), (-1.0, 0.5, False),
                                      (0.0, 2.0, True)])
def test_clip_cuts_on_the_right_side(A, r, kept):
    c = Case(1, 1, 40, 64, 100, "bf16", "all", seed=6, beta=0.0)
    q = R.logp_entropy(c.P)[0]
    old = torch.from_numpy((q - np.log(r)).astype(np.float32)).cuda()
    _, st, dH, dW = c.clip(torch.full((1,), A, device="cuda"), old, None, rg.clip_opts())
    assert bool(dH.any()) == (kept and A != 0) and bool(dW.any()) == (kept and A != 0)
    np.testing.assert_allclose(host(st)[:, 1], r, rtol=1e-4)


def test_clip_without_an_upper_border():
    c = Case(1, 1, 40, 64, 100, "bf16", "all", seed=6, beta=0.0)
    old = torch.from_numpy((R.logp_entropy(c.P)[0] - 2).astype(np.float32)).cuda()
    _, _, dH, _ = c.clip(torch.ones(1, device="cuda"), old, None, rg.clip_opts(clip_high=float("inf")))
    assert bool(dH.any())


PAIRS = [(n, L, d, V, dt, mask, cr) for n, L, d, V, dt, mask, cr in [
    (1, 1, 64, 5, "bf16", "all", 0),
    (3, 37, 128, 515, "bf16", "ragged", 0),
    (5, 50, 320, 300, "fp16", "holes", 128),       # one pair a chunk
    (7, 30, 192, 260, "bf16", "ragged", 256),      # several pairs a chunk, uneven
    (2, 150, 128, 700, "bf16", "ragged", 128),     # a pair does not fit: the logits twice
    (2, 150, 128, 700, "fp16", "all", 256),
    (4, 20, 64, 130, "bf16", "none", 0),
    (4, 20, 64, 130, "bf16", "one", 0),
]]


@pytest.mark.parametrize("s", PAIRS, ids=str)
@pytest.mark.parametrize("kind,e,mean,beta", [("sigmoid", 0.0, False, 0.1), ("sigmoid", 0.1, True, 2.0),
                                              ("hinge", 0.0, False, 0.05), ("square", 0.0, True, 0.5)])
def test_pair_loss(s, kind, e, mean, beta):
    n, L, d, V, dt, mask, cr = s
    c = Case(n, 2, L, d, V, dt, mask, seed=7, chunk_rows=cr, beta=beta)
    _, ref = c.old_ref()
    opts = rg.pair_opts(kind, e, mean)
    scale = 16.0 if dt == "fp16" else 1.0
    ref_d = torch.from_numpy(ref).cuda()
    loss, q, st, dH, dW = c.pair(ref_d, opts, scale)
    rl, rs, g, lp = R.pair_loss(c.P, clean(ref, c.P.mask), c.beta, kind, float(np.float32(e)), mean)
    check_logp(c, q, None)
    qb = R.logp_bound(c.P).max() + 1e-7 * np.abs(lp[np.arange(len(ref)), c.P.tokens]).max()
    S_err = (1 if mean else L) * qb
    step = max(1.0, np.abs(rs).max())
    assert np.all(np.abs(host(st)[:, :3] - rs[:, :3]) <= 2 * c.beta * S_err + 1e-6 * step)
    slope = 1.0 if kind != "square" else 2 * np.abs(rs[:, 2] / c.beta - 0.5 / c.beta).max() / c.beta + 1
    lb = slope * (2 * c.beta * S_err) + 1e-6 * step
    assert abs(float(loss) - rl) <= lb and np.all(np.abs(host(st)[:, 3] - rs[:, 3]) <= lb)
    # d loss / d q moves with the margin: its error is that of q times the curvature, at most 1 (square: 2)
    extra = (2 * c.beta * S_err) * 2 / max(1e-30, 1.0)
    rH, rW, aH, aW = R.gradients(c.P, g, lp)
    full = np.where(c.P.mask, (2 if kind == "square" else c.beta) / np.maximum(1, int(c.P.mask.any())), 0.0)
    _, _, xH, xW = R.gradients(c.P, full, lp)
    assert int(c.status) == 0 and int(c.inf) == 0
    qe = R.logp_bound(c.P).max()
    bH = R.grad_bound(scale * rH, scale * aH, dt, dt, qe, scale) + scale * extra * xH
    bW = R.grad_bound(scale * rW, scale * aW, dt, dt, qe, scale) + scale * extra * xW
    assert np.all(np.abs(host(dH) - scale * rH) <= bH)
    assert np.all(np.abs(host(dW) - scale * rW) <= bW)
    assert not host(dH)[~c.P.mask].any()
    l2, q2, s2 = c.pair(ref_d, opts, bwd=False)
    assert torch.equal(l2, loss) and torch.equal(q2, q) and torch.equal(s2, st)


@pytest.mark.parametrize("mask", ["ragged", "none"])
def test_pair_chunkings_agree(mask):
    """Whole pairs in one chunk, in several, and the logits twice: the same loss and log-probs, gradients within a rounding."""
    outs = []
    for cr in (0, 256, 128):
        c = Case(6, 2, 80, 128, 300, "bf16", mask, seed=8, chunk_rows=cr, beta=0.1)
        _, ref = c.old_ref()
        outs.append(c.pair(torch.from_numpy(ref).cuda(), rg.pair_opts()))
    for o in outs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(o[:3], outs[0][:3]))
        for k in (3, 4):
            torch.testing.assert_close(o[k].float(), outs[0][k].float(), rtol=2 ** -7, atol=1e-6)


def test_results_do_not_depend_on_the_workspace_or_the_stream():
    c = Case(2, 3, 120, 192, 600, "bf16", "ragged", seed=9, chunk_rows=256)
    old, ref = (torch.from_numpy(x).cuda() for x in c.old_ref())
    adv = torch.randn(6, device="cuda")
    a = c.clip(adv, old, ref, rg.clip_opts())
    b = c.clip(adv, old, ref, rg.clip_opts())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        d = c.clip(adv, old, ref, rg.clip_opts())
    for x, y, z in zip(a, b, d):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_calls_on_two_streams_at_once():
    """Two clipped steps and a few-row call in flight together, each with its own workspace: the bits of the calls alone."""
    cs = [Case(2, 3, 120, 192, 600, "bf16", "ragged", seed=s, chunk_rows=256) for s in (13, 14)]
    few = Case(1, 4, 1, 128, 400, "bf16", "all", seed=15)
    opts = rg.clip_opts()
    ins = [[torch.from_numpy(x).cuda() for x in c.old_ref()] + [torch.randn(6, device="cuda")] for c in cs]
    outs = [[c.ws("clip"), c.f32(1), *c.grads(), c.f32(len(c.tok), 3)] for c in cs]
    fws, fq = few.ws("logp"), few.f32(4)

    def call(k):
        c, (old, ref, adv), (ws, loss, dH, dW, st) = cs[k], ins[k], outs[k]
        rg.grpo_clip_loss_fwd_bwd(c.h, c.W, c.tok, c.mask, adv, old, ref, c.shape, opts, 1.0, ws, loss, dH, dW, c.inf, st,
                                  c.status)

    def call_few():
        rg.grpo_logprobs(few.h, few.W, few.tok, None, few.shape, 1.0, fws, fq, None, few.status)

    want = []
    for k in (0, 1):
        call(k)
        torch.cuda.synchronize()
        want.append([x.clone() for x in outs[k][1:]])
    call_few()
    torch.cuda.synchronize()
    want_q = fq.clone()
    for x in (*outs[0], *outs[1], fws, fq):
        x.zero_()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                call(k)
        with torch.cuda.stream(streams[2]):
            call_few()
    torch.cuda.synchronize()
    for k in (0, 1):
        assert all(torch.equal(x, y) for x, y in zip(outs[k][1:], want[k]))
        assert int(cs[k].status) == 0
    assert torch.equal(fq, want_q) and int(few.status) == 0


@pytest.mark.parametrize("loss_mode", [0, 1])
def test_shards_add_up_to_the_batch(loss_mode):
    """Prompt groups on two shards, loss and gradients weighted by the shard's share of what the mean counts."""
    c = Case(4, 2, 60, 128, 400, "bf16", "ragged", seed=16, loss_mode=loss_mode)
    old, ref = (torch.from_numpy(x).cuda() for x in c.old_ref())
    adv = torch.randn(8, device="cuda")
    opts = rg.clip_opts(clip_high=0.28, dw_f32=True)
    loss, _, dH, dW = c.clip(adv, old, ref, opts)
    counts = lambda m: (m.view(-1, 60).any(1) if loss_mode else m).ne(0).sum().item()  # noqa: E731
    total, sum_loss, sum_dW, rows = counts(c.mask), 0.0, torch.zeros_like(dW), []
    shape = rg.make_shape(2, 2, 60, 128, 400, CODE["bf16"], beta=c.beta, loss_mode=loss_mode)
    ws = torch.full((rg.grpo_policy_workspace_bytes(shape, "clip", True),), 255, dtype=torch.uint8, device="cuda")
    for r in (slice(0, 240), slice(240, 480)):
        h, tok, mask = c.h[r].contiguous(), c.tok[r].contiguous(), c.mask[r].contiguous()
        w = counts(mask) / total
        part, gH, gW = c.f32(1), torch.empty_like(h), torch.empty_like(dW)
        rg.grpo_clip_loss_fwd_bwd(h, c.W, tok, mask, adv[r.start // 60:r.stop // 60].contiguous(), old[r].contiguous(),
                                  ref[r].contiguous(), shape, opts, w, ws, part, gH, gW, c.inf, None, c.status)
        torch.cuda.synchronize()
        assert int(c.status) == 0 and int(c.inf) == 0
        sum_loss += w * part.item()
        sum_dW += gW
        rows.append(gH)
    # loss: fp32 sums of terms of order 1, whose q differ by fp32 roundings of logits below 64 (4e-6 each); gradients: two
    # 16-bit roundings on each side (dlogits and the output, or dlogits and the scaled row)
    assert abs(sum_loss - loss.item()) <= 1e-5 * (1 + abs(loss.item()))
    for got, want in ((torch.cat(rows).float(), dH.float()), (sum_dW, dW)):
        assert (got - want).norm() <= 4 * 2 ** -8 * want.norm()


def test_graph_replays_on_new_inputs():
    c = Case(2, 2, 90, 128, 400, "bf16", "ragged", seed=10, chunk_rows=128, beta=0.1)
    c2 = Case(2, 2, 90, 128, 400, "bf16", "holes", seed=11, chunk_rows=128, beta=0.1)
    _, ref = c.old_ref()
    ref = torch.from_numpy(clean(ref, c.P.mask).astype(np.float32)).cuda()
    ws, loss, q, st = c.ws("pair"), c.f32(1), c.f32(360), c.f32(2, 4)
    dH, dW = c.grads()
    few = Case(1, 4, 1, 128, 400, "bf16", "all", seed=12)
    fws, fq = few.ws("logp"), few.f32(4)

    def call():
        rg.grpo_pair_loss_fwd_bwd(c.h, c.W, c.tok, c.mask, ref, c.shape, rg.pair_opts(), 1.0, ws, loss, dH, dW, c.inf, q, st,
                                  c.status)
        rg.grpo_logprobs(few.h, few.W, few.tok, None, few.shape, 1.0, fws, fq, None, few.status)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for src in (c, c2):
        for name in ("h", "W", "tok", "mask"):
            getattr(c, name).copy_(getattr(src, name))
        few.h.copy_(src.h[:4])
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (loss, q, st, dH, dW, fq)]
        call()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, (loss, q, st, dH, dW, fq)))
        assert int(c.status) == 0 and int(few.status) == 0


@pytest.mark.parametrize("rows", [4, 100])
def test_a_bad_token_is_reported_and_contributes_nothing(rows):
    c = Case(1, 1, rows, 128, 200, "bf16", "all", seed=13)
    bad = c.tok.clone()
    bad[1], bad[2] = 200, -1
    c.tok, good = bad, c.tok
    q, e = c.logp()
    assert int(c.status) == 2 and host(q)[1] == host(q)[2] == host(e)[1] == 0
    dq = torch.ones(rows, device="cuda")
    dH, dW = c.logp_bwd(dq)
    assert int(c.status) == 2 and not dH[1].any() and not dH[2].any()
    c.tok = good
    c.P.mask[1:3] = False
    keep = np.ones(rows, bool)
    keep[1:3] = False
    rH, _, aH, _ = R.gradients(c.P, np.ones(rows), R.logp_entropy(c.P)[2])
    bH = R.grad_bound(rH, aH, "bf16", "bf16", 1e-4, 1.0)
    assert np.all(np.abs(host(dH) - rH)[keep] <= bH[keep])


def test_found_inf_is_set_when_a_gradient_leaves_the_type():
    c = Case(1, 1, 64, 128, 300, "fp16", "all", seed=14)
    dq = torch.ones(64, device="cuda")
    c.logp_bwd(dq, 1.0)
    assert int(c.inf) == 0
    c.logp_bwd(dq, 1e7)
    assert int(c.inf) == 1
    c.logp_bwd(dq * float("inf"), 1.0)
    assert int(c.inf) == 1


def test_mask_at_any_address_and_of_any_nonzero_value():
    c = Case(1, 3, 100, 64, 130, "bf16", "holes", seed=15)
    want, _ = c.logp()
    buf = torch.zeros(301, dtype=torch.uint8, device="cuda")
    buf[1:] = c.mask * 200
    c.mask = buf[1:]
    assert torch.equal(c.logp()[0], want)


def test_checked_build_finds_no_bad_index():
    from rl_fine_tuning_gb300 import build
    lib = ctypes.CDLL(build.LIB_CHECKED)
    rg._declare(lib)
    normal, rg._lib = rg.load(), lib
    try:
        for cr, G, L, V, d in ((0, 2, 100, 500, 128), (128, 2, 100, 500, 128), (256, 2, 40, 500, 128),
                               (0, 2, 100, 9000, 128), (128, 2, 100, 40000, 128), (0, 2, 1500, 2049, 1280)):
            c = Case(3, G, L, d, V, "bf16", "ragged", seed=16, chunk_rows=cr, beta=0.1)
            old, ref = (torch.from_numpy(x).cuda() for x in c.old_ref())
            check_logp(c, *c.logp())
            c.clip(torch.randn(c.n, device="cuda"), old, ref, rg.clip_opts())
            assert int(c.status) == 0
            c.pair(ref, rg.pair_opts())
            assert int(c.status) == 0
    finally:
        rg._lib = normal


def test_the_binding_refuses_what_the_c_interface_cannot_see():
    c = Case(1, 2, 10, 64, 100, "bf16", "all", seed=17)
    q = c.f32(20)
    call = lambda h=c.h, W=c.W, tok=c.tok, out=q: rg.grpo_logprobs(h, W, tok, c.mask, c.shape, 1.0, c.ws("logp"), out,  # noqa: E731
                                                                   None, c.status)
    call()
    wide = torch.zeros(20, 128, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(h=wide[:, ::2]), dict(h=c.h.float()), dict(h=c.h[:19]), dict(tok=c.tok.long()), dict(W=c.W.cpu()),
               dict(out=q.double()), dict(W=torch.empty(64, 100, dtype=torch.bfloat16, device="cuda").t())):
        with pytest.raises(ValueError):
            call(**kw)


def far_case(n_groups, G, L, V, chunk_rows, n_far, seed, **kw):
    """Large enough for dlogits relative to the token's logit (rows x V >= 2^24); n_far rows where another token is
    about 100 nats above the given one, which that form cannot hold."""
    c = Case(n_groups, G, L, 64, V, "bf16", "ragged", seed=seed, chunk_rows=chunk_rows, **kw)
    rows = c.P.rows[:: max(1, len(c.P.rows) // max(1, n_far))][:n_far]
    W = c.W.float().cpu()
    for t in rows:
        o = (int(c.tok[t]) + 17) % V
        c.h[t] = (100.0 * W[o] / float(W[o] @ W[o]) - 20.0 * W[int(c.tok[t])]).to(torch.bfloat16).cuda()
    c.P.h = c.h.double().cpu().numpy()
    return c


@pytest.mark.parametrize("n_far", [0, 1, 40])
@pytest.mark.parametrize("chunk_rows", [0, 128])
def test_relative_dlogits_clip(n_far, chunk_rows):
    c = far_case(1, 2, 125, 70001 if chunk_rows == 0 else 131080, chunk_rows, n_far, 20)
    adv = np.array([1.5, -0.75], np.float32)
    old, ref = c.old_ref()
    t = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    opts = rg.clip_opts(clip_high=0.28)
    loss, st, dH, dW = c.clip(t(adv), t(old), t(ref), opts)
    rl, rs, g, lp = R.clip_loss(c.P, adv, clean(old, c.P.mask), clean(ref, c.P.mask), c.beta, 0.2, 0.28, False)
    assert n_far == 0 or rs[:, 0].min() < -80
    qb = R.logp_bound(c.P)
    assert np.all(np.abs(host(st)[:, 0] - rs[:, 0]) <= qb * c.P.mask)
    assert abs(float(loss) - rl) <= (1.5 * rs[:, 1].max() + c.beta * 6) * qb.max() + 2e-6
    check_grads(c, dH, dW, g, lp)
    l2, s2 = c.clip(t(adv), t(old), t(ref), opts, bwd=False)
    assert torch.equal(l2, loss) and torch.equal(s2, st)


@pytest.mark.parametrize("n_far", [0, 3])
@pytest.mark.parametrize("chunk_rows", [0, 128, 256])
def test_relative_dlogits_pair(n_far, chunk_rows):
    c = far_case(2, 2, 90, 131080, chunk_rows, n_far, 21, beta=0.1)
    _, ref = c.old_ref()
    loss, q, st, dH, dW = c.pair(torch.from_numpy(ref).cuda(), rg.pair_opts())
    rl, rs, g, lp = R.pair_loss(c.P, clean(ref, c.P.mask), c.beta)
    check_logp(c, q, None)
    S_err = 90 * R.logp_bound(c.P).max()
    assert abs(float(loss) - rl) <= 2 * c.beta * S_err + 1e-6
    rH, rW, aH, aW = R.gradients(c.P, g, lp)
    rel = 2 * c.beta * S_err   # d log |sigmoid(-m)| / dm is at most 1
    assert np.all(np.abs(host(dH) - rH) <= R.grad_bound(rH, (1 + rel) * aH, "bf16", "bf16", 1e-4 + rel, 1.0))
    assert np.all(np.abs(host(dW) - rW) <= R.grad_bound(rW, (1 + rel) * aW, "bf16", "bf16", 1e-4 + rel, 1.0))
    l2, q2, s2 = c.pair(torch.from_numpy(ref).cuda(), rg.pair_opts(), bwd=False)
    assert torch.equal(l2, loss) and torch.equal(q2, q) and torch.equal(s2, st)


def test_relative_dlogits_of_given_gradients_and_bad_tokens():
    c = far_case(1, 1, 250, 70001, 0, 2, 22)
    dq = torch.randn(250, generator=torch.Generator().manual_seed(1))
    dH, dW = c.logp_bwd(dq.cuda(), 8.0, True)
    check_grads(c, dH, dW, clean(dq.numpy(), c.P.mask), R.logp_entropy(c.P)[2], 8.0, True)
    c = far_case(1, 1, 250, 70001, 0, 0, 23)
    c.tok = c.tok.clone()
    c.tok[3], c.tok[4] = 70001, -5
    dH, dW = c.logp_bwd(dq.cuda())
    assert int(c.status) == 2 and int(c.inf) == 0 and not dH[3:5].any() and bool(torch.isfinite(dW.float()).all())


def test_example_runs_the_operators_together():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "off_policy_steps.py")
    spec = importlib.util.spec_from_file_location("off_policy_steps", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    out = m.main(["--d", "128", "--V", "1000", "--L", "40", "--steps", "3"])
    assert out["clip"]["losses"][-1] < out["clip"]["losses"][0]
    assert out["pair"]["losses"][-1] < out["pair"]["losses"][0]
    assert all(np.isfinite(x) and x < 0 for x in out["token"])


def test_nan_in_rows_that_do_not_count_stays_there():
    """Masked rows of h, the stored log-probs of masked rows and the advantage of an empty completion are never used."""
    for rows in (4, 60):
        c = Case(1, 3, rows // 2, 128, 300, "bf16", "all", seed=30)
        c.P.mask[: rows // 2] = False                 # completion 0 is empty
        c.P.mask[-1] = False
        c.mask = torch.from_numpy(c.P.mask.astype(np.uint8)).cuda()
        c.h[~torch.from_numpy(c.P.mask)] = float("nan")
        old, ref = c.old_ref()
        q, e = c.logp()
        check_logp(c, q, e)
        adv = torch.tensor([float("nan"), 1.0, -1.0], device="cuda")
        loss, st, dH, dW = c.clip(adv, torch.from_numpy(old).cuda(), torch.from_numpy(ref).cuda(), rg.clip_opts())
        assert int(c.inf) == 0 and bool(torch.isfinite(loss)) and bool(torch.isfinite(dW.float()).all())
        assert not host(dH)[~c.P.mask].any()


def test_nan_in_a_row_that_counts_is_reported():
    c = Case(1, 1, 60, 128, 300, "bf16", "all", seed=31)
    c.h[5] = float("nan")
    q, _ = c.logp()
    assert np.isnan(host(q)[5]) and np.isfinite(np.delete(host(q), 5)).all()
    dq = torch.ones(60, device="cuda")
    dH, _ = c.logp_bwd(dq)
    assert int(c.inf) == 1 and int(c.status) == 0
    assert bool(torch.isfinite(dH[torch.arange(60) != 5].float()).all())


def test_offsets_past_32_bits():
    """A chunk of 19456 rows x 131072 columns: 2.55e9 dlogits.  Sampled rows and columns against fp64 on the GPU."""
    L, d, V = 9728, 64, 131072
    g = torch.Generator(device="cuda").manual_seed(3)
    N = 2 * L
    W = (torch.randn(V, d, device="cuda", generator=g) * d ** -0.5).bfloat16()
    tok = torch.randint(0, V, (N,), device="cuda", generator=g, dtype=torch.int32)
    h = (torch.randn(N, d, device="cuda", generator=g) + 8 * W[tok.long()].float()).bfloat16()
    mask = torch.ones(N, dtype=torch.uint8, device="cuda")
    ref = torch.full((N,), -1.0, device="cuda")
    shape = rg.make_shape(1, 2, L, d, V, beta=0.01)
    ws = torch.full((rg.grpo_policy_workspace_bytes(shape, "pair"),), 255, dtype=torch.uint8, device="cuda")
    dH, dW = torch.full_like(h, 7.0), torch.full_like(W, 7.0)
    loss, q, st = torch.empty(1, device="cuda"), torch.empty(N, device="cuda"), torch.empty(1, 4, device="cuda")
    status, inf = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    rg.grpo_pair_loss_fwd_bwd(h, W, tok, mask, ref, shape, rg.pair_opts(length_mean=True), 1024.0, ws, loss, dH, dW, inf, q, st,
                              status)
    torch.cuda.synchronize()
    assert int(status) == 0 and int(inf) == 0
    H, W64 = h.double(), W.double()
    q64, p_cols, parts = torch.empty(N, dtype=torch.float64, device="cuda"), [], []
    cols = torch.cat([torch.arange(32, device="cuda"), torch.arange(V - 32, V, device="cuda"), tok[-64:].long()])
    rows = torch.cat([torch.arange(64, device="cuda"), torch.arange(N - 64, N, device="cuda")])
    for r in torch.arange(N, device="cuda").split(512):
        z = H[r] @ W64.t()
        lp = z - torch.logsumexp(z, 1, keepdim=True)
        q64[r] = lp.gather(1, tok[r].long()[:, None])[:, 0]
        p_cols.append(lp[:, cols].exp())
        parts.append(lp[(r[:, None] == rows[None]).any(1)].exp())
    assert float((q.double() - q64).abs().max()) < 1e-5
    S = (q64 - ref.double()).reshape(2, L).mean(1)
    m = 0.01 * (S[0] - S[1])
    c = 0.01 * -torch.sigmoid(-m) / L * 1024.0
    gq = torch.cat([c.expand(L), -c.expand(L)])
    one = (tok.long()[:, None] == cols[None]).double()
    rW = ((one - torch.cat(p_cols)) * gq[:, None]).t() @ H
    P = torch.cat(parts)
    P = -P
    P[torch.arange(128, device="cuda"), tok[rows].long()] += 1
    rH = (P * gq[rows][:, None]) @ W64
    for got, want in ((dW[cols].double(), rW), (dH[rows].double(), rH)):
        assert float((got - want).norm() / want.norm()) < 3 * 2 ** -8
        assert float((got - want).abs().max() / want.abs().max()) < 4 * 2 ** -8


@pytest.mark.parametrize("dt,N,d,V,share,cr,dw_f32", [
    ("bf16", 8192, 1280, 2049, 0.03, 0, False),    # relative dlogits, dH and dW in launches of their own
    ("fp16", 8192, 1280, 2049, 0.03, 0, True),     # the dlogits pass
    ("bf16", 512, 5120, 8000, 0.1, 0, False),      # the dlogits pass in bf16
    ("bf16", 8192, 1280, 4100, 0.55, 4096, False),  # two chunks: dW's sum in the workspace
    ("fp16", 8192, 1280, 4100, 0.55, 4096, True),
    ("bf16", 8192, 2560, 2049, 0.03, 0, False),    # dH in units of 512 columns, all of them split
    ("fp16", 8192, 2560, 2049, 0.6, 0, False),     # whole and split ones
])
def test_large_chunks(dt, N, d, V, share, cr, dw_f32):
    """Chunks above the sizes where dH and dW share a launch; few of the rows count, and the reference holds those alone."""
    g = torch.Generator().manual_seed(40)
    rng = np.random.default_rng(40)
    keep = np.flatnonzero(rng.random(N) < share)
    W = (torch.randn(V, d, generator=g) * d ** -0.5).to(TORCH[dt])
    tok = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    h = (torch.randn(N, d, generator=g) + 8 * W[tok.long()].float()).to(TORCH[dt])
    mask = np.zeros(N, np.uint8)
    mask[keep] = 1
    dq = rng.normal(size=N).astype(np.float32)
    P = R.Problem(1, 1, len(keep), h[keep].double().numpy(), W.double().numpy(), tok[keep].numpy(),
                  np.ones(len(keep), bool))
    shape = rg.make_shape(1, 1, N, d, V, CODE[dt], chunk_rows=cr)
    hd, Wd, td, md, dqd = h.cuda(), W.cuda(), tok.cuda(), torch.from_numpy(mask).cuda(), torch.from_numpy(dq).cuda()
    ws = torch.full((rg.grpo_policy_workspace_bytes(shape, "logp_grad", dw_f32),), 255, dtype=torch.uint8, device="cuda")
    status, inf = (torch.full((1,), 9, dtype=torch.int32, device="cuda") for _ in range(2))
    outs = []
    for _ in range(2):
        dH = torch.full_like(hd, 7.0)
        dW = torch.full_like(Wd, 7.0, dtype=torch.float32 if dw_f32 else Wd.dtype)
        rg.grpo_logprobs_bwd(hd, Wd, td, md, dqd, shape, 1.0, 32.0, ws, dH, dW, inf, status, dw_f32=dw_f32)
        torch.cuda.synchronize()
        outs.append((dH, dW))
    assert int(status) == 0 and int(inf) == 0
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    lp = R.logp_entropy(P)[2]
    rH, rW, aH, aW = R.gradients(P, dq[keep].astype(np.float64), lp)
    qe = R.logp_bound(P).max()
    eH, eW = np.abs(host(dH)[keep] - 32 * rH), np.abs(host(dW) - 32 * rW)
    assert np.all(eH <= R.grad_bound(32 * rH, 32 * aH, dt, dt, qe, 32)) and not host(dH)[mask == 0].any()
    assert np.all(eW <= R.grad_bound(32 * rW, 32 * aW, dt, "f32" if dw_f32 else dt, qe, 32))


@pytest.mark.parametrize("size", [1e-12, 1e6])
def test_relative_dlogits_scale_with_their_input(size):
    """Tokens down to q of about -38, and d loss / d q of any size: row factors and relative dlogits stay in bf16's range."""
    c = far_case(1, 1, 250, 70001, 0, 0, 24)
    W = c.W.float().cpu()
    for n, t in enumerate(c.P.rows[::10]):
        o = (int(c.tok[t]) + 29) % 70001
        c.h[t] = ((5.0 + 1.4 * n) * W[o] / float(W[o] @ W[o])).to(torch.bfloat16).cuda()
    c.P.h = c.h.double().cpu().numpy()
    q, _, lp = R.logp_entropy(c.P)
    assert -42 < q.min() < -30
    dq = (size * c.rng.normal(size=250)).astype(np.float32)
    dH, dW = c.logp_bwd(torch.from_numpy(dq).cuda(), 1.0 / size)
    check_grads(c, dH, dW, clean(dq, c.P.mask), lp, 1.0 / size)
