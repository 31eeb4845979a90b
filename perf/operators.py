"""The operators on a language model's head that this file's cases measure: log-probabilities of given tokens, the
clipped policy loss, and the preference loss over pairs of completions.

All of them take hidden states h [N x d] (row t = i*L + j is position j of completion i), the head's weight W [V x d],
one token id per row and a mask of the rows that count, and never return the (N x V) logits.  With
z = h W^T / T and q = z[token] - logsumexp(z):

  logp       q and the entropy of softmax(z) for every row (0 on masked rows)
  logp_grad  the gradients of sum_t dq_t q_t for given dq
  clip       s = min(r A, clip(r, 1 - lo, 1 + hi) A) with r = exp(q - q_old), k = exp(x) - x - 1 with x = p - q;
             loss = mean(-s + beta k) over the rows, or over completions of their rows' means, and its gradients
  pair       completions 2i (preferred) and 2i + 1: S = sum (or mean) over the rows of q - p,
             m = beta (S_2i - S_2i+1); loss = mean over pairs of -(1-e) log sigmoid(m) - e log sigmoid(-m),
             of max(0, 1 - m), or of (m / beta - 1 / (2 beta))^2, and its gradients

`run` computes the plain forms (own = False) or calls the library (own = True) on the same state.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}

#: the tests' small head, and the heads that the benchmark's workloads have
TINY = {"d": 128, "V": 1024}
HEAD_1_5B = {"d": 1536, "V": 151936}
HEAD_8B = {"d": 4096, "V": 128256}
HEAD_14B = {"d": 5120, "V": 100352}


def _case(name, op, head, groups, G, L, **more):
    c = {"name": name, "op": op, "groups": groups, "G": G, "L": L, **head, "dtype": "bf16", "fill": 1.0, "empty": False,
         "temperature": 1.0, "beta": 0.04, "seq_mean": False, "kind": "sigmoid", "smoothing": 0.0, "length_mean": False,
         "scale": 1.0}
    c.update(more)
    return c


def listed():
    return [
        # one token of one sequence while it is generated: W is read once, latency counts
        _case("logp one token", "logp", HEAD_8B, 1, 1, 1),
        # one token for each of the 8 completions of a group, at the sampling temperature
        _case("logp a token for each of 8", "logp", HEAD_1_5B, 1, 8, 1, temperature=1.5),
        # scoring short completions of uneven length, one of them empty
        _case("logp short ragged fp16", "logp", HEAD_14B, 1, 8, 257, dtype="fp16", fill=0.6, empty=True),
        # recording the reference's log-probs of a group's completions
        _case("logp a group", "logp", HEAD_1_5B, 1, 8, 1024, fill=0.6),
        # the gradient for a loss that the caller has computed from the log-probs
        _case("logp gradient", "logp_grad", HEAD_8B, 1, 4, 333, fill=0.7),
        # the smallest step of the tests: launches and waits are all that counts
        _case("clip smallest", "clip", TINY, 1, 4, 64, fill=0.8),
        # a later minibatch over a group of 8 completions
        _case("clip a group", "clip", HEAD_1_5B, 1, 8, 1024, fill=0.6),
        # the largest: eight completions of the 8B head
        _case("clip a long group", "clip", HEAD_8B, 1, 8, 1250, fill=0.75),
        # fp16 with a loss scale, odd lengths, the mean over completions, no reference
        _case("clip odd fp16", "clip", HEAD_14B, 1, 5, 301, dtype="fp16", fill=0.7, empty=True, beta=0.0, seq_mean=True,
              scale=4096.0),
        # the smallest preference step
        _case("pair smallest", "pair", TINY, 3, 2, 37, fill=0.7, beta=0.1),
        # short answers, one of them empty, means instead of sums and smoothed labels
        _case("pair short answers", "pair", HEAD_1_5B, 4, 2, 333, fill=0.6, empty=True, beta=2.0, smoothing=0.1,
              length_mean=True),
        # long answers
        _case("pair long answers", "pair", HEAD_8B, 2, 2, 1500, fill=0.7, beta=0.1),
    ]


MOST_ROWS_FLOPS = 6.0 * 7500 * 128256 * 4096   # the largest listed case


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["logp", "logp_grad", "clip", "clip", "pair"])
    d, V = 64 * spread(2, 80), spread(1000, 152064)
    groups, G = (spread(1, 8), 2) if op == "pair" else (rng.choice([1, 1, 2]), rng.choice([1, 2, 4, 5, 8]))
    L = spread(1, 1500)
    fill = rng.choice([0.5, 0.7, 1.0])
    most = MOST_ROWS_FLOPS / (6.0 * V * d * groups * G * fill)
    L = max(1, min(L, int(most)))
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    c = _case("", op, {"d": d, "V": V}, groups, G, L, dtype=dtype, fill=fill, empty=groups * G > 2 and rng.random() < 0.3,
              temperature=1.0 if op == "pair" else rng.choice([1.0, 1.0, 0.7, 1.5]),
              beta=rng.choice([0.0, 0.04]), seq_mean=rng.random() < 0.3,
              kind=rng.choice(["sigmoid", "sigmoid", "hinge", "square"]), smoothing=rng.choice([0.0, 0.1]),
              length_mean=rng.random() < 0.3,
              scale=1.0 if dtype == "bf16" or op == "logp" else 256.0 if op == "pair" else 4096.0)
    if c["kind"] != "sigmoid":
        c["smoothing"] = 0.0
    if c["kind"] == "square":
        c["length_mean"] = True
    if op == "pair":
        c["beta"] = rng.choice([0.5, 2.0]) if c["length_mean"] else rng.choice([0.05, 0.1])
    del c["name"]
    return c


def _lengths(case):
    """Completion lengths, spread evenly around fill * L; the same for every seed up to their order."""
    n, L = case["groups"] * case["G"], case["L"]
    half = min(1.0 - case["fill"], case["fill"])
    ln = [int(round(L * (case["fill"] + half * (2.0 * ((7 * i + 3) % n + 0.5) / n - 1.0)))) for i in range(n)]
    ln = [min(L, max(1, x)) for x in ln]
    if case["empty"]:
        ln[n // 2] = 0
    return ln


def _logp32(h, W, tokens, rows, T):
    """q of the given rows, in 32 bits, 2048 rows at a time."""
    Wf, out = W.float(), []
    for r in rows.split(2048):
        z = (h[r].float() @ Wf.t()) / T
        out.append(z.gather(1, tokens[r].long()[:, None])[:, 0] - torch.logsumexp(z, 1))
    return torch.cat(out) if out else h.new_zeros(0, dtype=torch.float32)


CLIP_LOW, CLIP_HIGH = 0.2, 0.28


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, d, V, L, T = DTYPES[case["dtype"]], case["d"], case["V"], case["L"], case["temperature"]
    n = case["groups"] * case["G"]
    N = n * L

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    # a head whose sampled tokens are likely ones, as a model's are: logits of about N(0, 1), the token's 2 to 16 higher
    W = (randn(V, d) * d ** -0.5).to(dt)
    tokens = torch.randint(0, V, (N,), device="cuda", generator=g, dtype=torch.int32)
    h = randn(N, d)
    a = T * (2.0 + 14.0 * torch.rand(N, 1, device="cuda", generator=g))
    h = (h + a * W[tokens.long()].float()).to(dt)
    order = torch.randperm(n, device="cuda", generator=g)
    lengths = torch.tensor(_lengths(case), device="cuda", dtype=torch.int32)[order]
    mask = (torch.arange(L, device="cuda")[None, :] < lengths[:, None]).reshape(N).to(torch.uint8).contiguous()
    s = {"case": case, "h": h, "W": W, "tokens": tokens, "mask": mask, "rows": mask.nonzero()[:, 0], "seq": n}
    if case["op"] == "logp" and case["fill"] == 1.0 and not case["empty"]:
        s["mask"] = None   # every row counts: a user passes no mask
    if case["op"] == "logp_grad":
        s["dlogp"] = randn(N) * mask / max(1, int(mask.sum()))
    if case["op"] in ("clip", "pair"):
        q = torch.zeros(N, device="cuda")
        q[s["rows"]] = _logp32(h, W, tokens, s["rows"], T)
    if case["op"] == "clip":
        # log-probs under the policy that sampled: ratios of about exp(N(0, 0.15)).  Rows whose ratio is within a
        # thousandth of a clip border are moved off it: on which side the last bit falls is not what is compared.
        lr = 0.15 * randn(N)
        r = lr.exp()
        near = ((r - (1 - CLIP_LOW)).abs() < 1e-3) | ((r - (1 + CLIP_HIGH)).abs() < 1e-3)
        s["old"] = (q - torch.where(near, lr + 0.005, lr)) * mask
        s["ref"] = (q + 0.3 * randn(N)) * mask if case["beta"] else None
        rewards = randn(case["groups"], case["G"])
        adv = rewards - rewards.mean(1, keepdim=True) if case["G"] > 1 else rewards
        s["adv"] = (adv + 0.25).reshape(n).contiguous()
    if case["op"] == "pair":
        # log-ratios as after some training: preferred completions up by 8, the others down by 12, noise per token
        drift = torch.where(torch.arange(n, device="cuda") % 2 == 0, -8.0, 12.0) / max(16.0, case["fill"] * L)
        s["ref"] = (q + (drift[:, None] + 0.1 * randn(n, L)).reshape(N)) * mask
    return s


def _plain_grads(s, z, q_index, lse, g):
    """dH (all rows) and dW of sum_t g_t q_t over the valid rows, from their logits z (overwritten)."""
    case, rows, h, W = s["case"], s["rows"], s["h"], s["W"]
    dz = torch.exp(z - lse[:, None])
    dz = dz.neg_()
    dz[torch.arange(rows.numel(), device=dz.device), q_index] += 1.0
    dz *= (g * (case["scale"] / case["temperature"]))[:, None]
    dH = torch.zeros_like(h)
    dH[rows] = (dz @ W.float()).to(h.dtype)
    return dH, (dz.t() @ h[rows].float()).to(W.dtype)


def _plain(s):
    case, rows, h, W = s["case"], s["rows"], s["h"], s["W"]
    N, n, L, T = h.shape[0], s["seq"], case["L"], case["temperature"]
    z = h[rows].float() @ W.float().t()
    if T != 1.0:
        z /= T
    tok = s["tokens"][rows].long()
    # the given token's logit in 64 bits: its error would stay in q, in ratios near 1 and in long sums of q
    zt = torch.cat([(h[r].double() * W[s["tokens"][r].long()].double()).sum(1) for r in rows.split(4096)]) / T
    z[torch.arange(rows.numel(), device=z.device), tok] = zt.float()
    lse = torch.logsumexp(z, 1)
    q = (zt - lse.double()).float()
    logp = torch.zeros(N, device=h.device)
    logp[rows] = q
    if case["op"] == "logp":
        ent = torch.zeros(N, device=h.device)
        ent[rows] = lse - (torch.exp(z - lse[:, None]) * z).sum(1)
        return {"logp": logp, "entropy": ent}
    if case["op"] == "logp_grad":
        dH, dW = _plain_grads(s, z, tok, lse, s["dlogp"][rows])
        return {"dH": dH, "dW": dW}
    seq = rows // L
    count = torch.zeros(n, device=h.device).index_add_(0, seq, torch.ones_like(q))
    if case["op"] == "clip":
        A = s["adv"][seq]
        r = torch.exp(q - s["old"][rows])
        low, high = r < 1 - CLIP_LOW, r > 1 + CLIP_HIGH
        clipped = torch.where(low, 1 - CLIP_LOW, torch.where(high, 1 + CLIP_HIGH, r))
        ell = -torch.minimum(r * A, clipped * A)
        g = torch.where((high & (A > 0)) | (low & (A < 0)), 0.0, -A * r)
        kl = torch.zeros_like(q)
        if case["beta"]:
            x = s["ref"][rows] - q
            kl = torch.expm1(x) - x
            ell = ell + case["beta"] * kl
            g = g - case["beta"] * torch.expm1(x)
        w = 1.0 / (count[seq] * (count > 0).sum()) if case["seq_mean"] else torch.full_like(q, 1.0 / max(1, rows.numel()))
        stats = torch.zeros(N, 3, device=h.device)
        stats[rows] = torch.stack([q, r, kl], 1)
        loss = (ell.double() * w.double()).sum().float().reshape(1)
        dH, dW = _plain_grads(s, z, tok, lse, g * w)
        return {"loss": loss, "row_stats": stats, "dH": dH, "dW": dW}
    beta, e = case["beta"], case["smoothing"]
    S = torch.zeros(n, device=h.device, dtype=torch.float64).index_add_(0, seq, (q.double() - s["ref"][rows].double()))
    each = torch.where(count > 0, 1.0 / count.clamp(min=1), 0.0) if case["length_mean"] else torch.ones_like(count)
    S = S * each.double()
    m = beta * (S[0::2] - S[1::2])
    active = (count[0::2] + count[1::2]) > 0
    if case["kind"] == "sigmoid":
        up = torch.log1p(torch.exp(-m.abs())) + torch.clamp(-m, min=0)      # -log sigmoid(m)
        ell, dm = (1 - e) * up + e * (up + m), -(1 - e) / (1 + torch.exp(m)) + e / (1 + torch.exp(-m))
    elif case["kind"] == "hinge":
        ell, dm = torch.clamp(1 - m, min=0), torch.where(m < 1, -1.0, 0.0).double()
    else:
        t = m / beta - 1 / (2 * beta)
        ell, dm = t * t, 2 * t / beta
    pairs = max(1, int(active.sum()))
    ell, dm = torch.where(active, ell, 0.0), torch.where(active, dm, 0.0) / pairs
    dS = (beta * torch.stack([dm, -dm], 1).reshape(n)) * each.double()
    dH, dW = _plain_grads(s, z, tok, lse, dS[seq].float())
    stats = torch.stack([beta * S[0::2], beta * S[1::2], m, ell], 1).float()
    return {"loss": (ell.sum() / pairs).float().reshape(1), "pair_stats": stats, "logp": logp, "dH": dH, "dW": dW}


def _own(s):
    import rl_fine_tuning_gb300 as rg
    case, h, W = s["case"], s["h"], s["W"]
    op, T, scale = case["op"], case["temperature"], case["scale"]
    if "shape" not in s:
        # what a training or serving loop keeps between its calls: the shape, the options, the workspace and its buffers
        s["shape"] = rg.make_shape(case["groups"], case["G"], case["L"], case["d"], case["V"],
                                   rg.BF16 if case["dtype"] == "bf16" else rg.FP16, beta=case["beta"],
                                   loss_mode=rg.SEQUENCE_MEAN if case["seq_mean"] and op == "clip" else rg.TOKEN_MEAN)
        s["ws"] = torch.empty(rg.grpo_policy_workspace_bytes(s["shape"], op), dtype=torch.uint8, device=h.device)
        s["status"] = torch.zeros(1, dtype=torch.int32, device=h.device)
        s["inf"] = torch.zeros(1, dtype=torch.int32, device=h.device)
        s["f32"] = lambda *n: torch.empty(*n, dtype=torch.float32, device=h.device)
        s["clip"] = rg.clip_opts(temperature=T, clip_low=CLIP_LOW, clip_high=CLIP_HIGH)
        s["pair"] = rg.pair_opts(kind=case["kind"], label_smoothing=case["smoothing"], length_mean=case["length_mean"])
    N, f32 = h.shape[0], s["f32"]
    if op == "logp":
        logp, ent = f32(N), f32(N)
        rg.grpo_logprobs(h, W, s["tokens"], s["mask"], s["shape"], T, s["ws"], logp, ent, s["status"])
        return {"logp": logp, "entropy": ent}
    dH, dW = torch.empty_like(h), torch.empty_like(W)
    if op == "logp_grad":
        rg.grpo_logprobs_bwd(h, W, s["tokens"], s["mask"], s["dlogp"], s["shape"], T, scale, s["ws"], dH, dW, s["inf"],
                             s["status"])
        return {"dH": dH, "dW": dW}
    loss = f32(1)
    if op == "clip":
        stats = f32(N, 3)
        rg.grpo_clip_loss_fwd_bwd(h, W, s["tokens"], s["mask"], s["adv"], s["old"], s["ref"], s["shape"], s["clip"], scale,
                                  s["ws"], loss, dH, dW, s["inf"], stats, s["status"])
        return {"loss": loss, "row_stats": stats, "dH": dH, "dW": dW}
    stats, logp = f32(case["groups"], 4), f32(N)
    rg.grpo_pair_loss_fwd_bwd(h, W, s["tokens"], s["mask"], s["ref"], s["shape"], s["pair"], scale, s["ws"], loss, dH, dW,
                              s["inf"], logp, stats, s["status"])
    return {"loss": loss, "pair_stats": stats, "logp": logp, "dH": dH, "dW": dW}


def run(state):
    return _own(state) if own else _plain(state)


def _valid(case):
    return sum(_lengths(case))


def work(case):
    Nv, N, d, V = _valid(case), case["groups"] * case["G"] * case["L"], case["d"], case["V"]
    unit = 2.0 * Nv * V * d
    read = 2.0 * (Nv * d + V * d) + 4.0 * Nv + (0 if case["op"] == "logp" and case["fill"] == 1.0 else N)
    if case["op"] == "logp":
        return {"bytes": read + 8.0 * N, "flops": unit}
    grads = 2.0 * (N * d + V * d)
    rows = {"logp_grad": 4.0 * Nv, "clip": (8.0 if case["beta"] else 4.0) * Nv + 12.0 * N, "pair": 4.0 * Nv + 4.0 * N}
    return {"bytes": read + grads + rows[case["op"]], "flops": 3 * unit}


def exact(case, seed):
    """The definition in 64 bits, gradients by differentiating the loss; None where that would take too long."""
    Nv = _valid(case)
    if (2.0 if case["op"] == "logp" else 6.0) * Nv * case["V"] * case["d"] > 9e12:
        return None
    s = prepare(case, seed)
    N, n, L, T = s["h"].shape[0], s["seq"], case["L"], case["temperature"]
    rows = s["rows"]
    H = s["h"][rows].double().requires_grad_(case["op"] != "logp")
    W = s["W"].double().requires_grad_(case["op"] != "logp")
    lp = torch.log_softmax(torch.matmul(H, W.transpose(0, 1)) / T, dim=-1)
    q = lp[torch.arange(Nv, device=lp.device), s["tokens"][rows].long()]

    def whole(x, *more):
        return torch.zeros(N, *more, dtype=torch.float64, device=x.device).index_copy(0, rows, x.detach())

    if case["op"] == "logp":
        return {"logp": whole(q), "entropy": whole(-(lp.exp() * lp).sum(-1))}
    member = torch.nn.functional.one_hot(torch.div(rows, L, rounding_mode="floor"), n).double()   # [Nv x n]
    length = member.sum(0)
    out = {}
    if case["op"] == "logp_grad":
        total = (s["dlogp"][rows].double() * q).sum()
    elif case["op"] == "clip":
        A = member @ s["adv"].double()
        ratio = (q - s["old"][rows].double()).exp()
        per = -torch.min(ratio * A, ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * A)
        kl = torch.zeros_like(q)
        if case["beta"]:
            x = s["ref"][rows].double() - q
            kl = x.exp() - x - 1
        per = per + case["beta"] * kl
        if case["seq_mean"]:
            means = (member.t() @ per)[length > 0] / length[length > 0]
            total = means.mean()
        else:
            total = per.mean()
        out = {"loss": total.detach().reshape(1), "row_stats": whole(torch.stack([q, ratio, kl], 1), 3)}
    else:
        beta, e = case["beta"], case["smoothing"]
        S = member.t() @ (q - s["ref"][rows].double())
        if case["length_mean"]:
            S = S / length.clamp(min=1)
        S = S.reshape(-1, 2)
        m = beta * (S[:, 0] - S[:, 1])
        if case["kind"] == "sigmoid":
            per = -(1 - e) * torch.nn.functional.logsigmoid(m) - e * torch.nn.functional.logsigmoid(-m)
        elif case["kind"] == "hinge":
            per = torch.relu(1 - m)
        else:
            per = (S[:, 0] - S[:, 1] - 0.5 / beta) ** 2
        live = length.reshape(-1, 2).sum(1) > 0
        per = per * live
        total = per.sum() / live.sum().clamp(min=1)
        out = {"loss": total.detach().reshape(1), "logp": whole(q),
               "pair_stats": torch.stack([beta * S[:, 0], beta * S[:, 1], m, per], 1).detach()}
    gH, gW = torch.autograd.grad(case["scale"] * total, [H, W])
    return {**out, "dH": whole(gH, case["d"]), "dW": gW}
