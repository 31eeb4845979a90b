"""The operators before a language model's head that this file's cases measure: the root-mean-square norm with the
residual's addition and its gradient, and 8-bit checkpoints of activations.

Matrices have N = G * L rows (row t = i*L + j is position j of sequence i) of d columns, of a 16-bit type; a mask says
which rows count, the others are not read and their outputs are zeros.

  norm       s = x + r in 16 bits, or s decoded from a checkpoint; y = s / sqrt(mean s^2 + eps) * w (or * (1 + w)), in 16
             bits or as 8-bit codes with a scale per row (max |y| / the type's largest value) or a given scale; s is
             written in 16 bits, as a checkpoint, or not at all
  norm_grad  dx and dw for a given dy, from s in 16 bits or from a checkpoint; the gradient that reaches s on its other
             way is added to dx
  pack       a checkpoint: in each block of 64 columns of a row scale = max |x| / 127 in bf16, code = round(x / scale)
  unpack     code * scale in 16 bits

`run` computes the plain forms (own = False) or calls the library (own = True) on the same state.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
LEAST = 2.0 ** -126      # the least scale
BLOCK = 64               # columns that share a checkpoint's scale
EPS = 1e-6


def _case(name, op, G, L, d, **more):
    c = {"name": name, "op": op, "G": G, "L": L, "d": d, "dtype": "bf16", "fill": 1.0, "empty": False,
         "weight_f32": False, "plus_one": False, "residual": op == "norm", "from_ckpt": False, "out": "16",
         "given_scale": 0.0, "sum": op == "norm", "keep_ckpt": False, "dsum": False, "dweight": True}
    c.update(more)
    return c


def listed():
    return [
        # one token of one sequence while it is generated: latency counts
        _case("norm one token", "norm", 1, 1, 4096),
        # scoring short fp16 completions of uneven length, one of them empty, for a head in 8 bits
        _case("norm short ragged fp16", "norm", 8, 257, 5120, dtype="fp16", fill=0.6, empty=True, residual=False, sum=False,
              out="e4m3"),
        # a training step: codes for the 8-bit head, and of the residual stream only an 8-bit checkpoint is kept
        _case("norm to 8 bits, checkpoint", "norm", 8, 1250, 4096, out="e4m3", given_scale=0.0625, sum=False, keep_ckpt=True),
        # eight completions in a context of 20K tokens, padded
        _case("norm 20K context", "norm", 8, 20000, 4096, fill=0.54),
        # the smallest step of the tests: launches and waits are all that counts
        _case("gradient smallest", "norm_grad", 4, 64, 128),
        # a norm inside the model on a group of completions: gradients from both ways, an fp32 weight
        _case("gradient a group", "norm_grad", 8, 1024, 1536, fill=0.6, weight_f32=True, dsum=True),
        # fp16 under a loss scale, odd lengths, the weight stored as its difference from 1
        _case("gradient odd fp16", "norm_grad", 5, 301, 5120, dtype="fp16", fill=0.7, empty=True, plus_one=True),
        # the step's gradient at 20K context, from the 8-bit checkpoint
        _case("gradient 20K, checkpoint", "norm_grad", 8, 20000, 4096, fill=0.54, from_ckpt=True),
        # a layer's input, short answers
        _case("pack short answers", "pack", 8, 333, 1536, dtype="fp16"),
        # a layer's input at 20K context
        _case("pack 20K", "pack", 8, 20000, 4096),
        # the same two when the layer's backward pass needs them again
        _case("unpack short answers", "unpack", 8, 333, 1536, dtype="fp16"),
        _case("unpack 20K", "unpack", 8, 20000, 4096),
    ]


MOST = 8 * 20000 * 4096      # elements of the largest listed cases


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "norm", "norm_grad", "norm_grad", "pack", "unpack"])
    d = BLOCK * spread(1, 128)
    G = rng.choice([1, 2, 4, 5, 8])
    L = max(1, min(spread(1, 20000), MOST // (2 * G * d)))
    c = _case("", op, G, L, d, dtype=rng.choice(["bf16", "bf16", "fp16"]), fill=rng.choice([0.55, 0.8, 1.0]),
              empty=G > 2 and rng.random() < 0.3)
    if op in ("norm", "norm_grad"):
        c["weight_f32"], c["plus_one"], c["from_ckpt"] = rng.random() < 0.4, rng.random() < 0.3, rng.random() < 0.35
    if op == "norm":
        c["residual"] = not c["from_ckpt"] and rng.random() < 0.7
        c["out"] = rng.choice(["16", "e4m3", "e4m3", "e5m2"])
        if c["out"] != "16":
            c["given_scale"] = rng.choice([0.0, 0.0625])
        c["sum"] = c["residual"] and rng.random() < 0.6
        c["keep_ckpt"] = not c["from_ckpt"] and rng.random() < 0.5
    if op == "norm_grad":
        c["dsum"], c["dweight"] = rng.random() < 0.5, rng.random() < 0.75
    del c["name"]
    return c


def _lengths(case):
    """Lengths of the sequences, spread evenly around fill * L; the same for every seed up to their order."""
    n, L = case["G"], case["L"]
    half = min(1.0 - case["fill"], case["fill"])
    ln = [int(round(L * (case["fill"] + half * (2.0 * ((7 * i + 3) % n + 0.5) / n - 1.0)))) for i in range(n)]
    ln = [min(L, max(1, x)) for x in ln]
    if case["empty"]:
        ln[n // 2] = 0
    return ln


def _padded(case):
    return case["fill"] < 1.0 or case["empty"]


def _pack(x):
    """(codes, scales) of a matrix."""
    b = x.float().view(x.shape[0], -1, BLOCK)
    scale = (b.abs().amax(-1) * (1.0 / 127)).clamp(min=LEAST).to(torch.bfloat16)
    codes = torch.round(b * (1.0 / scale.float())[:, :, None]).clamp(-128, 127).to(torch.int8)
    return codes.view(x.shape), scale


def _unpack(codes, scale, dtype):
    b = codes.view(codes.shape[0], -1, BLOCK).float() * scale.float()[:, :, None]
    return b.view(codes.shape).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt, d, L, n = DTYPES[case["dtype"]], case["d"], case["L"], case["G"]
    N = n * L

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    s = {"case": case, "mask": None, "rows": torch.arange(N, device="cuda")}
    order = torch.randperm(n, device="cuda", generator=g)
    if _padded(case):
        lengths = torch.tensor(_lengths(case), device="cuda")[order]
        s["mask"] = (torch.arange(L, device="cuda")[None, :] < lengths[:, None]).reshape(N).to(torch.uint8).contiguous()
        s["rows"] = s["mask"].nonzero()[:, 0]
    # a residual stream: channels of different size, one in 500 of them thirty times as large
    channel = torch.exp(0.5 * randn(d)) * torch.where(torch.rand(d, device="cuda", generator=g) < 0.002, 30.0, 1.0)
    x = (randn(N, d) * channel).to(dt)
    if case["residual"]:
        s["residual"] = (0.3 * randn(N, d) * channel).to(dt)
    if case["from_ckpt"] or case["op"] == "unpack":
        s["codes"], s["scales"] = _pack(x)
        x = None
    s["x"] = x
    if case["op"] in ("norm", "norm_grad"):
        w = 0.2 * randn(d) + (0.0 if case["plus_one"] else 1.0)
        s["w"] = w if case["weight_f32"] else w.to(dt)
    if case["op"] == "norm_grad":
        # the head's gradient: rows of different size, some of them zero (clipped tokens)
        row = torch.exp(randn(N, 1)) * (torch.rand(N, 1, device="cuda", generator=g) < 0.9)
        s["dy"] = (0.02 * row * randn(N, d)).to(dt)
        if case["dsum"]:
            s["dsum"] = (0.01 * randn(N, d)).to(dt)
    return s


def _whole(s, part, fill=0.0):
    """The rows that count among all rows; the others hold `fill`."""
    if s["mask"] is None:
        return part
    out = torch.full((s["mask"].numel(), *part.shape[1:]), fill, device=part.device, dtype=torch.float32).to(part.dtype)
    return out.index_copy_(0, s["rows"], part)


def _stream(s):
    """s in 32 bits, rows that count only: the rounded sum, or the checkpoint's values."""
    case, rows = s["case"], s["rows"]
    dt = DTYPES[case["dtype"]]
    if case["from_ckpt"]:
        return _unpack(s["codes"][rows], s["scales"][rows], dt).float()
    x = s["x"][rows].float()
    if case["residual"]:
        x = (x + s["residual"][rows].float()).to(dt).float()
    return x


def _plain(s):
    case, op, rows = s["case"], s["case"]["op"], s["rows"]
    dt = DTYPES[case["dtype"]]
    if op == "pack":
        codes, scales = _pack(s["x"][rows])
        return {"codes": _whole(s, codes.view(torch.uint8)).view(torch.int8), "scales": _whole(s, scales, LEAST)}
    if op == "unpack":
        return {"x": _whole(s, _unpack(s["codes"][rows], s["scales"][rows], dt))}
    v = _stream(s)
    w = s["w"].float() + (1.0 if case["plus_one"] else 0.0)
    r = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    if op == "norm":
        y = v * r * w
        out = {}
        if case["out"] == "16":
            out["y"] = _whole(s, y.to(dt))
        else:
            top = LARGEST[case["out"]]
            scale = (y.abs().amax(1) * (1.0 / top)).clamp(min=LEAST)
            out["scale"] = _whole(s, scale, LEAST)
            by = (1.0 / scale)[:, None] if not case["given_scale"] else 1.0 / case["given_scale"]
            codes = (y * by).clamp(-top, top).to(E8[case["out"]])
            out["y"] = _whole(s, codes.view(torch.uint8)).view(E8[case["out"]])
        if case["sum"]:
            out["sum"] = _whole(s, v.to(dt))
        if case["keep_ckpt"]:
            codes, scales = _pack(v)
            out["codes"] = _whole(s, codes.view(torch.uint8)).view(torch.int8)
            out["scales"] = _whole(s, scales, LEAST)
        return out
    dy = s["dy"][rows].float()
    g = dy * w
    dx = r * (g - v * (r * r * (g * v).mean(1, keepdim=True)))
    if case["dsum"]:
        dx = dx + s["dsum"][rows].float()
    out = {"dx": _whole(s, dx.to(dt))}
    bad = ~torch.isfinite(out["dx"]).all()
    if case["dweight"]:
        out["dw"] = (dy * v * r).sum(0).to(s["w"].dtype)
        bad = bad | ~torch.isfinite(out["dw"]).all()
    return {**out, "found_inf": bad.to(torch.int32).reshape(1)}


def _keep(s):
    """What a training or serving loop keeps between its calls: the shape, the options, the workspace and its buffers."""
    import rl_fine_tuning_gb300 as rg
    case, op = s["case"], s["case"]["op"]
    dt, N, d = DTYPES[case["dtype"]], case["G"] * case["L"], case["d"]

    def empty(*shape, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    def ckpt():
        return empty(N, d, dtype=torch.int8), empty(N, d // BLOCK, dtype=torch.bfloat16)

    k = {"shape": rg.make_shape(1, case["G"], case["L"], d, 1, rg.BF16 if case["dtype"] == "bf16" else rg.FP16)}
    kept = (s["codes"], s["scales"]) if case["from_ckpt"] or op == "unpack" else None
    if op == "norm":
        y_type = {"16": k["shape"].dtype, "e4m3": rg.E4M3, "e5m2": rg.E5M2}[case["out"]]
        k["opts"] = rg.norm_opts(eps=EPS, weight_f32=case["weight_f32"], plus_one=case["plus_one"], y_type=y_type,
                                 y_scale=case["given_scale"])
        k["src"], out = kept if kept else s["x"], {}
        out["y"] = empty(N, d, dtype=dt if case["out"] == "16" else E8[case["out"]])
        if case["out"] != "16":
            out["scale"] = empty(N, dtype=torch.float32)
        if case["sum"]:
            out["sum"] = empty(N, d)
        if case["keep_ckpt"]:
            k["ckpt"] = ckpt()
            out["codes"], out["scales"] = k["ckpt"]
    elif op == "norm_grad":
        k["opts"] = rg.norm_opts(eps=EPS, weight_f32=case["weight_f32"], plus_one=case["plus_one"], y_type=k["shape"].dtype)
        k["ws"] = empty(rg.grpo_norm_workspace_bytes(k["shape"]), dtype=torch.uint8)
        k["src"] = kept if kept else s["x"]
        out = {"dx": empty(N, d), "found_inf": empty(1, dtype=torch.int32)}
        if case["dweight"]:
            out["dw"] = torch.empty_like(s["w"])
    elif op == "pack":
        k["ckpt"] = ckpt()
        out = {"codes": k["ckpt"][0], "scales": k["ckpt"][1]}
    else:
        k["ckpt"], out = kept, {"x": empty(N, d)}
    k["out"] = out
    return k


def _own(s):
    import rl_fine_tuning_gb300 as rg
    if "kept" not in s:
        s["kept"] = _keep(s)
    k, op = s["kept"], s["case"]["op"]
    out, shape, mask = k["out"], k["shape"], s["mask"]
    if op == "norm":
        rg.grpo_norm_fwd(k["src"], s.get("residual"), s["w"], mask, shape, k["opts"], out["y"], out.get("scale"),
                         out.get("sum"), k.get("ckpt"))
    elif op == "norm_grad":
        rg.grpo_norm_bwd(s["dy"], k["src"], s["w"], s.get("dsum"), mask, shape, k["opts"], k["ws"], out["dx"], out.get("dw"),
                         out["found_inf"])
    elif op == "pack":
        rg.grpo_ckpt_pack(s["x"], mask, shape, k["ckpt"])
    else:
        rg.grpo_ckpt_unpack(k["ckpt"], mask, shape, out["x"])
    return out


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    N, d, op = case["G"] * case["L"], case["d"], case["op"]
    Nv = sum(_lengths(case)) if _padded(case) else N
    packed = 1.0 + 2.0 / BLOCK
    rows = N if _padded(case) else 0          # the mask
    if op == "pack":
        return {"bytes": rows + d * (2.0 * Nv + packed * N), "flops": 3.0 * Nv * d}
    if op == "unpack":
        return {"bytes": rows + d * (packed * Nv + 2.0 * N), "flops": 1.0 * Nv * d}
    weight = d * (4.0 if case["weight_f32"] else 2.0)
    read = packed if case["from_ckpt"] else 2.0
    if op == "norm":
        read += 2.0 * case["residual"]
        write = (2.0 if case["out"] == "16" else 1.0) + 2.0 * case["sum"] + packed * case["keep_ckpt"]
        scales = 0.0 if case["out"] == "16" else 4.0 * N
        return {"bytes": rows + weight + scales + d * (read * Nv + write * N), "flops": 5.0 * Nv * d}
    read += 2.0 + 2.0 * case["dsum"]
    return {"bytes": rows + weight * (1 + case["dweight"]) + d * (read * Nv + 2.0 * N), "flops": 12.0 * Nv * d}


def exact(case, seed):
    """The definitions in 64 bits, the gradients by differentiating y.  8-bit values are given before their rounding where
    a type's rounding lies below its bound (E4M3), and not at all for E5M2 and for a checkpoint's codes."""
    s = prepare(case, seed)
    N, d, op = case["G"] * case["L"], case["d"], case["op"]
    dt = DTYPES[case["dtype"]]
    alive = torch.ones(N, 1, dtype=torch.float64, device="cuda") if s["mask"] is None else s["mask"].double()[:, None]

    def block_scale(m):
        return (torch.linalg.vector_norm(m.reshape(N, d // BLOCK, BLOCK), ord=math.inf, dim=2) / 127).clamp(min=LEAST)

    def decoded():
        each = torch.repeat_interleave(s["scales"].double(), BLOCK, dim=1)
        return each.mul_(s["codes"])

    if op == "pack":
        return {"codes": None, "scales": block_scale(s["x"].double() * alive)}
    if op == "unpack":
        return {"x": decoded() * alive}
    w = s["w"].double() + case["plus_one"]
    if case["from_ckpt"]:
        total = decoded()
    else:
        total = s["x"].double()
        if case["residual"]:
            total += s["residual"]
    stored = total.to(dt).double()             # the residual stream is a 16-bit matrix
    if op == "norm":
        y = stored / torch.sqrt(stored.square().sum(1, keepdim=True) / d + EPS) * w * alive
        out = {"y": y}
        if case["out"] != "16":
            out["scale"] = torch.clamp(torch.linalg.vector_norm(y, ord=math.inf, dim=1) / LARGEST[case["out"]], min=LEAST)
            per = out["scale"][:, None] if case["given_scale"] == 0.0 else case["given_scale"]
            out["y"] = (y / per).clamp(-LARGEST[case["out"]], LARGEST[case["out"]]) if case["out"] == "e4m3" else None
        if case["sum"]:
            out["sum"] = total * alive
        if case["keep_ckpt"]:
            out["codes"], out["scales"] = None, block_scale(stored * alive)
        return out
    dx, dw = torch.empty_like(stored), torch.zeros_like(w)
    for a in range(0, N, 1 << 15):             # rows are independent: a part of them at a time
        v = stored[a:a + (1 << 15)].requires_grad_()
        wp = w.clone().requires_grad_()
        y = v / torch.sqrt(v.square().sum(1, keepdim=True) / d + EPS) * wp
        gv, gw = torch.autograd.grad((y * s["dy"][a:a + (1 << 15)] * alive[a:a + (1 << 15)]).sum(), [v, wp])
        dx[a:a + (1 << 15)] = gv
        dw += gw
    if case["dsum"]:
        dx += s["dsum"] * alive
    out = {"dx": dx, "found_inf": None}
    if case["dweight"]:
        out["dw"] = dw
    return out
