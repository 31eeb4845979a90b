"""The norm before the head, its gradient and the 8-bit checkpoints on the GPU against their definitions in 64 bits
(norm_reference), within bounds counted from the roundings, and against one another bit for bit."""
import threading

import numpy as np
import pytest

import norm_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import rl_fine_tuning_gb300 as rg  # noqa: E402

DT = {"bf16": rg.BF16, "fp16": rg.FP16, "e4m3": rg.E4M3, "e5m2": rg.E5M2}
EPS = 1e-6
GUARD = 3        # rows behind the last one, left as they were


def host(t):
    return t.double().cpu().numpy()


def bits(t):
    return t.contiguous().view(torch.uint8).cpu()


def same(a, b):
    return torch.equal(bits(a), bits(b))


def make_mask(kind, N, rng):
    if kind is None:
        return None
    if kind == "none":
        return np.zeros(N, bool)
    if kind == "tail":
        return np.arange(N) < max(1, N // 2)
    return rng.random(N) < 0.6


class Case:
    """Inputs on the device; rows that do not count hold NaN and infinities, and so do GUARD rows behind the last."""

    def __init__(self, N, d, dt="bf16", mask=None, seed=0, weight="16", plus_one=False, scale=1.0):
        rng = np.random.default_rng(seed + 1000 * N + d)
        self.N, self.d, self.dt, self.plus_one = N, d, dt, plus_one
        self.rng = rng
        self.m = make_mask(mask, N, rng)
        self.keep = np.ones(N, bool) if self.m is None else self.m
        self.mask = None if self.m is None else torch.from_numpy(self.m.astype(np.uint8)).cuda()
        channel = np.exp(0.5 * rng.normal(size=d))
        channel[rng.integers(d)] *= 30
        rows = np.exp(rng.normal(size=(N, 1))) * scale
        self.x = self.put(rng.normal(size=(N, d)) * channel * rows)
        self.r = self.put(0.3 * rng.normal(size=(N, d)) * channel * rows)
        self.dy = self.put(0.05 * rng.normal(size=(N, d)) * (rng.random((N, 1)) < 0.9))
        self.ds = self.put(0.03 * rng.normal(size=(N, d)))
        w = 0.2 * rng.normal(size=d) + (0 if plus_one else 1)
        self.w = torch.from_numpy(w).to(torch.float32 if weight == "f32" else R.TORCH[dt]).cuda()
        self.weight_f32 = weight == "f32"
        self.shape = rg.make_shape(1, 1, N, d, 1, DT[dt])

    def put(self, a):
        t = torch.from_numpy(np.ascontiguousarray(a)).to(R.TORCH[self.dt])
        odd = torch.tensor([float("nan"), float("inf"), -float("inf")], dtype=t.dtype)
        t[~torch.from_numpy(self.keep)] = odd[torch.arange(self.d) % 3]
        return t.cuda()

    def clean(self, t):
        return np.where(self.keep[:, None], np.nan_to_num(host(t)), 0.0)

    def weight(self):
        return host(self.w) + self.plus_one

    def out(self, dtype, cols=None, fill=7):
        """An output with guard rows: (the N rows, all rows)."""
        cols = self.d if cols is None else cols
        whole = torch.full(((self.N + GUARD) * cols * torch.empty(0, dtype=dtype).element_size(),), fill, dtype=torch.uint8,
                           device="cuda").view(dtype)
        return whole[:self.N * cols].view(self.N, cols), whole

    def guarded(self, whole, cols):
        rest = bits(whole)[self.N * cols * whole.element_size():]
        assert rest.numel() and bool((rest == 7).all()), "rows behind the last were written"

    def fwd(self, x=None, residual=False, y="16", y_scale=0.0, row_scale=None, sum_out=False, ckpt=False, eps=EPS):
        """Dict of outputs."""
        t16 = R.TORCH[self.dt]
        yt = self.dt if y == "16" else y
        o = rg.norm_opts(eps=eps, weight_f32=self.weight_f32, plus_one=self.plus_one, y_type=DT[yt], y_scale=y_scale)
        outs = {"y": self.out(R.TORCH[yt])}
        if row_scale is None:
            row_scale = y != "16"
        if row_scale:
            outs["scale"] = self.out(torch.float32, 1)
        if sum_out:
            outs["sum"] = self.out(t16)
        if ckpt:
            outs["codes"], outs["scales"] = self.out(torch.int8), self.out(torch.bfloat16, self.d // 64)
        g = lambda k: outs[k][0] if k in outs else None  # noqa: E731
        rg.grpo_norm_fwd(self.x if x is None else x, self.r if residual else None, self.w, self.mask, self.shape, o, g("y"),
                         g("scale"), g("sum"), (g("codes"), g("scales")) if ckpt else None)
        torch.cuda.synchronize()
        for a, whole in outs.values():
            self.guarded(whole, a.shape[1])
        return {k: v[0] for k, v in outs.items()}

    def bwd(self, x=None, dsum=False, dweight=True, eps=EPS):
        o = rg.norm_opts(eps=eps, weight_f32=self.weight_f32, plus_one=self.plus_one)
        ws = torch.full((rg.grpo_norm_workspace_bytes(self.shape) + 256,), 255, dtype=torch.uint8, device="cuda")
        dx, whole = self.out(R.TORCH[self.dt])
        dw = torch.full_like(self.w, 7.0) if dweight else None
        inf = torch.full((1,), -1, dtype=torch.int32, device="cuda")
        rg.grpo_norm_bwd(self.dy, self.x if x is None else x, self.w, self.ds if dsum else None, self.mask, self.shape, o,
                         ws[:-256], dx, dw, inf)
        torch.cuda.synchronize()
        self.guarded(whole, self.d)
        assert bool((ws[-256:] == 255).all())
        return dx, dw, int(inf)

    def pack(self, x=None):
        (c, cw), (s, sw) = self.out(torch.int8), self.out(torch.bfloat16, self.d // 64)
        rg.grpo_ckpt_pack(self.x if x is None else x, self.mask, self.shape, (c, s))
        torch.cuda.synchronize()
        self.guarded(cw, self.d)
        self.guarded(sw, self.d // 64)
        return c, s

    def unpack(self, ck):
        x, whole = self.out(R.TORCH[self.dt])
        rg.grpo_ckpt_unpack(ck, self.mask, self.shape, x)
        torch.cuda.synchronize()
        self.guarded(whole, self.d)
        return x


def torch_pack(x):
    """The definition in fp32 operations, on the rows of x."""
    b = x.float().view(x.shape[0], -1, 64)
    s = (b.abs().amax(-1) * (1.0 / 127)).clamp(min=R.LEAST).to(torch.bfloat16)
    return torch.round(b * (1.0 / s.float())[:, :, None]).to(torch.int8).view(x.shape), s


def check_y(c, s, got, y, y_scale, eps=EPS):
    ref, _ = R.norm(s, c.weight(), eps)
    ref[~c.keep] = 0.0
    if y == "16":
        assert np.all(np.abs(host(got["y"]) - ref) <= R.y_bound(ref, c.d, c.dt))
        return
    scale = R.row_scale(ref, y)
    if "scale" in got:
        e = R.rel32(c.d) + 4 * R.STEP32
        assert np.all(np.abs(host(got["scale"])[:, 0] - scale) <= e * scale)
    scale = host(got["scale"]) if y_scale == 0.0 else np.full((c.N, 1), np.float64(np.float32(y_scale)))
    top = R.LARGEST[y]
    want = np.clip(ref / scale, -top, top) * scale
    # where nothing saturates; a value within the bound of the largest may do either
    assert np.all(np.abs(host(got["y"]) * scale - want) <= R.code_bound(want, scale, c.d, y))
    assert not np.isnan(host(got["y"])).any()


# ---------------------------------------------------------------- forward

SIZES = [(1, 64), (1, 4096), (2, 128), (7, 192), (33, 1536), (5, 4160), (3, 8192), (2, 16384), (300, 320), (1000, 64), (40, 5120)]


@pytest.mark.parametrize("N,d", SIZES)
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("y,y_scale", [("16", 0.0), ("e4m3", 0.0), ("e5m2", 0.0), ("e4m3", 0.05)])
def test_forward(N, d, dt, y, y_scale):
    """Every output at once, with a residual and a ragged mask."""
    c = Case(N, d, dt, "some" if N > 1 else None, weight="f32" if d % 128 else "16", plus_one=N % 2 == 1)
    got = c.fwd(residual=True, y=y, y_scale=y_scale, sum_out=True, ckpt=True)
    want = (c.x.float() + c.r.float()).to(c.x.dtype)
    if c.mask is not None:
        want[~c.mask.bool()] = 0
    assert same(got["sum"], want)
    codes, scales = torch_pack(want)
    assert torch.equal(got["codes"], codes) and same(got["scales"], scales)
    check_y(c, c.clean(want), got, y, y_scale)


@pytest.mark.parametrize("mask", [None, "some", "tail", "none"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("y,y_scale,row_scale", [("16", 0.0, False), ("e4m3", 0.0, True), ("e5m2", 2.0 ** -9, False)])
def test_forward_without_a_residual(mask, dt, y, y_scale, row_scale):
    c = Case(77, 448, dt, mask, weight="f32")
    got = c.fwd(y=y, y_scale=y_scale, row_scale=row_scale)
    s = c.clean(c.x)
    check_y(c, s, got, y, y_scale)
    if y == "16" and mask != "none":
        assert (np.abs(host(got["y"])) > 4 * R.y_bound(host(got["y"]), 448, dt)).mean() > 0.2
    again = c.fwd(y=y, y_scale=y_scale, sum_out=True, ckpt=True)     # other outputs beside it: the same y
    assert same(got["y"], again["y"]) and np.array_equal(host(again["sum"]), s)


@pytest.mark.parametrize("eps", [2.0 ** -126, 1e-12, 1e-5, 1.0, 1e30])
def test_forward_eps_and_tiny_rows(eps):
    c = Case(12, 256, "bf16", scale=1.0)
    c.x[3] = 0
    c.x[4] *= 1e-18
    c.x[5] = 0
    c.x[5, 7] = 1.0
    check_y(c, host(c.x), c.fwd(eps=eps), "16", 0.0, float(np.float32(eps)))
    got = c.fwd(y="e4m3", eps=eps)
    check_y(c, host(c.x), got, "e4m3", 0.0, float(np.float32(eps)))
    assert not host(got["y"])[3].any() and float(got["scale"][3]) == R.LEAST


def test_saturation_and_values_that_are_not_finite():
    c = Case(6, 128, "bf16")
    c.x[1, 5] = float("inf")
    c.x[2, 6] = float("nan")
    for y, scale in (("16", 0.0), ("e4m3", 0.0), ("e4m3", 2.0 ** -20), ("e5m2", 2.0 ** -20)):
        got = c.fwd(y=y, y_scale=scale, ckpt=True)
        v = host(got["y"])
        assert np.isnan(v[1, 5]) and not np.delete(v[1], 5).any()     # 1 / sqrt(inf) = 0; inf * 0
        assert np.isnan(v[2]).all()
        assert np.isfinite(v[[0, 3, 4, 5]]).all()
        if scale:
            assert np.abs(v[[0, 3, 4, 5]]).max() == R.LARGEST[y]
        s = host(got["scales"])
        assert not np.isfinite(s[1, 0]) and np.isfinite(s[1, 1]) and np.isnan(s[2, 0]) and np.isfinite(s[2, 1])
        back = host(c.unpack((got["codes"], got["scales"])))
        assert np.isnan(back[1, :64]).all() and np.isfinite(back[1, 64:]).all() and np.isnan(back[2, :64]).all()


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_in_place(dt):
    """sum_out may be x or the residual."""
    c = Case(50, 512, dt, "some")
    want = c.fwd(residual=True, sum_out=True)
    for which in ("x", "r"):
        x, r = c.x.clone(), c.r.clone()
        y = torch.empty_like(x)
        rg.grpo_norm_fwd(x, r, c.w, c.mask, c.shape, rg.norm_opts(eps=EPS, y_type=DT[dt]), y, None, x if which == "x" else r)
        assert same(y, want["y"]) and same(x if which == "x" else r, want["sum"])


# ---------------------------------------------------------------- checkpoints

@pytest.mark.parametrize("N,d", SIZES + [(3, 65536)])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("mask", [None, "some"])
def test_checkpoints(N, d, dt, mask):
    c = Case(N, d, dt, mask if N > 1 else None)
    clean = torch.from_numpy(c.clean(c.x)).to(c.x.dtype).cuda()
    codes, scales = c.pack()
    wc, ws = torch_pack(clean)
    assert torch.equal(codes, wc) and same(scales, ws)
    back = c.unpack((codes, scales))
    want = (codes.view(N, -1, 64).float() * scales.float()[:, :, None]).view(N, d).to(c.x.dtype)
    assert np.array_equal(host(back), host(want))
    x = host(clean)
    assert np.all(np.abs(host(back) - x) <= R.ckpt_bound(x, host(scales), dt))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_checkpoints_at_the_ends_of_the_type(dt):
    c = Case(8, 128, dt)
    top = float(torch.finfo(R.TORCH[dt]).max)
    c.x[0] = top
    c.x[1] = -top
    c.x[2, ::2] = top
    c.x[3] = float(torch.finfo(R.TORCH[dt]).tiny)
    c.x[4] = 0.0
    c.x[4, 3] = -float(torch.finfo(R.TORCH[dt]).smallest_normal) / 4
    c.x[5, 100] = float("inf")
    c.x[6, 3] = float("nan")
    codes, scales = c.pack()
    back, x = host(c.unpack((codes, scales))), host(c.x)
    fine = np.isfinite(x).reshape(8, 2, 64).all(2).repeat(64, 1)
    assert np.isfinite(back[fine]).all() and np.isnan(back[~fine]).all()
    each = np.repeat(host(scales), 64, axis=1)
    assert np.all(np.abs(back - x)[fine] <= (1.0 * each + R.HALF_STEP[dt] * np.abs(x) + R.TINY[dt])[fine])
    assert np.all(np.abs(back - x)[3:5] <= R.ckpt_bound(x, host(scales), dt)[3:5])
    assert int(codes.min()) >= -127


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_checkpoint_scales_of_every_size(dt):
    """Each positive finite number of the type as a block's largest value: scales and codes are the definition's bit for bit, so
    the reciprocal of every scale is the correctly rounded one.  (Blocks whose scale would be past its limit are left to
    the test above.)"""
    t = R.TORCH[dt]
    limit = 2.0 ** 121 if dt == "bf16" else 512.0
    top = torch.arange(1, 0x7f80 if dt == "bf16" else 0x7c00, dtype=torch.int32).to(torch.int16).view(t)
    top = top[(top.double() / 127 <= limit)]
    n = (len(top) + 1) // 2 * 2
    top = torch.cat([top, top[:n - len(top)]])
    part = torch.linspace(-1, 1, 63, dtype=torch.float64)
    x = torch.cat([top.double()[:, None], top.double()[:, None] * part], 1).to(t).view(n // 2, 128).cuda()
    c = Case(n // 2, 128, dt)
    codes, scales = c.pack(x)
    wc, ws = torch_pack(x)
    assert same(scales, ws) and torch.equal(codes, wc)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("y", ["16", "e4m3"])
def test_norm_of_a_checkpoint_is_the_norm_of_its_values(dt, y):
    for N, d in ((1, 64), (60, 1536), (9, 4160), (2, 16384)):
        c = Case(N, d, dt, "some" if N > 1 else None)
        ck = c.pack()
        x = c.unpack(ck)
        a, b = c.fwd(x=ck, y=y, sum_out=True), c.fwd(x=x, y=y, sum_out=True)
        assert same(a["y"], b["y"]) and np.array_equal(host(a["sum"]), host(x))
        ga, gb = c.bwd(x=ck, dsum=True), c.bwd(x=x, dsum=True)
        assert same(ga[0], gb[0]) and same(ga[1], gb[1]) and ga[2] == gb[2] == 0


# ---------------------------------------------------------------- gradient

def check_grad(c, s, dsum, dweight, got, eps=EPS):
    dx, dw, inf = got
    dy = np.where(c.keep[:, None], np.nan_to_num(host(c.dy)), 0.0)
    rx, rw, bx, bw = R.norm_grad(s, c.weight(), dy, eps)
    if dsum:
        rx = rx + c.clean(c.ds)
        bx = bx + 2.0 ** -24 * np.abs(rx)
    rx[~c.keep] = 0.0
    assert np.all(np.abs(host(dx) - rx) <= R.rounding(rx, bx, c.dt))
    assert not host(dx)[~c.keep].any()
    if dweight:
        assert np.all(np.abs(host(dw) - rw) <= R.rounding(rw, bw, "f32" if c.weight_f32 else c.dt))
    assert inf == 0
    return rx, bx, rw, bw


@pytest.mark.parametrize("N,d", SIZES + [(700, 448)])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("dsum,dweight,ckpt", [(False, True, False), (True, True, False), (True, False, True), (False, True, True)])
def test_gradient(N, d, dt, dsum, dweight, ckpt):
    c = Case(N, d, dt, "some" if N > 1 else None, weight="f32" if dsum else "16", plus_one=N % 2 == 1)
    ck = c.pack() if ckpt else None
    got = c.bwd(x=ck, dsum=dsum, dweight=dweight)
    s = host(c.unpack(ck)) if ckpt else c.clean(c.x)
    rx, bx, rw, bw = check_grad(c, s, dsum, dweight, got)
    assert (np.abs(rx[c.keep]) > 4 * R.rounding(rx, bx, dt)[c.keep]).mean() > 0.4     # zeros would not pass
    again = c.bwd(x=ck, dsum=dsum, dweight=dweight)
    assert same(got[0], again[0]) and (not dweight or same(got[1], again[1]))


@pytest.mark.parametrize("mask", ["none", "tail"])
def test_gradient_masks(mask):
    c = Case(90, 256, "bf16", mask)
    got = c.bwd(dsum=True)
    check_grad(c, c.clean(c.x), True, True, got)
    if mask == "none":
        assert not host(got[0]).any() and not host(got[1]).any()


@pytest.mark.parametrize("d,eps", [(64, 1e-6), (320, 0.5)])
def test_gradient_is_the_differences(d, eps):
    """Along random directions, the differences of the loss in 64 bits against the kernel's gradients."""
    c = Case(20, d, "bf16", weight="f32")
    dx, dw, _ = c.bwd(eps=eps)
    s, w, dy, h = host(c.x), c.weight(), host(c.dy), 1e-4
    _, _, bx, bw = R.norm_grad(s, w, dy, eps)
    bx, bw = R.rounding(host(dx), bx, "bf16"), R.rounding(host(dw), bw, "f32")
    f = lambda s, w: (R.norm(s, w, eps)[0] * dy).sum()  # noqa: E731
    for _ in range(6):
        u, v = c.rng.normal(size=s.shape) * np.abs(s).max(1, keepdims=True), c.rng.normal(size=d)
        want = (f(s + h * u, w + h * v) - f(s - h * u, w - h * v)) / (2 * h)
        third = h * h * 100 * (np.abs(host(dx) * u).sum() + np.abs(host(dw) * v).sum())   # the differences' own error
        assert abs((host(dx) * u).sum() + (host(dw) * v).sum() - want) <= (bx * np.abs(u)).sum() + (bw * np.abs(v)).sum() + third


def test_found_inf():
    c = Case(40, 128, "fp16", "tail")
    assert c.bwd()[2] == 0                         # NaN in rows that do not count
    c.dy[7, 3] = 60000.0
    c.x[7] *= 1e-3                                 # rstd of about 1000: dx overflows
    dx, dw, inf = c.bwd()
    assert inf == 1 and not np.isfinite(host(dx)[7]).all() and np.isfinite(host(dx)[8]).all()
    assert c.bwd(dweight=False)[2] == 1
    c = Case(4000, 64, "fp16")
    c.x[:] = 1.0
    c.dy[:] = 100.0                                # dx is about 20, dw = 400000 in fp16 is not finite
    dx, dw, inf = c.bwd()
    assert inf == 1 and np.isfinite(host(dx)).all() and not np.isfinite(host(dw)).any()
    assert c.bwd(dweight=False)[2] == 0
    c = Case(10, 64, "bf16")
    c.dy[9, 63] = float("nan")
    assert c.bwd()[2] == 1


@pytest.mark.parametrize("which", ["dy", "dsum", "x"])
def test_gradient_in_place(which):
    c = Case(333, 320, "bf16", "some")
    want = c.bwd(dsum=True)
    t = {"dy": c.dy.clone(), "dsum": c.ds.clone(), "x": c.x.clone()}
    dw, inf = torch.empty_like(c.w), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(rg.grpo_norm_workspace_bytes(c.shape), dtype=torch.uint8, device="cuda")
    rg.grpo_norm_bwd(t["dy"], t["x"], c.w, t["dsum"], c.mask, c.shape, rg.norm_opts(eps=EPS), ws, t[which], dw, inf)
    assert same(t[which], want[0]) and same(dw, want[1])


# ---------------------------------------------------------------- sizes, streams, graphs, threads

def test_offsets_beyond_32_bits():
    """More than 2^32 bytes and 2^31 elements: the last rows are the same as in a call of their own."""
    d, tail = 4096, 8
    N = (1 << 31) // d + 300
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(N, d, device="cuda", generator=g, dtype=torch.bfloat16)
    w = torch.randn(d, device="cuda", generator=g, dtype=torch.bfloat16)
    s, one = rg.make_shape(1, 1, N, d, 1), rg.make_shape(1, 1, tail, d, 1)
    o = rg.norm_opts()
    ck = torch.empty(N, d, dtype=torch.int8, device="cuda"), torch.empty(N, d // 64, dtype=torch.bfloat16, device="cuda")
    y, t = torch.empty_like(x), x[-tail:].contiguous()
    rg.grpo_norm_fwd(x, None, w, None, s, o, y, None, None, ck)
    yt, ct = torch.empty_like(t), tuple(torch.empty_like(a[-tail:]) for a in ck)
    rg.grpo_norm_fwd(t, None, w, None, one, o, yt, None, None, ct)
    assert same(y[-tail:], yt) and all(same(a[-tail:], b) for a, b in zip(ck, ct))
    rg.grpo_ckpt_pack(x, None, s, ck)
    assert all(same(a[-tail:], b) for a, b in zip(ck, ct))
    rg.grpo_ckpt_unpack(ck, None, s, y)
    back = torch.empty_like(t)
    rg.grpo_ckpt_unpack(ct, None, one, back)
    assert same(y[-tail:], back)
    ws = torch.empty(rg.grpo_norm_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    inf = torch.zeros(1, dtype=torch.int32, device="cuda")
    for src, st in ((x, t), (ck, ct)):
        rg.grpo_norm_bwd(x, src, w, None, None, s, o, ws, y, None, inf)
        rg.grpo_norm_bwd(t, st, w, None, None, one, o, ws, back, None, inf)
        assert same(y[-tail:], back)


def _everything(c, keep):
    """Calls of all entry points, as a step makes them, into the buffers of `keep`."""
    o8 = rg.norm_opts(eps=EPS, y_type=rg.E4M3, y_scale=0.05)
    o = rg.norm_opts(eps=EPS)
    rg.grpo_norm_fwd(c.x, c.r, c.w, c.mask, c.shape, o8, keep["y8"], keep["scale"], keep["sum"], keep["ck"])
    rg.grpo_norm_fwd(keep["ck"], None, c.w, c.mask, c.shape, o, keep["y"])
    rg.grpo_norm_bwd(c.dy, keep["ck"], c.w, c.ds, c.mask, c.shape, o, keep["ws"], keep["dx"], keep["dw"], keep["inf"])
    rg.grpo_ckpt_pack(keep["y"], c.mask, c.shape, keep["ck2"])
    rg.grpo_ckpt_unpack(keep["ck2"], c.mask, c.shape, keep["x"])


def _buffers(c):
    e = lambda t, *n: torch.full(n, 3, dtype=t, device="cuda")  # noqa: E731
    b, N, d = torch.bfloat16, c.N, c.d
    return {"y8": torch.zeros(N, d, dtype=torch.uint8, device="cuda"), "scale": e(torch.float32, N), "sum": e(b, N, d),
            "ck": (e(torch.int8, N, d), e(b, N, d // 64)), "ck2": (e(torch.int8, N, d), e(b, N, d // 64)), "y": e(b, N, d),
            "x": e(b, N, d), "dx": e(b, N, d), "dw": e(b, d), "inf": e(torch.int32, 1),
            "ws": torch.empty(rg.grpo_norm_workspace_bytes(c.shape), dtype=torch.uint8, device="cuda")}


def _results(k):
    return [x.clone() for n in ("y8", "scale", "sum", "y", "x", "dx", "dw", "inf") for x in (k[n],)] + [
        x.clone() for n in ("ck", "ck2") for x in k[n]]


def _all_same(a, b):
    return all(same(x, y) for x, y in zip(a, b))


def test_streams_and_graphs():
    """Two calls in flight at once on two streams, and replays of a captured step, give the bits of calls in turn; new
    inputs in the captured buffers give theirs."""
    a, b = Case(900, 1536, "bf16", "some"), Case(333, 4160, "bf16", "tail")
    ka, kb = _buffers(a), _buffers(b)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    _everything(a, ka)
    _everything(b, kb)
    torch.cuda.synchronize()
    wa, wb = _results(ka), _results(kb)
    for _ in range(3):
        ka, kb = _buffers(a), _buffers(b)
        torch.cuda.synchronize()
        for c, k, st in ((a, ka, s1), (b, kb, s2)):
            with torch.cuda.stream(st):
                _everything(c, k)
        torch.cuda.synchronize()
        assert _all_same(_results(ka), wa) and _all_same(_results(kb), wb)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _everything(a, ka)
    for _ in range(2):
        for k in ("y8", "sum", "dx", "dw"):
            ka[k].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert _all_same(_results(ka), wa)
    other = Case(900, 1536, "bf16", "tail", seed=5)
    fresh = _buffers(other)
    _everything(other, fresh)
    for n in ("x", "r", "dy", "ds", "w", "mask"):
        getattr(a, n).copy_(getattr(other, n))
    graph.replay()
    torch.cuda.synchronize()
    assert _all_same(_results(ka), _results(fresh))


def test_a_captured_fork_and_join():
    """Calls that wait for two streams, captured and replayed, and next to other kernels, copies and memsets on their own."""
    c = Case(600, 1536, "bf16")
    o = rg.norm_opts(eps=EPS)
    ws = torch.empty(rg.grpo_norm_workspace_bytes(c.shape), dtype=torch.uint8, device="cuda")
    y, y2, dx, dw = torch.empty_like(c.x), torch.empty_like(c.x), torch.empty_like(c.x), torch.empty_like(c.w)
    dy, x = torch.empty_like(c.x), torch.empty_like(c.x)
    inf = torch.zeros(1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()

    def go():
        main = torch.cuda.current_stream()
        x.copy_(c.x)
        side.wait_stream(main)
        rg.grpo_norm_fwd(x, None, c.w, None, c.shape, o, y)
        with torch.cuda.stream(side):
            y2.zero_()
            rg.grpo_norm_fwd(x, c.r, c.w, None, c.shape, o, y2)
            dy.copy_(y2)
        main.wait_stream(side)
        rg.grpo_norm_bwd(dy, y, c.w, y2, None, c.shape, o, ws, dx, dw, inf)
        dx.mul_(0.5)
        rg.grpo_norm_bwd(dx, y, c.w, None, None, c.shape, o, ws, dx, dw, inf)

    go()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, y2, dx, dw, inf)]
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        go()
    for _ in range(3):
        for t in (y, y2, dx, dw):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert _all_same([y, y2, dx, dw, inf], want)


def test_two_host_threads():
    a, b = Case(500, 1536, "bf16", "some"), Case(1, 4096, "bf16")
    ka, kb = _buffers(a), _buffers(b)
    _everything(a, ka)
    _everything(b, kb)
    torch.cuda.synchronize()
    wa, wb = _results(ka), _results(kb)
    errors = []

    def work(c, k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    _everything(c, k)
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=x) for x in ((a, ka), (b, kb))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and _all_same(_results(ka), wa) and _all_same(_results(kb), wb)


def test_two_host_threads_with_different_shared_memory():
    """The same kernel with 30 KB a block from one thread and 200 KB from another, first and in turn: no call takes the other's
    permission away."""
    cases = [Case(300, 1536, "fp16"), Case(40, 8128, "fp16"), Case(200, 5120, "fp16")]
    want = [c.bwd(dsum=True) for c in cases]
    start, errors = threading.Barrier(3), []

    def work(c, w):
        try:
            start.wait(timeout=60)
            with torch.cuda.stream(torch.cuda.Stream()):
                o, ws = rg.norm_opts(eps=EPS), torch.empty(rg.grpo_norm_workspace_bytes(c.shape), dtype=torch.uint8, device="cuda")
                dx, dw, inf = torch.empty_like(c.dy), torch.empty_like(c.w), torch.zeros(1, dtype=torch.int32, device="cuda")
                for _ in range(300):
                    rg.grpo_norm_bwd(c.dy, c.x, c.w, c.ds, None, c.shape, o, ws, dx, dw, inf)
                torch.cuda.current_stream().synchronize()
                assert same(dx, w[0]) and same(dw, w[1])
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=x) for x in zip(cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_rows_alone_or_together():
    """A row's y, checkpoint and dx do not depend on the rows beside it."""
    c = Case(257, 1536, "bf16")
    whole, grad = c.fwd(residual=True, y="e4m3", ckpt=True), c.bwd(dsum=True)[0]
    for t in (0, 100, 256):
        one = Case(1, 1536, "bf16")
        for n in ("x", "r", "dy", "ds"):
            setattr(one, n, getattr(c, n)[t:t + 1].contiguous())
        one.w = c.w
        got = one.fwd(residual=True, y="e4m3", ckpt=True)
        assert all(same(got[k], whole[k][t:t + 1]) for k in got)
        assert same(one.bwd(dsum=True)[0], grad[t:t + 1])


def test_profile_counts_the_launches():
    c = Case(10, 128, "bf16")
    k = _buffers(c)
    before = rg.grpo_kernel_launches()
    rg.grpo_profile_enable(True)
    try:
        rg.grpo_profile_collect()
        _everything(c, k)
        torch.cuda.synchronize()
        got = rg.grpo_profile_collect()
    finally:
        rg.grpo_profile_enable(False)
    assert got["norm"][1] == 2 and got["norm_bwd"][1] in (1, 2) and got["ckpt"][1] == 2
    assert rg.grpo_kernel_launches() - before == sum(n for _, n in got.values())


# ---------------------------------------------------------------- many rows: blocks that take several, rings, lookahead

def gpu64(c, s, dsum):
    """y's and the gradient's definitions in 64 bits on the GPU, with the bounds of norm_reference."""
    d, e = c.d, R.rel32(c.d)
    w, keep = c.w.double() + c.plus_one, torch.from_numpy(c.keep).cuda()[:, None]
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    s = torch.where(keep, s.double(), zero)
    dy = torch.where(keep, c.dy.double(), zero)
    rstd = 1 / torch.sqrt((s * s).mean(1, keepdim=True) + EPS)
    y = s * rstd * w
    g = dy * w
    dx = rstd * (g - s * rstd ** 2 * (g * s).mean(1, keepdim=True))
    bx = 4 * e * rstd * (g.abs() + s.abs() * rstd ** 2 * (g * s).abs().mean(1, keepdim=True))
    if dsum:
        ds = torch.where(keep, c.ds.double(), zero)
        dx, bx = dx + ds, bx + 2.0 ** -24 * (dx + ds).abs()
    each = dy * s * rstd
    return y, dx, bx, each.sum(0), (4 * e + (c.N + 16) * R.STEP32) * each.abs().sum(0)


def within(got, want, bound, dtype):
    return bool(((got.double() - want).abs() <= bound + R.HALF_STEP[dtype] * (want.abs() + bound) + R.TINY[dtype]).all())


MANY = [(40000, 64), (30001, 192), (20000, 512), (9999, 576), (9000, 1088), (10001, 2048), (12000, 4096), (3000, 5120),
        (2000, 6208), (1500, 8192), (900, 16384)]


@pytest.mark.parametrize("N,d", MANY)
@pytest.mark.parametrize("mask", ["some", "runs"])
@pytest.mark.parametrize("dsum,ckpt", [(False, False), (True, False), (False, True), (True, True)])
def test_many_rows(N, d, mask, dsum, ckpt):
    """More rows than blocks, with masks that leave whole windows of rows out, and others in part."""
    dt = "fp16" if N % 2 else "bf16"
    c = Case(N, d, dt, weight="f32" if dsum else "16", seed=3)
    if mask == "runs":                       # runs of 1 to 5000 rows that count or do not
        ends = np.cumsum(np.exp(c.rng.uniform(0, np.log(5000), size=4000)).astype(int))
        c.m = np.searchsorted(ends, np.arange(N), side="right") % 2 == 0
    else:
        c.m = c.rng.random(N) < 0.7
    c.keep = c.m
    c.mask = torch.from_numpy(c.m.astype(np.uint8)).cuda()
    out = torch.from_numpy(~c.keep).cuda()
    for t in (c.x, c.r, c.dy, c.ds):
        t[out] = float("nan")
    ck = c.pack() if ckpt else None
    s = c.unpack(ck) if ckpt else c.x
    y, dx, bx, dw, bw = gpu64(c, s, dsum)
    got = c.fwd(x=ck)["y"]
    assert within(got, y, R.rel32(d) * y.abs(), dt)
    gx, gw, inf = c.bwd(x=ck, dsum=dsum)
    dx[out] = 0.0
    assert inf == 0 and not bool(gx[out].any())
    assert within(gx, dx, bx, dt) and within(gw, dw, bw, "f32" if c.weight_f32 else dt)


@pytest.mark.parametrize("d", [64, 128, 192, 512, 576, 4096])
@pytest.mark.parametrize("turns", [1, 2, 3, 7, 8, 9, 15, 16, 17])
def test_few_turns_of_rows(d, turns):
    """Grids of one cluster, and the first ones beyond."""
    rows = {64: 32, 128: 16, 192: 8, 512: 4}.get(d, 1)
    for N in {turns * rows, max(1, turns * rows - rows + 1)}:
        c = Case(N, d, "bf16", "some" if N > 3 else None)
        check_grad(c, c.clean(c.x), True, True, c.bwd(dsum=True))
        assert c.bwd(dsum=True, dweight=False)[2] == 0
        c.dy[int(np.flatnonzero(c.keep)[-1]), d - 1] = float("inf")
        assert c.bwd()[2] == 1 and c.bwd(dweight=False)[2] == 1


@pytest.mark.parametrize("d", [6208, 8192, 16384])
@pytest.mark.parametrize("N", [1, 8, 9, 16, 17])
@pytest.mark.parametrize("dsum,ckpt", [(True, False), (False, True), (True, True)])
def test_the_widest_rows_of_one_cluster(d, N, dsum, ckpt):
    """Up to eight blocks of a cluster, each with most of an SM's shared memory, and the first grid beyond."""
    c = Case(N, d, "fp16" if N % 2 else "bf16", "some" if N > 3 else None, weight="f32")
    ck = c.pack() if ckpt else None
    check_grad(c, host(c.unpack(ck)) if ckpt else c.clean(c.x), dsum, True, c.bwd(x=ck, dsum=dsum))


@pytest.mark.parametrize("N,d", [(40, 64), (40, 1536)])
def test_weights_that_are_not_finite(N, d):
    """They reach their own column of the rows that count, and nothing of the others."""
    c = Case(N, d, "bf16", "some", weight="f32")
    c.w[3], c.w[5] = float("inf"), float("nan")
    for y in ("16", "e4m3"):
        v = host(c.fwd(y=y, y_scale=0.0 if y == "16" else 0.05, row_scale=False)["y"])
        assert not v[~c.keep].any() and np.isnan(v[c.keep, 5]).all()
        assert np.isfinite(np.delete(v, (3, 5), 1)).all()
        assert (np.isinf(v) if y == "16" else np.abs(v) == 448)[c.keep, 3].all()
    dx, _, inf = c.bwd()
    assert inf == 1 and not host(dx)[~c.keep].any()


def test_checked_build_gives_the_same_bits(monkeypatch):
    from rl_fine_tuning_gb300 import build
    c = Case(500, 1536, "bf16", "some")
    k = _buffers(c)
    _everything(c, k)
    torch.cuda.synchronize()
    want = _results(k)
    monkeypatch.setattr(build, "LIB", build.LIB_CHECKED)
    monkeypatch.setattr(rg, "_lib", None)
    assert rg.grpo_device_checks()
    k = _buffers(c)
    _everything(c, k)
    torch.cuda.synchronize()
    assert _all_same(_results(k), want)


def test_calls_follow_one_another_without_waits():
    """Each call's input is the output of the one before, over and over on one stream, with other kernels between: the same
    bits as with the device waited for after each."""
    c = Case(700, 1536, "bf16")
    o = rg.norm_opts(eps=EPS)
    e = torch.empty_like
    ws = torch.empty(rg.grpo_norm_workspace_bytes(c.shape), dtype=torch.uint8, device="cuda")
    ck = torch.empty(c.N, c.d, dtype=torch.int8, device="cuda"), torch.empty(c.N, c.d // 64, dtype=torch.bfloat16, device="cuda")

    def go(wait):
        x, r, dx, dw = c.x.clone(), c.r.clone(), e(c.x), e(c.w)
        y, inf = e(c.x), torch.zeros(1, dtype=torch.int32, device="cuda")
        for i in range(12):
            for call in (lambda: rg.grpo_norm_fwd(x, r, c.w, None, c.shape, o, y, None, r, ck),
                         lambda: rg.grpo_ckpt_unpack(ck, None, c.shape, x),
                         lambda: rg.grpo_norm_bwd(y, ck, c.w, x, None, c.shape, o, ws, dx, dw, inf),
                         lambda: x.add_(dx, alpha=0.1),
                         lambda: rg.grpo_ckpt_pack(x, None, c.shape, ck),
                         lambda: rg.grpo_norm_bwd(x, ck, c.w, None, None, c.shape, o, ws, x, dw, inf)):
                call()
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return [x, r, y, dx, dw, *ck]

    want = [t.clone() for t in go(True)]
    for _ in range(3):
        assert _all_same(go(False), want)


def test_binding_checks_tensors():
    c = Case(4, 64, "bf16")
    o = rg.norm_opts()
    y = torch.empty_like(c.x)
    for bad in (c.x.cpu(), c.x.half(), c.x[:3], torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")[:, :64]):
        with pytest.raises(ValueError):
            rg.grpo_norm_fwd(bad, None, c.w, None, c.shape, o, y)
        with pytest.raises(ValueError):
            rg.grpo_norm_fwd(c.x, bad, c.w, None, c.shape, o, y)
        with pytest.raises(ValueError):
            rg.grpo_ckpt_unpack((torch.empty_like(y, dtype=torch.int8), y.new_empty(4)), None, c.shape, bad)
    with pytest.raises(ValueError):
        rg.grpo_norm_fwd(c.x, None, c.w.float(), None, c.shape, o, y)
    with pytest.raises(ValueError):
        rg.grpo_norm_fwd(c.x, None, c.w, None, c.shape, rg.norm_opts(y_type=rg.E4M3), y, torch.empty(4, device="cuda"))
    with pytest.raises(rg.GrpoError):
        rg.grpo_norm_fwd(c.x, None, c.w, None, c.shape, o, y, torch.empty(4, device="cuda"))
    with pytest.raises(rg.GrpoError):
        rg.grpo_norm_bwd(c.dy, c.x, c.w, None, None, c.shape, o, torch.empty(256, dtype=torch.uint8, device="cuda"), y, c.w,
                         torch.zeros(1, dtype=torch.int32, device="cuda"))


# ---------------------------------------------------------------- gradients from a checkpoint, many rows

def _gpu_stream(N, d, dt="bf16", seed=0):
    """dy and a checkpoint of random rows, made on the device."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, dy = (torch.randn(N, d, device="cuda", generator=g).to(R.TORCH[dt]) for _ in range(2))
    ck = torch.empty(N, d, dtype=torch.int8, device="cuda"), torch.empty(N, d // 64, dtype=torch.bfloat16, device="cuda")
    rg.grpo_ckpt_pack(x, None, rg.make_shape(1, 1, N, d, 1, DT[dt]), ck)
    return dy, ck


def _ckpt_grad(dy, ck, w, dt="bf16"):
    N, d = dy.shape
    s = rg.make_shape(1, 1, N, d, 1, DT[dt])
    ws = torch.empty(rg.grpo_norm_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    dx, dw, inf = torch.empty_like(dy), torch.empty_like(w), torch.zeros(1, dtype=torch.int32, device="cuda")
    rg.grpo_norm_bwd(dy, ck, w, None, None, s, rg.norm_opts(eps=EPS), ws, dx, dw, inf)
    return dx, dw, inf


@pytest.mark.parametrize("N", [9700, 9728, 40000])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("mask", [None, "some"])
def test_gradient_of_rows_in_one_warp(N, dt, mask):
    """1024 columns from a checkpoint, after calls of other widths, which leave their rows' sums in shared memory: within the
    bounds, and the same bits each time."""
    c = Case(N, 1024, dt, mask, seed=11)
    ck = c.pack()
    _, dx, bx, dw, bw = gpu64(c, c.unpack(ck), False)
    dx[~torch.from_numpy(c.keep).cuda()] = 0.0
    first = None
    for d in (2048, 4096, 512):
        other = _gpu_stream(9728, d, dt)
        _ckpt_grad(*other, torch.ones(d, dtype=R.TORCH[dt], device="cuda"), dt)
        gx, gw, inf = c.bwd(x=ck)
        assert inf == 0 and within(gx, dx, bx, dt) and within(gw, dw, bw, dt)
        first = first or (gx, gw)
        assert same(gx, first[0]) and same(gw, first[1])


@pytest.mark.parametrize("d", [1024, 2048, 4096, 6144, 8192])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_rows_from_a_checkpoint_alone_or_together(d, dt):
    """dx of a row from a checkpoint does not depend on how many rows are beside it."""
    dy, ck = _gpu_stream(10000, d, dt, seed=d)
    w = torch.ones(d, dtype=R.TORCH[dt], device="cuda")
    whole = _ckpt_grad(dy, ck, w, dt)[0]
    for a, b in ((0, 1), (3, 20), (100, 1000), (9990, 10000), (0, 9727)):
        part = _ckpt_grad(dy[a:b], (ck[0][a:b], ck[1][a:b]), w, dt)[0]
        assert same(part, whole[a:b]), (a, b)


# ---------------------------------------------------------------- together with the losses

def _chain(dt8):
    """One prompt group through norm, loss and back; returns what both references need."""
    G, L, d, V = 4, 60, 256, 700
    c = Case(G * L, d, "bf16", "some", seed=9)
    c.shape = rg.make_shape(1, G, L, d, V)
    rng = c.rng
    W = torch.from_numpy(rng.normal(size=(V, d)) * d ** -0.5).to(torch.bfloat16).cuda()
    tok = torch.from_numpy(rng.integers(0, V, G * L).astype(np.int32)).cuda()
    adv = torch.from_numpy(rng.normal(size=G).astype(np.float32)).cuda()
    return c, W, tok, adv


def test_norm_clipped_loss_and_back():
    """norm (keeping a checkpoint) -> log-probs and clipped loss -> the norm's gradient, against 64 bits end to end."""
    c, W, tok, adv = _chain(False)
    N, d, sh = c.N, c.d, c.shape
    y = torch.empty_like(c.x)
    ck = torch.empty(N, d, dtype=torch.int8, device="cuda"), torch.empty(N, d // 64, dtype=torch.bfloat16, device="cuda")
    sm = torch.empty_like(c.x)
    o = rg.norm_opts(eps=EPS)
    rg.grpo_norm_fwd(c.x, c.r, c.w, c.mask, sh, o, y, None, sm, ck)
    ws = torch.empty(max(rg.grpo_policy_workspace_bytes(sh, k) for k in ("logp", "clip")), dtype=torch.uint8, device="cuda")
    old, status = torch.empty(N, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    rg.grpo_logprobs(y, W, tok, c.mask, sh, 1.0, ws, old, None, status)
    loss, dW, dH = torch.empty(1, device="cuda"), torch.empty_like(W), torch.empty_like(y)
    inf, inf2 = torch.ones(1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    s0 = rg.make_shape(1, sh.G, sh.L, d, sh.V, beta=0.0)
    rg.grpo_clip_loss_fwd_bwd(y, W, tok, c.mask, adv, old, None, s0, rg.clip_opts(), 1.0, ws, loss, dH, dW, inf, None, status)
    nws = torch.empty(rg.grpo_norm_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
    grads = []
    for src in (sm, ck):
        dx, dw = torch.empty_like(y), torch.empty_like(c.w)
        rg.grpo_norm_bwd(dH, src, c.w, None, c.mask, sh, o, nws, dx, dw, inf2)
        grads.append((host(dx), host(dw)))
    assert int(status) == 0 and int(inf) == 0 and int(inf2) == 0
    # 64 bits: ratios are 1, so the loss is -sum over the rows of A q / rows
    S = torch.from_numpy(R.stream(c.clean(c.x), c.clean(c.r), "bf16")).requires_grad_()
    w = c.w.double().cpu().requires_grad_()
    h = S / torch.sqrt((S * S).mean(1, keepdim=True) + EPS) * w
    q = torch.log_softmax(h @ W.double().cpu().t(), 1)[torch.arange(N), tok.cpu().long()]
    keep = torch.from_numpy(c.keep)
    A = adv.double().cpu().repeat_interleave(sh.L)
    (-(A * torch.exp(q - q.detach()))[keep].sum() / keep.sum()).backward()
    # roundings on the way: h, dlogits, dH to bf16, each a relative error of at most 2^-8 of its matrix's entries, summed
    # over a row or a column of products that add up like random ones: together below 3% of the norm, the checkpoint's
    # (0.501 of a scale, at most 1/127 of the block's largest) below 6%
    for (dx, dw), tol in zip(grads, (0.03, 0.06)):
        for got, want in ((dx, S.grad.numpy()), (dw, w.grad.numpy())):
            assert np.linalg.norm(got - want) <= tol * np.linalg.norm(want)


def test_norm_to_8_bits_grpo_loss_and_back():
    """norm to E4M3 codes with one scale -> the 8-bit GRPO loss -> the norm's gradient: the loss is the definition's at the
    codes' values, and the gradients are the chain's."""
    c, W, tok, adv = _chain(True)
    N, d = c.N, c.d
    sh = rg.make_shape(1, 4, 60, d, 700, rg.E4M3)
    y, yr = torch.empty(N, d, dtype=torch.uint8, device="cuda"), torch.empty(N, d, dtype=torch.uint8, device="cuda")
    scale = float(np.sqrt(d) * c.w.abs().max() / 448)            # nothing saturates
    o = rg.norm_opts(eps=EPS, y_type=rg.E4M3, y_scale=scale)
    sm = torch.empty_like(c.x)
    rg.grpo_norm_fwd(c.x, c.r, c.w, c.mask, c.shape, o, y, None, sm)
    rg.grpo_norm_fwd(c.x, None, c.w, c.mask, c.shape, o, yr)     # the reference model's
    w_scale = 2.0 ** -9
    W8 = (W.float() / w_scale).to(torch.float8_e4m3fn)
    ws = torch.empty(rg.grpo_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
    loss, dW = torch.empty(1, device="cuda"), torch.empty(700, d, device="cuda")
    dH, status = torch.empty(N, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    rg.grpo_loss_fwd_bwd_fp8(y, yr, W8.view(torch.uint8), scale, scale, w_scale, tok, c.mask, adv, sh, ws, loss, dH, dW, None,
                             status)
    nws = torch.empty(rg.grpo_norm_workspace_bytes(c.shape), dtype=torch.uint8, device="cuda")
    dx, dw, inf = torch.empty_like(c.x), torch.empty_like(c.w), torch.ones(1, dtype=torch.int32, device="cuda")
    rg.grpo_norm_bwd(dH, sm, c.w, None, c.mask, c.shape, rg.norm_opts(eps=EPS), nws, dx, dw, inf)
    assert int(status) == 0 and int(inf) == 0
    dec = lambda a, s: a.view(torch.float8_e4m3fn).double().cpu() * float(np.float32(s))  # noqa: E731
    h, hr, Wd = dec(y, scale).requires_grad_(), dec(yr, scale), dec(W8, w_scale)
    idx, keep = torch.arange(N), torch.from_numpy(c.keep)
    q = torch.log_softmax(h @ Wd.t(), 1)[idx, tok.cpu().long()]
    p = torch.log_softmax(hr @ Wd.t(), 1)[idx, tok.cpu().long()]
    A = adv.double().cpu().repeat_interleave(60)
    x = p - q
    ell = -(A * torch.exp(q - q.detach()) - 0.04 * (torch.exp(x) - x - 1))
    total = ell[keep].sum() / keep.sum()
    total.backward()
    assert abs(float(loss) - float(total.detach())) <= 1e-3 * abs(float(total.detach()))
    s = host(sm)
    wx, ww, _, _ = R.norm_grad(s, c.weight(), h.grad.numpy(), EPS)
    # the 8-bit loss's own dH is within 2e-2 of its largest entry; the rest is bf16's
    for got, want in ((host(dx), wx), (host(dw), ww)):
        assert np.linalg.norm(got - want) <= 0.05 * np.linalg.norm(want)


def test_the_bench_runs_the_step_from_the_stream():
    """Both norms, the 8-bit loss and its gradients, and the norm's gradient from the checkpoint, as one command."""
    import json
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "bench.py", "--stream", "--config", "tiny", "--steps", "2", "--warmup", "1"], cwd=root,
                         capture_output=True, text=True, timeout=280)
    assert out.returncode == 0, out.stderr[-2000:]
    line = json.loads(out.stdout.strip().splitlines()[-1])
    assert np.isfinite(line["loss"]) and line["kernel_ms_per_step"]["norm"] > 0 and line["kernel_ms_per_step"]["norm_bwd"] > 0
    assert line["checkpoint_bytes"] * 2 < line["stream_bytes"] * 1.04
