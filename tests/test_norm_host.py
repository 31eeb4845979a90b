"""Host-side checks of the norm's and the checkpoints' entry points that need no GPU: refusals, workspace sizes, structs."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20      # an address that every alignment check accepts; no call here gets as far as a launch
OK_SO_FAR = 7, 4  # GRPO_ERR_DEVICE or GRPO_ERR_LAUNCH: all arguments were accepted, there is no device


@pytest.fixture(scope="module")
def lib():
    from rl_fine_tuning_gb300 import build
    build.build()
    import rl_fine_tuning_gb300 as rg
    return rg.load()


def _has_gpu():
    """On a machine with a GPU these addresses must not come to a launch."""
    import torch
    return torch.cuda.is_available()


def shape(**over):
    import rl_fine_tuning_gb300 as rg
    s = rg.make_shape(1, 2, 64, 128, 1)
    for k, v in over.items():
        setattr(s, k, v)
    return s


def ckpt(codes=P, scales=P):
    import rl_fine_tuning_gb300 as rg
    return rg.GrpoCkpt(codes, scales)


def fwd(lib, x=P, xc=None, r=P, w=P, mask=P, s=None, o=None, y=P, rs=None, sum_=P, out=None, **opts):
    import rl_fine_tuning_gb300 as rg
    o = rg.norm_opts(**opts) if o is None else o
    return lib.grpo_norm_fwd(x, xc, r, w, mask, shape() if s is None else s or None, o or None, y, rs, sum_, out, None)


def bwd(lib, dy=P, x=P, xc=None, w=P, ds=P, mask=P, s=None, o=None, ws=P, n=1 << 30, dx=P, dw=P, inf=P, **opts):
    import rl_fine_tuning_gb300 as rg
    o = rg.norm_opts(**opts) if o is None else o
    return lib.grpo_norm_bwd(dy, x, xc, w, ds, mask, shape() if s is None else s or None, o or None, ws, n, dx, dw, inf, None)


def test_norm_forward_refusals(lib):
    import rl_fine_tuning_gb300 as rg
    for kw, code in ((dict(x=None), 1), (dict(x=P + 8), 1), (dict(xc=ckpt()), 1), (dict(x=None, xc=ckpt()), 1),
                     (dict(x=None, xc=ckpt(), r=None, out=ckpt()), 1), (dict(x=None, r=None, xc=ckpt(codes=None)), 1),
                     (dict(x=None, r=None, xc=ckpt(codes=P + 8)), 1), (dict(x=None, r=None, xc=ckpt(scales=P + 1)), 1),
                     (dict(x=None, r=None, xc=ckpt(scales=None)), 1), (dict(r=P + 2), 1), (dict(w=None), 1), (dict(w=P + 8), 1),
                     (dict(x=P + 16), 1), (dict(r=P + 16), 1), (dict(y=P + 16), 1), (dict(sum_=P + 16), 1),
                     (dict(y=P + 8, y_type=rg.E4M3, rs=P), 1), (dict(y=None), 1), (dict(y=P + 8), 1), (dict(sum_=P + 8), 1),
                     (dict(out=ckpt(codes=P + 4)), 1),
                     (dict(out=ckpt(scales=None)), 1), (dict(rs=P), 1), (dict(y_type=rg.E4M3), 1),
                     (dict(y_type=rg.E4M3, rs=P + 2), 1), (dict(y_type=rg.E4M3, y_scale=1.0, rs=P + 1), 1),
                     (dict(s=False), 2), (dict(o=False), 2), (dict(eps=0.0), 2), (dict(eps=1e-39), 2), (dict(eps=-1.0), 2),
                     (dict(eps=float("nan")), 2), (dict(eps=float("inf")), 2), (dict(y_scale=1.0), 2),
                     (dict(y_type=rg.E5M2, y_scale=-1.0, rs=P), 2), (dict(y_type=rg.E5M2, y_scale=1e-39, rs=P), 2),
                     (dict(y_type=rg.E5M2, y_scale=2e38, rs=P), 2), (dict(y_type=rg.E5M2, y_scale=float("nan"), rs=P), 2),
                     (dict(y_type=rg.FP16), 5), (dict(y_type=7), 5), (dict(y_type=-1), 5)):
        assert fwd(lib, **kw) == code, kw
    for field, val, code in (("d", 100, 2), ("d", 16448, 2), ("L", 0, 2), ("chunk_rows", -1, 2),
                             ("dtype", rg.E4M3, 5), ("dtype", 7, 5)):
        s = shape(**{field: val})
        assert fwd(lib, s=s) == code and bwd(lib, s=s) == code, field
        assert rg.grpo_norm_workspace_bytes(s) == 0
    for field in ("weight_f32", "plus_one"):
        for val in (2, -1):
            o = rg.norm_opts()
            setattr(o, field, val)
            assert fwd(lib, o=o) == 2 and bwd(lib, o=o) == 2, field
    # calls that have nothing wrong with them come to the device
    for kw in (dict(), dict(r=None, sum_=None, mask=None), dict(x=None, xc=ckpt(), r=None), dict(out=ckpt(scales=P + 2)),
               dict(y_type=rg.E4M3, rs=P, y=P + 16), dict(w=P + 16), dict(y_type=rg.E5M2, y_scale=2.0 ** -126),
               dict(y_type=rg.E5M2, y_scale=2.0 ** 126),
               dict(y_type=rg.E4M3, y_scale=0.1, rs=P), dict(s=shape(d=16384)), dict(weight_f32=True, plus_one=True)):
        assert _has_gpu() or fwd(lib, **kw) in OK_SO_FAR, kw


def test_norm_gradient_refusals(lib):
    import rl_fine_tuning_gb300 as rg
    need = rg.grpo_norm_workspace_bytes(shape())
    for kw, code in ((dict(dy=None), 1), (dict(dy=P + 16), 1), (dict(x=P + 16), 1), (dict(ds=P + 16), 1),
                     (dict(dx=P + 16), 1), (dict(x=None), 1), (dict(xc=ckpt()), 1), (dict(x=P + 2), 1),
                     (dict(x=None, xc=ckpt(scales=P + 1)), 1), (dict(w=None), 1), (dict(w=P + 4), 1), (dict(ds=P + 8), 1),
                     (dict(ws=None), 1), (dict(ws=P + 128), 1), (dict(dx=None), 1), (dict(dx=P + 8), 1), (dict(dw=P + 8), 1),
                     (dict(inf=None), 1), (dict(inf=P + 2), 1), (dict(n=need - 1), 3), (dict(n=0), 3), (dict(s=False), 2),
                     (dict(o=False), 2), (dict(eps=0.0), 2), (dict(eps=float("nan")), 2)):
        assert bwd(lib, **kw) == code, kw
    for kw in (dict(n=need), dict(ds=None, dw=None, mask=None), dict(x=None, xc=ckpt())):
        assert _has_gpu() or bwd(lib, **kw) in OK_SO_FAR, kw


def test_checkpoint_refusals(lib):
    import rl_fine_tuning_gb300 as rg
    huge = rg.make_shape(1, 1 << 10, (1 << 21) - (1 << 7), 65536, 1)     # 2^47 elements
    assert rg.grpo_workspace_bytes(huge) > 0
    pack = lambda x=P, mask=None, s=shape(), c=ckpt(): lib.grpo_ckpt_pack(x, mask, s, c, None)  # noqa: E731
    unpack = lambda c=ckpt(), mask=None, s=shape(), x=P: lib.grpo_ckpt_unpack(c, mask, s, x, None)  # noqa: E731
    for f in (pack, unpack):
        for kw, code in ((dict(x=None), 1), (dict(x=P + 16), 1), (dict(s=huge), 2), (dict(c=None), 1), (dict(c=ckpt(codes=P + 8)), 1),
                         (dict(c=ckpt(codes=None)), 1), (dict(c=ckpt(scales=None)), 1), (dict(c=ckpt(scales=P + 1)), 1),
                         (dict(s=None), 2), (dict(s=shape(d=96)), 2), (dict(s=shape(G=0)), 2), (dict(s=shape(dtype=rg.E5M2)), 5)):
            assert f(**kw) == code, kw
        assert _has_gpu() or f() in OK_SO_FAR


def test_norm_workspace(lib):
    """4 d for each of a limited number of partial sums, whatever the number of rows."""
    import rl_fine_tuning_gb300 as rg
    w = lambda L, d: rg.grpo_norm_workspace_bytes(rg.make_shape(1, 8, L, d, 1))  # noqa: E731
    assert 456 * 4 * 4096 <= w(20000, 4096) < 456 * 4 * 4096 + 4096 and w(20000, 4096) == w(1000, 4096)
    assert 4 * 64 <= w(1, 64) <= 1024 and all(w(100000, d) <= 12 * 152 * 4 * d + 8192 for d in range(64, 16385, 64))


def test_norm_structs_and_binding_refusals(tmp_path, lib):
    import torch

    import rl_fine_tuning_gb300 as rg
    prog = tmp_path / "o.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "grpo.h"\nint main(void){'
                    'printf("%zu %zu %zu %zu %zu %zu %d %d", sizeof(grpo_norm_opts), offsetof(grpo_norm_opts,plus_one),'
                    'offsetof(grpo_norm_opts,y_type), offsetof(grpo_norm_opts,y_scale), sizeof(grpo_ckpt),'
                    'offsetof(grpo_ckpt,scales), GRPO_CKPT_BLOCK, GRPO_PROF_KINDS);return 0;}\n')
    exe = tmp_path / "o"
    subprocess.check_call(["gcc", "-I" + os.path.join(ROOT, "include"), str(prog), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    O, C = rg.GrpoNormOpts, rg.GrpoCkpt
    assert got == [ctypes.sizeof(O), O.plus_one.offset, O.y_type.offset, O.y_scale.offset, ctypes.sizeof(C), C.scales.offset,
                   rg.CKPT_BLOCK, len(rg.PROF_KINDS)]
    o = rg.norm_opts()
    assert (o.weight_f32, o.plus_one, o.y_type, o.y_scale) == (0, 0, rg.BF16, 0.0) and o.eps == pytest.approx(1e-6)
    if not torch.cuda.is_available():
        return
    # (binding) tensors of another type, size, layout or place; nothing is launched
    s = rg.make_shape(1, 1, 4, 64, 1)
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    for bad in (x.cpu(), x.half(), x[:3], torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")[:, :64], x.t()):
        with pytest.raises(ValueError):
            rg.grpo_norm_fwd(bad, None, w, None, s, o, x)
        with pytest.raises(ValueError):
            rg.grpo_ckpt_unpack((x, w), None, s, bad)


def test_binding_refusals_of_types(lib):
    import torch

    import rl_fine_tuning_gb300 as rg
    s8 = rg.make_shape(1, 1, 4, 128, 100, rg.E4M3)
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    for call in (lambda: rg.grpo_norm_fwd(x, None, x, None, s8, rg.norm_opts(), x),
                 lambda: rg.grpo_norm_bwd(x, x, x, None, None, s8, rg.norm_opts(), x, x, None, x),
                 lambda: rg.grpo_ckpt_pack(x, None, s8, (x, x)), lambda: rg.grpo_ckpt_unpack((x, x), None, s8, x)):
        with pytest.raises(rg.GrpoError):
            call()


def test_plans_fit_an_sm(tmp_path, lib):
    """How rows are dealt to blocks, for every width and a range of row counts: all of a row has a thread, the blocks an SM is
    to have fit its registers and shared memory, and the partial sums fit the workspace."""
    from rl_fine_tuning_gb300 import build
    csrc, cuda = build.CSRC, os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    prog = tmp_path / "p.cpp"
    prog.write_text('''#include <cstdio>
#include "norm.h"
using namespace grpo;
int main() {
    long n = 0, bad = 0;
    for (int d = 64; d <= kNormMaxD; d += 64)
        for (long N : {1L, 2L, 8L, 9L, 16L, 17L, 100L, 1000L, 9727L, 9728L, 1000000L, 2147418112L})
            for (int i = 0; i < 4; ++i) {
                const bool ck = i & 1, ds = i & 2;
                const NormPlan o = norm_bwd_plan(N, d, kSmCount, ck, ds), f = norm_fwd_plan(N, d, kSmCount);
                bool ok = o.width * o.upt * kUnit >= d && o.grid >= 1 && o.grid <= norm_parts(N, d) && o.threads <= kBlockMax;
                ok = ok && norm_parts(N, d) <= 12 * kSmCount && (!o.joined || (o.grid <= 8 && (o.grid & (o.grid - 1)) == 0));
                if (o.wide) {
                    const long weight = long(o.width) * o.upt * kUnit * 4, row = weight / 4 * (2 + (ck ? 1 : 2) + (ds ? 2 : 0));
                    ok = ok && o.threads == o.width && o.width % 32 == 0 && o.threads * (o.upt == 1 ? 80 : 128) * o.per_sm <= 65536;
                    ok = ok && (weight + row + 2048) * o.per_sm <= 226 * 1024;          // one stage of the ring at least
                } else {
                    ok = ok && o.upt == 1 && o.threads == kWarpThreads && o.threads % o.width == 0;
                    ok = ok && o.threads * 96 * o.per_sm <= 65536;
                }
                ok = ok && f.width * f.upt * kUnit >= d && f.grid >= 1 && f.upt <= 2;
                ok = ok && f.per_sm >= 1 && f.threads * (f.upt == 1 ? 64 : 128) * f.per_sm <= 65536;
                const long turns = (N + f.threads / f.width - 1) / (f.threads / f.width);
                ok = ok && f.grid <= turns && (f.grid >= turns || f.grid >= f.per_sm * kSmCount);
                ++n;
                bad += !ok;
            }
    printf("%ld %ld", n, bad);
    return 0;
}
''')
    exe = tmp_path / "p"
    subprocess.check_call(["g++", "-std=c++17", "-I" + os.path.join(ROOT, "include"), "-I" + csrc, "-I" + cuda,
                           "-x", "c++", str(prog), os.path.join(csrc, "norm_plan.cu"), "-o", str(exe)])
    n, bad = (int(x) for x in subprocess.check_output([str(exe)], text=True).split())
    assert n == 256 * 12 * 4 and bad == 0


def test_blocks_of_wide_rows(tmp_path, lib):
    """What the kernels of wide rows ask of a block: whole warps, one at least, as many as their sums in shared memory have
    places for, and elements for every one of the warps."""
    from rl_fine_tuning_gb300 import build
    csrc, cuda = build.CSRC, os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    prog = tmp_path / "p.cpp"
    prog.write_text('''#include <cstdio>
#include "norm.h"
using namespace grpo;
int main() {
    int bad = 0;
    for (int d = 64; d <= kNormMaxD; d += 64)
        for (long N : {1L, 9727L, 9728L, 1000000L})
            for (int i = 0; i < 5; ++i) {
                const NormPlan o = i < 4 ? norm_bwd_plan(N, d, kSmCount, i & 1, i & 2) : norm_fwd_plan(N, d, kSmCount);
                if (!o.wide) continue;
                bad += o.threads != o.width || o.threads % 32 || o.threads < 32 || o.threads > kBlockMax;
                bad += (o.width - 32) * o.upt * kUnit >= d || o.upt < 1 || o.upt > 2;
            }
    printf("%d", bad);
    return 0;
}
''')
    exe = tmp_path / "p"
    subprocess.check_call(["g++", "-std=c++17", "-I" + os.path.join(ROOT, "include"), "-I" + csrc, "-I" + cuda,
                           "-x", "c++", str(prog), os.path.join(csrc, "norm_plan.cu"), "-o", str(exe)])
    assert subprocess.check_output([str(exe)], text=True) == "0"
