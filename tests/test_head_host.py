"""Host-side checks of the log-prob and off-policy entry points that need no GPU: refusals, workspace sizes, structs."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from rl_fine_tuning_gb300 import build
    build.build()
    import rl_fine_tuning_gb300 as rg
    return rg.load()


def test_head_operator_refusals_without_a_device(lib):
    """The log-prob and off-policy entry points reject bad arguments before any launch."""
    import rl_fine_tuning_gb300 as rg
    P = 1 << 20
    f = ctypes.c_float
    s = rg.make_shape(1, 2, 64, 128, 1024)
    ref = ctypes.byref
    need = {op: rg.grpo_policy_workspace_bytes(s, op) for op in rg.HEAD_OPS}
    assert 0 < need["logp"] < need["logp_grad"] <= need["pair"]
    lp = lambda shape=s, h=P, W=P, tok=P, mask=P, T=1.0, ws=P, n=None, q=P, ent=P, st=P: lib.grpo_logprobs(  # noqa: E731
        h, W, tok, mask, ref(shape) if shape else None, f(T), ws, need["logp"] if n is None else n, q, ent, st, None)
    for kw, code in ((dict(h=None), 1), (dict(W=P + 8), 1), (dict(tok=None), 1), (dict(tok=P + 2), 1), (dict(ws=None), 1),
                     (dict(ws=P + 128), 1), (dict(q=None), 1), (dict(ent=P + 1), 1), (dict(st=None), 1),
                     (dict(n=need["logp"] - 1), 3), (dict(T=0.0), 2), (dict(T=-1.0), 2), (dict(T=float("nan")), 2),
                     (dict(T=float("inf")), 2), (dict(T=1e-45), 2), (dict(shape=None), 2)):
        assert lp(**kw) == code, kw
    for dt in (rg.E4M3, rg.E5M2, 7):
        b = rg.make_shape(1, 2, 64, 128, 1024, dt)
        assert lp(shape=b) == 5 and rg.grpo_policy_workspace_bytes(b, "logp") == 0
    for field, val in (("d", 100), ("V", 0), ("L", 0), ("chunk_rows", -1)):
        b = rg.make_shape(1, 2, 64, 128, 1024)
        setattr(b, field, val)
        assert lp(shape=b) == 2 and rg.grpo_policy_workspace_bytes(b, "clip") == 0, field
    for op in (-1, 4):
        assert rg.grpo_policy_workspace_bytes(s, op) == 0

    bw = lambda mask=P, dq=P, T=1.0, sc=1.0, f32=0, n=need["logp_grad"], dH=P, dW=P, inf=P: lib.grpo_logprobs_bwd(  # noqa: E731
        P, P, P, mask, dq, ref(s), f(T), f(sc), f32, P, n, dH, dW, inf, P, None)
    for kw, code in ((dict(mask=None), 1), (dict(dq=None), 1), (dict(dH=P + 16), 1), (dict(dW=None), 1), (dict(inf=None), 1),
                     (dict(sc=0.0), 2), (dict(sc=float("inf")), 2), (dict(f32=2), 2), (dict(n=need["logp"]), 3)):
        assert bw(**kw) == code, kw

    def clip(shape=s, o=None, adv=P, old=P, pref=P, n=need["clip"], loss=P, stats=P, sc=1.0, **opts):
        o = rg.clip_opts(**opts) if o is None else o
        return lib.grpo_clip_loss_fwd_bwd(P, P, P, P, adv, old, pref, ref(shape), ref(o), f(sc), P, n, loss, P, P, P, stats, P,
                                          None)
    for kw, code in ((dict(adv=None), 1), (dict(old=None), 1), (dict(pref=None), 1), (dict(loss=None), 1),
                     (dict(stats=P + 2), 1), (dict(old=P + 1), 1), (dict(n=need["clip"] - 1), 3),
                     (dict(clip_low=-0.1), 2), (dict(clip_low=1.1), 2), (dict(clip_low=float("nan")), 2),
                     (dict(clip_high=-1.0), 2), (dict(temperature=0.0), 2), (dict(sc=-1.0), 2)):
        assert clip(**kw) == code, kw
    assert lib.grpo_clip_loss_fwd(P, P, P, P, P, P, P, ref(s), None, P, need["clip"], P, None, P, None) == 2
    b = rg.make_shape(1, 2, 64, 128, 1024, objective="forward_kl")
    assert clip(shape=b) == 2
    b = rg.make_shape(1, 2, 64, 128, 1024, beta=float("nan"))
    assert clip(shape=b) == 2

    def pair(shape=s, pref=P, n=need["pair"], loss=P, q=P, stats=P, bwd=True, **opts):
        o = rg.pair_opts(**opts)
        if bwd:
            return lib.grpo_pair_loss_fwd_bwd(P, P, P, P, pref, ref(shape), ref(o), f(1.0), P, n, loss, P, P, P, q, stats, P,
                                              None)
        return lib.grpo_pair_loss_fwd(P, P, P, P, pref, ref(shape), ref(o), P, n, loss, q, stats, P, None)
    for bwd in (True, False):
        for kw, code in ((dict(pref=None), 1), (dict(loss=None), 1), (dict(q=P + 2), 1), (dict(stats=P + 1), 1),
                         (dict(n=need["pair"] - 1), 3), (dict(kind=3), 2), (dict(kind=-1), 2), (dict(label_smoothing=0.5), 2),
                         (dict(label_smoothing=-0.1), 2), (dict(kind="hinge", label_smoothing=0.1), 2)):
            assert pair(bwd=bwd, **kw) == code, kw
        assert pair(shape=rg.make_shape(1, 4, 64, 128, 1024), bwd=bwd) == 2          # pairs: G is 2
        assert pair(shape=rg.make_shape(1, 2, 64, 128, 1024, beta=0.0), bwd=bwd) == 2


def test_head_operator_workspaces(lib):
    """O(chunk (V + d) + N); a preference chunk holds a whole pair up to 19456 rows; a 16-bit dW over several chunks adds
    its fp32 sum."""
    import rl_fine_tuning_gb300 as rg
    V, d = 128256, 4096
    w = rg.grpo_policy_workspace_bytes
    long = rg.make_shape(1, 8, 20000, d, V)
    assert w(long, "clip") - w(long, "clip", True) == 4 * V * d
    R = 9728                                                            # 76 tiles of 128 rows by default
    assert R * V * 2 < w(long, "clip", True) < R * V * 2 * 5 // 4 < 2 * 2 * long.N * V // 25
    small = rg.make_shape(1, 8, 20000, d, V, chunk_rows=1000)           # rounded up to 8 tiles
    assert 1024 * V * 2 < w(small, "clip", True) < 1024 * V * 2 * 2
    assert w(long, "logp") < 1 << 28
    one = rg.make_shape(1, 2, 1000, d, V)
    assert w(one, "clip") == w(one, "clip", True)                       # one chunk: no fp32 sum
    fits, not_ = rg.make_shape(4, 2, 9728, d, V), rg.make_shape(4, 2, 9729, d, V)
    assert w(fits, "pair", True) > 19456 * 2 * V > w(not_, "pair", True)


def test_head_operator_structs_and_binding_refusals(tmp_path, lib):
    import torch

    import rl_fine_tuning_gb300 as rg
    prog = tmp_path / "o.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "grpo.h"\nint main(void){'
                    'printf("%zu %zu %zu %zu %zu %zu %zu", sizeof(grpo_clip_opts), offsetof(grpo_clip_opts,clip_low),'
                    'offsetof(grpo_clip_opts,clip_high), offsetof(grpo_clip_opts,dw_f32), sizeof(grpo_pair_opts),'
                    'offsetof(grpo_pair_opts,label_smoothing), offsetof(grpo_pair_opts,dw_f32));return 0;}\n')
    exe = tmp_path / "o"
    subprocess.check_call(["gcc", "-I" + os.path.join(ROOT, "include"), str(prog), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    C, Q = rg.GrpoClipOpts, rg.GrpoPairOpts
    assert got == [ctypes.sizeof(C), C.clip_low.offset, C.clip_high.offset, C.dw_f32.offset, ctypes.sizeof(Q),
                   Q.label_smoothing.offset, Q.dw_f32.offset]
    o = rg.clip_opts()
    assert (o.temperature, o.dw_f32) == (1.0, 0) and o.clip_low == o.clip_high == pytest.approx(0.2)
    s = rg.make_shape(1, 1, 4, 64, 100)
    h = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):       # a tensor in host memory
        rg.grpo_logprobs(h, h, h, None, s, 1.0, h, h, None, h)
    s8 = rg.make_shape(1, 1, 4, 128, 100, rg.E4M3)
    with pytest.raises(rg.GrpoError):
        rg.grpo_logprobs(h, h, h, None, s8, 1.0, h, h, None, h)
