"""Python binding of libgrpo, the fused linear GRPO loss for GB300 (sm_103a).

Argument marshalling only: every function forwards to the C entry point of
the same name in libgrpo.so, whose kernels do all the work.  Tensors are
torch CUDA tensors (only their device pointers are passed); the stream
defaults to torch's current stream.  A nonzero return code raises
GrpoError.  There is no CPU fallback: importing the binding without the
built library raises.
"""
from __future__ import annotations

import ctypes
import os

from . import build as _build

__all__ = [
    "GrpoError", "GrpoShape", "BF16", "FP16", "E4M3", "E5M2", "TOKEN_MEAN", "SEQUENCE_MEAN", "OBJECTIVES", "load",
    "make_shape", "grpo_workspace_bytes", "grpo_chunk_rows", "grpo_group_advantages", "grpo_build_mask",
    "grpo_valid_rows", "grpo_loss_fwd", "grpo_loss_fwd_bwd", "grpo_loss_fwd_fp8", "grpo_loss_fwd_noalloc",
    "grpo_shard_counts", "grpo_loss_fwd_shard", "grpo_loss_fwd_bwd_shard", "grpo_loss_fwd_bwd_fp8",
    "grpo_status_string", "grpo_version", "library_path", "grpo_profile_enable", "grpo_profile_collect",
    "grpo_kernel_launches", "grpo_device_checks", "grpo_selftest_bounds_check", "grpo_selftest_wait_timeout",
    "PROF_KINDS", "GrpoClipOpts", "GrpoPairOpts", "HEAD_OPS", "PAIR_KINDS", "clip_opts", "pair_opts",
    "grpo_policy_workspace_bytes", "grpo_logprobs", "grpo_logprobs_bwd", "grpo_clip_loss_fwd", "grpo_clip_loss_fwd_bwd",
    "grpo_pair_loss_fwd", "grpo_pair_loss_fwd_bwd", "GrpoCkpt", "GrpoNormOpts", "CKPT_BLOCK", "norm_opts",
    "grpo_norm_workspace_bytes", "grpo_norm_fwd", "grpo_norm_bwd", "grpo_ckpt_pack", "grpo_ckpt_unpack",
]

# kernel kinds of the diagnostics interface, in the order of the GRPO_PROF_* enum
PROF_KINDS = ("advantages", "mask", "index", "fwd", "merge", "clear", "gather", "dlogits", "dh", "dw", "f8_prep",
              "norm", "norm_bwd", "ckpt")

BF16, FP16, E4M3, E5M2 = 0, 1, 2, 3
TOKEN_MEAN, SEQUENCE_MEAN = 0, 1
# operators of grpo_policy_workspace_bytes, and kinds of preference loss
HEAD_OPS = {"logp": 0, "logp_grad": 1, "clip": 2, "pair": 3}
PAIR_KINDS = {"sigmoid": 0, "hinge": 1, "square": 2}
CKPT_BLOCK = 64      # columns that share a scale of an 8-bit checkpoint
OBJECTIVES = {"grpo": 0, "no_detach": 1, "reverse_kl_q": 2, "forward_kl": 3}


class GrpoError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        super().__init__(f"libgrpo {what} failed: {code} ({_status_string(code)})")


class GrpoShape(ctypes.Structure):
    """Mirror of grpo_shape in include/grpo.h."""
    _fields_ = [
        ("n_groups", ctypes.c_int), ("G", ctypes.c_int), ("L", ctypes.c_int), ("d", ctypes.c_int),
        ("V", ctypes.c_int), ("dtype", ctypes.c_int), ("beta", ctypes.c_float), ("eps", ctypes.c_float),
        ("std_unbiased", ctypes.c_int), ("chunk_rows", ctypes.c_int), ("loss_mode", ctypes.c_int),
        ("objective", ctypes.c_int),
    ]

    @property
    def N(self) -> int:
        return self.n_groups * self.G * self.L


class GrpoClipOpts(ctypes.Structure):
    """Mirror of grpo_clip_opts in include/grpo.h."""
    _fields_ = [("temperature", ctypes.c_float), ("clip_low", ctypes.c_float), ("clip_high", ctypes.c_float),
                ("dw_f32", ctypes.c_int)]


class GrpoPairOpts(ctypes.Structure):
    """Mirror of grpo_pair_opts in include/grpo.h."""
    _fields_ = [("kind", ctypes.c_int), ("label_smoothing", ctypes.c_float), ("length_mean", ctypes.c_int),
                ("dw_f32", ctypes.c_int)]


class GrpoCkpt(ctypes.Structure):
    """Mirror of grpo_ckpt in include/grpo.h."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class GrpoNormOpts(ctypes.Structure):
    """Mirror of grpo_norm_opts in include/grpo.h."""
    _fields_ = [("eps", ctypes.c_float), ("weight_f32", ctypes.c_int), ("plus_one", ctypes.c_int), ("y_type", ctypes.c_int),
                ("y_scale", ctypes.c_float)]


_lib = None


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = False):
    """The loaded libgrpo.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB
    if build_if_missing:
        path = _build.build()
    if not os.path.exists(path):
        raise ImportError(f"libgrpo.so is not built ({path}); run `python -m rl_fine_tuning_gb300.build`")
    lib = ctypes.CDLL(path)
    _declare(lib)
    _lib = lib
    return lib


def _declare(lib):
    """Argument and result types of every entry point of include/grpo.h."""
    p, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    sp, ck = ctypes.POINTER(GrpoShape), ctypes.POINTER(GrpoCkpt)
    sigs = {
        "grpo_shape_init": ([sp, i32, i32, i32, i32, i32, i32], None),
        "grpo_workspace_bytes": ([sp], sz),
        "grpo_chunk_rows": ([sp], i32),
        "grpo_group_advantages": ([p, i32, i32, f32, i32, p, p], i32),
        "grpo_build_mask": ([p, sp, p, p], i32),
        "grpo_valid_rows": ([p, sp, p, p, p, sz, p], i32),
        "grpo_loss_fwd": ([p, p, p, p, p, p, sp, p, sz, p, p, p, p], i32),
        "grpo_loss_fwd_bwd": ([p, p, p, p, p, p, sp, f32, p, sz, p, p, p, p, p, p, p], i32),
        "grpo_loss_fwd_fp8": ([p, p, p, f32, f32, f32, p, p, p, sp, p, sz, p, p, p, p], i32),
        "grpo_loss_fwd_bwd_fp8": ([p, p, p, f32, f32, f32, p, p, p, sp, p, sz, p, p, p, p, p, p], i32),
        "grpo_loss_fwd_noalloc": ([p, p, p, p, p, p, sp, p, p, p, p], i32),
        "grpo_shard_counts": ([p, sp, p, p], i32),
        "grpo_loss_fwd_shard": ([p, p, p, p, p, p, sp, p, p, sz, p, p, p, p], i32),
        "grpo_loss_fwd_bwd_shard": ([p, p, p, p, p, p, sp, p, f32, p, sz, p, p, p, p, p, p, p], i32),
        "grpo_clip_opts_init": ([ctypes.POINTER(GrpoClipOpts)], None),
        "grpo_pair_opts_init": ([ctypes.POINTER(GrpoPairOpts)], None),
        "grpo_policy_workspace_bytes": ([sp, i32, i32], sz),
        "grpo_logprobs": ([p, p, p, p, sp, f32, p, sz, p, p, p, p], i32),
        "grpo_logprobs_bwd": ([p, p, p, p, p, sp, f32, f32, i32, p, sz, p, p, p, p, p], i32),
        "grpo_clip_loss_fwd": ([p, p, p, p, p, p, p, sp, ctypes.POINTER(GrpoClipOpts), p, sz, p, p, p, p], i32),
        "grpo_clip_loss_fwd_bwd": ([p, p, p, p, p, p, p, sp, ctypes.POINTER(GrpoClipOpts), f32, p, sz, p, p, p, p, p, p,
                                    p], i32),
        "grpo_pair_loss_fwd": ([p, p, p, p, p, sp, ctypes.POINTER(GrpoPairOpts), p, sz, p, p, p, p, p], i32),
        "grpo_pair_loss_fwd_bwd": ([p, p, p, p, p, sp, ctypes.POINTER(GrpoPairOpts), f32, p, sz, p, p, p, p, p, p, p, p],
                                   i32),
        "grpo_norm_opts_init": ([ctypes.POINTER(GrpoNormOpts), i32], None),
        "grpo_norm_workspace_bytes": ([sp], sz),
        "grpo_norm_fwd": ([p, ck, p, p, p, sp, ctypes.POINTER(GrpoNormOpts), p, p, p, ck, p], i32),
        "grpo_norm_bwd": ([p, p, ck, p, p, p, sp, ctypes.POINTER(GrpoNormOpts), p, sz, p, p, p, p], i32),
        "grpo_ckpt_pack": ([p, p, sp, ck, p], i32),
        "grpo_ckpt_unpack": ([ck, p, sp, p, p], i32),
        "grpo_profile_enable": ([i32], i32),
        "grpo_profile_collect": ([ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_longlong), i32], i32),
        "grpo_kernel_launches": ([], ctypes.c_ulonglong),
        "grpo_device_checks": ([], i32),
        "grpo_selftest_bounds_check": ([p, p], i32),
        "grpo_selftest_wait_timeout": ([p, p, p], i32),
        "grpo_status_string": ([i32], ctypes.c_char_p),
        "grpo_version": ([], i32),
    }
    for name, (args, res) in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res


def _status_string(code: int) -> str:
    try:
        return load().grpo_status_string(int(code)).decode()
    except Exception:
        return "?"


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return ctypes.c_void_p(x)
    return ctypes.c_void_p(x.data_ptr())


def _nbytes(x) -> int:
    return x.numel() * x.element_size()


_raw_stream = None   # torch's current stream as a number, without a Stream object (3 us less a call)


def _stream(stream):
    global _raw_stream
    if stream is None:
        if _raw_stream is None:
            import torch
            get, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), torch.cuda.current_device
            _raw_stream = (lambda: get(device())) if get else lambda: torch.cuda.current_stream().cuda_stream
        return ctypes.c_void_p(_raw_stream())
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _check(code: int, what: str):
    if code != 0:
        raise GrpoError(code, what)


def make_shape(n_groups, G, L, d, V, dtype=BF16, beta=0.04, eps=1e-4, std_unbiased=True, chunk_rows=0,
               loss_mode=TOKEN_MEAN, objective=0):
    s = GrpoShape()
    load().grpo_shape_init(ctypes.byref(s), n_groups, G, L, d, V, dtype)
    s.beta, s.eps, s.std_unbiased, s.chunk_rows = beta, eps, int(bool(std_unbiased)), chunk_rows
    s.loss_mode = int(loss_mode)
    s.objective = OBJECTIVES[objective] if isinstance(objective, str) else int(objective)
    return s


def grpo_workspace_bytes(shape: GrpoShape) -> int:
    return int(load().grpo_workspace_bytes(ctypes.byref(shape)))


def grpo_chunk_rows(shape: GrpoShape) -> int:
    return int(load().grpo_chunk_rows(ctypes.byref(shape)))


def grpo_group_advantages(rewards, n_groups, G, eps, std_unbiased, adv_out, stream=None):
    _check(load().grpo_group_advantages(_ptr(rewards), n_groups, G, eps, int(bool(std_unbiased)), _ptr(adv_out),
                                        _stream(stream)), "grpo_group_advantages")


def grpo_build_mask(lengths, shape, mask_out, stream=None):
    _check(load().grpo_build_mask(_ptr(lengths), ctypes.byref(shape), _ptr(mask_out), _stream(stream)),
           "grpo_build_mask")


def grpo_valid_rows(mask, shape, rows_out, n_valid_out, workspace, stream=None):
    _check(load().grpo_valid_rows(_ptr(mask), ctypes.byref(shape), _ptr(rows_out), _ptr(n_valid_out),
                                  _ptr(workspace), _nbytes(workspace), _stream(stream)), "grpo_valid_rows")


def grpo_loss_fwd(h_pol, h_ref, W, tokens, mask, adv, shape, workspace, loss_out, row_stats, status,
                  stream=None):
    _check(load().grpo_loss_fwd(_ptr(h_pol), _ptr(h_ref), _ptr(W), _ptr(tokens), _ptr(mask), _ptr(adv),
                                ctypes.byref(shape), _ptr(workspace), _nbytes(workspace), _ptr(loss_out),
                                _ptr(row_stats), _ptr(status), _stream(stream)), "grpo_loss_fwd")


def grpo_loss_fwd_bwd(h_pol, h_ref, W, tokens, mask, adv, shape, loss_scale, workspace, loss_out, dH, dW,
                      found_inf, row_stats, status, stream=None):
    _check(load().grpo_loss_fwd_bwd(_ptr(h_pol), _ptr(h_ref), _ptr(W), _ptr(tokens), _ptr(mask), _ptr(adv),
                                    ctypes.byref(shape), float(loss_scale), _ptr(workspace), _nbytes(workspace),
                                    _ptr(loss_out), _ptr(dH), _ptr(dW), _ptr(found_inf), _ptr(row_stats),
                                    _ptr(status), _stream(stream)), "grpo_loss_fwd_bwd")


def grpo_shard_counts(mask, shape, counts_out, stream=None):
    _check(load().grpo_shard_counts(_ptr(mask), ctypes.byref(shape), _ptr(counts_out), _stream(stream)),
           "grpo_shard_counts")


def grpo_loss_fwd_shard(h_pol, h_ref, W, tokens, mask, adv, shape, global_counts, workspace, loss_out, row_stats,
                        status, stream=None):
    _check(load().grpo_loss_fwd_shard(_ptr(h_pol), _ptr(h_ref), _ptr(W), _ptr(tokens), _ptr(mask), _ptr(adv),
                                      ctypes.byref(shape), _ptr(global_counts), _ptr(workspace), _nbytes(workspace),
                                      _ptr(loss_out), _ptr(row_stats), _ptr(status), _stream(stream)),
           "grpo_loss_fwd_shard")


def grpo_loss_fwd_bwd_shard(h_pol, h_ref, W, tokens, mask, adv, shape, global_counts, loss_scale, workspace,
                            loss_out, dH, dW, found_inf, row_stats, status, stream=None):
    _check(load().grpo_loss_fwd_bwd_shard(_ptr(h_pol), _ptr(h_ref), _ptr(W), _ptr(tokens), _ptr(mask), _ptr(adv),
                                          ctypes.byref(shape), _ptr(global_counts), float(loss_scale),
                                          _ptr(workspace), _nbytes(workspace), _ptr(loss_out), _ptr(dH), _ptr(dW),
                                          _ptr(found_inf), _ptr(row_stats), _ptr(status), _stream(stream)),
           "grpo_loss_fwd_bwd_shard")


def grpo_status_string(code: int) -> str:
    return _status_string(code)


def grpo_version() -> int:
    return int(load().grpo_version())


def grpo_profile_enable(on: bool = True):
    _check(load().grpo_profile_enable(int(bool(on))), "grpo_profile_enable")


def grpo_profile_collect() -> dict:
    """{kind: (milliseconds, launches)} accumulated since the last collect."""
    n = len(PROF_KINDS)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_longlong * n)()
    _check(load().grpo_profile_collect(ms, cnt, n), "grpo_profile_collect")
    return {k: (float(ms[i]), int(cnt[i])) for i, k in enumerate(PROF_KINDS)}


def grpo_kernel_launches() -> int:
    return int(load().grpo_kernel_launches())


def grpo_loss_fwd_noalloc(h_pol, h_ref, W, tokens, mask, adv, shape, loss_out, row_stats, status, stream=None):
    """grpo_loss_fwd on the library's own fixed scratch array (no workspace argument)."""
    _check(load().grpo_loss_fwd_noalloc(_ptr(h_pol), _ptr(h_ref), _ptr(W), _ptr(tokens), _ptr(mask), _ptr(adv),
                                        ctypes.byref(shape), _ptr(loss_out), _ptr(row_stats), _ptr(status),
                                        _stream(stream)), "grpo_loss_fwd_noalloc")


def grpo_loss_fwd_fp8(h_pol, h_ref, W, scale_h_pol, scale_h_ref, scale_w, tokens, mask, adv, shape, workspace,
                      loss_out, row_stats, status, stream=None):
    _check(load().grpo_loss_fwd_fp8(_ptr(h_pol), _ptr(h_ref), _ptr(W), float(scale_h_pol), float(scale_h_ref),
                                    float(scale_w), _ptr(tokens), _ptr(mask), _ptr(adv), ctypes.byref(shape),
                                    _ptr(workspace), _nbytes(workspace), _ptr(loss_out), _ptr(row_stats),
                                    _ptr(status), _stream(stream)), "grpo_loss_fwd_fp8")


def grpo_loss_fwd_bwd_fp8(h_pol, h_ref, W, scale_h_pol, scale_h_ref, scale_w, tokens, mask, adv, shape, workspace,
                          loss_out, dH, dW, row_stats, status, stream=None):
    _check(load().grpo_loss_fwd_bwd_fp8(_ptr(h_pol), _ptr(h_ref), _ptr(W), float(scale_h_pol), float(scale_h_ref),
                                        float(scale_w), _ptr(tokens), _ptr(mask), _ptr(adv), ctypes.byref(shape),
                                        _ptr(workspace), _nbytes(workspace), _ptr(loss_out), _ptr(dH), _ptr(dW),
                                        _ptr(row_stats), _ptr(status), _stream(stream)), "grpo_loss_fwd_bwd_fp8")


def grpo_device_checks() -> bool:
    """True when the loaded library is the build with device-side index checks."""
    return bool(load().grpo_device_checks())


def grpo_selftest_bounds_check(status, stream=None):
    _check(load().grpo_selftest_bounds_check(_ptr(status), _stream(stream)), "grpo_selftest_bounds_check")


def grpo_selftest_wait_timeout(status, waited_ns, stream=None):
    _check(load().grpo_selftest_wait_timeout(_ptr(status), _ptr(waited_ns), _stream(stream)),
           "grpo_selftest_wait_timeout")


# ---------------------------------------------------------------- log-probs and off-policy losses
# Tensor arguments of these are checked: a tensor has to be a contiguous CUDA
# tensor of the stated type and number of elements (the C interface sees only
# its pointer).  Integers pass as raw pointers, unchecked.

_types_of = None   # type name -> tuple of torch types, set at the first check


def _types():
    global _types_of
    if _types_of is None:
        import torch
        _types_of = {"f32": (torch.float32,), "i32": (torch.int32,), "mask": (torch.uint8, torch.bool),
                     BF16: (torch.bfloat16,), FP16: (torch.float16,)}
    return _types_of


def _arg(x, name, types, numel):
    if x is None or isinstance(x, int):
        return x
    if x.dtype in types and x.numel() == numel and x.is_cuda and x.is_contiguous():
        return x.data_ptr()
    raise ValueError(f"{name}: a contiguous CUDA tensor of {numel} elements of type {' or '.join(map(str, types))} is "
                     f"wanted, not {x.dtype}, shape {tuple(x.shape)}, strides {x.stride()}, on {x.device}")


def _inputs(h, W, tokens, mask, shape):
    """(the four pointers), rows, type tables"""
    ty = _types()
    t = ty.get(shape.dtype)
    if t is None:
        raise GrpoError(5, "dtype check")
    N, d = shape.N, shape.d
    return (_arg(h, "h", t, N * d), _arg(W, "W", t, shape.V * d), _arg(tokens, "tokens", ty["i32"], N),
            _arg(mask, "mask", ty["mask"], N)), N, ty


def _grads(dH, dW, found_inf, shape, dw_f32, ty):
    t, d = ty[shape.dtype], shape.d
    return (_arg(dH, "dH", t, shape.N * d), _arg(dW, "dW", ty["f32"] if dw_f32 else t, shape.V * d),
            _arg(found_inf, "found_inf", ty["i32"], 1))


def _workspace(ws):
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("workspace: a contiguous CUDA tensor is wanted")
    return _ptr(ws), _nbytes(ws)


def clip_opts(temperature=1.0, clip_low=0.2, clip_high=0.2, dw_f32=False) -> GrpoClipOpts:
    o = GrpoClipOpts()
    load().grpo_clip_opts_init(ctypes.byref(o))
    o.temperature, o.clip_low, o.clip_high, o.dw_f32 = temperature, clip_low, clip_high, int(bool(dw_f32))
    return o


def pair_opts(kind="sigmoid", label_smoothing=0.0, length_mean=False, dw_f32=False) -> GrpoPairOpts:
    o = GrpoPairOpts()
    load().grpo_pair_opts_init(ctypes.byref(o))
    o.kind = PAIR_KINDS[kind] if isinstance(kind, str) else int(kind)
    o.label_smoothing, o.length_mean, o.dw_f32 = label_smoothing, int(bool(length_mean)), int(bool(dw_f32))
    return o


def grpo_policy_workspace_bytes(shape: GrpoShape, op, dw_f32=False) -> int:
    """Workspace of an operator: "logp", "logp_grad", "clip" or "pair" (or its GRPO_OP_* number)."""
    code = HEAD_OPS[op] if isinstance(op, str) else int(op)
    return int(load().grpo_policy_workspace_bytes(ctypes.byref(shape), code, int(bool(dw_f32))))


def grpo_logprobs(h, W, tokens, mask, shape, temperature, workspace, logp_out, entropy_out, status, stream=None):
    """q (and the entropy, unless None) of every row's token; mask None counts every row."""
    x, N, ty = _inputs(h, W, tokens, mask, shape)
    f, i = ty["f32"], ty["i32"]
    _check(load().grpo_logprobs(*x, ctypes.byref(shape), temperature, *_workspace(workspace),
                                _arg(logp_out, "logp_out", f, N), _arg(entropy_out, "entropy_out", f, N),
                                _arg(status, "status", i, 1), _stream(stream)), "grpo_logprobs")


def grpo_logprobs_bwd(h, W, tokens, mask, dlogp, shape, temperature, loss_scale, workspace, dH, dW, found_inf, status,
                      dw_f32=False, stream=None):
    """Gradients of sum dlogp q."""
    x, N, ty = _inputs(h, W, tokens, mask, shape)
    g = _grads(dH, dW, found_inf, shape, dw_f32, ty)
    _check(load().grpo_logprobs_bwd(*x, _arg(dlogp, "dlogp", ty["f32"], N), ctypes.byref(shape), temperature, loss_scale,
                                    int(bool(dw_f32)), *_workspace(workspace), *g, _arg(status, "status", ty["i32"], 1),
                                    _stream(stream)), "grpo_logprobs_bwd")


def _clip_args(h, W, tokens, mask, adv, logp_old, logp_ref, shape):
    x, N, ty = _inputs(h, W, tokens, mask, shape)
    f = ty["f32"]
    return (*x, _arg(adv, "adv", f, shape.n_groups * shape.G), _arg(logp_old, "logp_old", f, N),
            _arg(logp_ref, "logp_ref", f, N), ctypes.byref(shape)), N, ty


def grpo_clip_loss_fwd(h, W, tokens, mask, adv, logp_old, logp_ref, shape, opts, workspace, loss_out, row_stats, status,
                       stream=None):
    x, N, ty = _clip_args(h, W, tokens, mask, adv, logp_old, logp_ref, shape)
    f, i = ty["f32"], ty["i32"]
    _check(load().grpo_clip_loss_fwd(*x, ctypes.byref(opts), *_workspace(workspace), _arg(loss_out, "loss_out", f, 1),
                                     _arg(row_stats, "row_stats", f, 3 * N), _arg(status, "status", i, 1),
                                     _stream(stream)), "grpo_clip_loss_fwd")


def grpo_clip_loss_fwd_bwd(h, W, tokens, mask, adv, logp_old, logp_ref, shape, opts, loss_scale, workspace, loss_out, dH,
                           dW, found_inf, row_stats, status, stream=None):
    x, N, ty = _clip_args(h, W, tokens, mask, adv, logp_old, logp_ref, shape)
    f, i = ty["f32"], ty["i32"]
    g = _grads(dH, dW, found_inf, shape, opts.dw_f32, ty)
    _check(load().grpo_clip_loss_fwd_bwd(*x, ctypes.byref(opts), loss_scale, *_workspace(workspace),
                                         _arg(loss_out, "loss_out", f, 1), *g, _arg(row_stats, "row_stats", f, 3 * N),
                                         _arg(status, "status", i, 1), _stream(stream)), "grpo_clip_loss_fwd_bwd")


def _pair_args(h, W, tokens, mask, logp_ref, shape):
    x, N, ty = _inputs(h, W, tokens, mask, shape)
    return (*x, _arg(logp_ref, "logp_ref", ty["f32"], N), ctypes.byref(shape)), N, ty


def grpo_pair_loss_fwd(h, W, tokens, mask, logp_ref, shape, opts, workspace, loss_out, logp_out, pair_stats, status,
                       stream=None):
    x, N, ty = _pair_args(h, W, tokens, mask, logp_ref, shape)
    f, i = ty["f32"], ty["i32"]
    _check(load().grpo_pair_loss_fwd(*x, ctypes.byref(opts), *_workspace(workspace), _arg(loss_out, "loss_out", f, 1),
                                     _arg(logp_out, "logp_out", f, N), _arg(pair_stats, "pair_stats", f, 4 * shape.n_groups),
                                     _arg(status, "status", i, 1), _stream(stream)), "grpo_pair_loss_fwd")


def grpo_pair_loss_fwd_bwd(h, W, tokens, mask, logp_ref, shape, opts, loss_scale, workspace, loss_out, dH, dW, found_inf,
                           logp_out, pair_stats, status, stream=None):
    x, N, ty = _pair_args(h, W, tokens, mask, logp_ref, shape)
    f, i = ty["f32"], ty["i32"]
    g = _grads(dH, dW, found_inf, shape, opts.dw_f32, ty)
    _check(load().grpo_pair_loss_fwd_bwd(*x, ctypes.byref(opts), loss_scale, *_workspace(workspace),
                                         _arg(loss_out, "loss_out", f, 1), *g, _arg(logp_out, "logp_out", f, N),
                                         _arg(pair_stats, "pair_stats", f, 4 * shape.n_groups),
                                         _arg(status, "status", i, 1), _stream(stream)), "grpo_pair_loss_fwd_bwd")


# ---------------------------------------------------------------- the norm before the head, 8-bit checkpoints
# A checkpoint is a pair (codes, scales): int8 of N d elements, bfloat16 of N d / CKPT_BLOCK.  Tensors are checked as above,
# and have to be on torch's current device.  None stands for what the C interface takes as NULL.

_norm_types = None   # type name -> tuple of torch types
_device = None       # torch's current device as a number
_stream_of = None    # a device's current stream as a number


def _norm_setup():
    global _norm_types, _device, _stream_of
    import torch
    _norm_types = {**_types(), "codes": (torch.int8,), "scales": (torch.bfloat16,),
                   E4M3: (torch.float8_e4m3fn, torch.uint8), E5M2: (torch.float8_e5m2, torch.uint8)}
    _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _stream_of = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
                  or (lambda device: torch.cuda.current_stream(device).cuda_stream))


def _norm_table(shape):
    """(type tables, the 16-bit type, the current device's number, rows, columns)"""
    if _norm_types is None:
        _norm_setup()
    dtype = shape.dtype
    if dtype != BF16 and dtype != FP16:
        raise GrpoError(5, "dtype check")
    return _norm_types, _norm_types[dtype], _device(), shape.n_groups * shape.G * shape.L, shape.d


def _here(x, name, types, numel, device):
    """As _arg, on the current device (a tensor in host memory has the number -1)."""
    if x is None or type(x) is int:
        return x
    if x.dtype in types and x.numel() == numel and x.get_device() == device and x.is_contiguous():
        return x.data_ptr()
    raise ValueError(f"{name}: a contiguous tensor of {numel} elements of type {' or '.join(map(str, types))} on the current "
                     f"CUDA device is wanted, not {x.dtype}, shape {tuple(x.shape)}, strides {x.stride()}, on {x.device}")


def _ckpt(pair, name, n, ty, device):
    codes, scales = pair
    return GrpoCkpt(_here(codes, name + " codes", ty["codes"], n, device),
                    _here(scales, name + " scales", ty["scales"], n // CKPT_BLOCK, device))


def _source(src, n, ty, t, device):
    """(x, x_ckpt) of a 16-bit matrix or a checkpoint"""
    if isinstance(src, tuple):
        return None, _ckpt(src, "checkpoint", n, ty, device)
    return _here(src, "x", t, n, device), None


def norm_opts(eps=1e-6, weight_f32=False, plus_one=False, y_type=BF16, y_scale=0.0) -> GrpoNormOpts:
    o = GrpoNormOpts()
    load().grpo_norm_opts_init(ctypes.byref(o), int(y_type))
    o.eps, o.weight_f32, o.plus_one, o.y_scale = eps, int(bool(weight_f32)), int(bool(plus_one)), y_scale
    return o


def grpo_norm_workspace_bytes(shape: GrpoShape) -> int:
    return int(load().grpo_norm_workspace_bytes(ctypes.byref(shape)))


def _on(stream, device):
    return _stream_of(device) if stream is None else stream if isinstance(stream, int) else stream.cuda_stream


def grpo_norm_fwd(x, residual, weight, mask, shape, opts, y, row_scale=None, sum_out=None, sum_ckpt=None, stream=None):
    """y (16 or 8 bits, as opts.y_type says) of s = x + residual; x may be a checkpoint (codes, scales)."""
    ty, t, dev, N, d = _norm_table(shape)
    n, f, y_type = N * d, ty["f32"], opts.y_type
    px, pc = _source(x, n, ty, t, dev)
    yt = t if y_type == shape.dtype else ty[y_type] if y_type in (E4M3, E5M2) else None
    if yt is None:
        raise GrpoError(5, "y_type check")
    _check(load().grpo_norm_fwd(px, pc, _here(residual, "residual", t, n, dev),
                                _here(weight, "weight", f if opts.weight_f32 else t, d, dev),
                                _here(mask, "mask", ty["mask"], N, dev), shape, opts, _here(y, "y", yt, n, dev),
                                _here(row_scale, "row_scale", f, N, dev), _here(sum_out, "sum_out", t, n, dev),
                                None if sum_ckpt is None else _ckpt(sum_ckpt, "sum_ckpt", n, ty, dev), _on(stream, dev)),
           "grpo_norm_fwd")


def grpo_norm_bwd(dy, x, weight, dsum, mask, shape, opts, workspace, dx, dweight, found_inf, stream=None):
    """dx and dweight (None: frozen) at s = x, a 16-bit matrix or a checkpoint (codes, scales).  found_inf: 1 if they are not
    all finite, 2 if a wait on the device ran out of time and they are no gradients, else 0."""
    ty, t, dev, N, d = _norm_table(shape)
    n, wt = N * d, ty["f32"] if opts.weight_f32 else t
    px, pc = _source(x, n, ty, t, dev)
    size = workspace.numel()
    _check(load().grpo_norm_bwd(_here(dy, "dy", t, n, dev), px, pc, _here(weight, "weight", wt, d, dev),
                                _here(dsum, "dsum", t, n, dev), _here(mask, "mask", ty["mask"], N, dev), shape, opts,
                                _here(workspace, "workspace", (workspace.dtype,), size, dev), size * workspace.element_size(),
                                _here(dx, "dx", t, n, dev), _here(dweight, "dweight", wt, d, dev),
                                _here(found_inf, "found_inf", ty["i32"], 1, dev), _on(stream, dev)), "grpo_norm_bwd")


def grpo_ckpt_pack(x, mask, shape, ckpt, stream=None):
    """A checkpoint (codes, scales) of x."""
    ty, t, dev, N, d = _norm_table(shape)
    n = N * d
    _check(load().grpo_ckpt_pack(_here(x, "x", t, n, dev), _here(mask, "mask", ty["mask"], N, dev), shape,
                                 _ckpt(ckpt, "ckpt", n, ty, dev), _on(stream, dev)), "grpo_ckpt_pack")


def grpo_ckpt_unpack(ckpt, mask, shape, x_out, stream=None):
    """A checkpoint's values in 16 bits."""
    ty, t, dev, N, d = _norm_table(shape)
    n = N * d
    _check(load().grpo_ckpt_unpack(_ckpt(ckpt, "ckpt", n, ty, dev), _here(mask, "mask", ty["mask"], N, dev), shape,
                                   _here(x_out, "x_out", t, n, dev), _on(stream, dev)), "grpo_ckpt_unpack")
