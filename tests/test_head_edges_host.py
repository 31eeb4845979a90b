"""Host-side limits of the head operators' arguments, without a GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from rl_fine_tuning_gb300 import build
    build.build()
    import rl_fine_tuning_gb300 as rg
    return rg.load()


@pytest.mark.parametrize("T", [1.01e20, 1e28, 1e30, 3e38, 0.99e-6, 1e-20, 1e-38])
def test_temperatures_that_the_sums_cannot_hold_are_refused(lib, T):
    """Above 1e20 the stand-in for columns that do not count would come near the logits, below 1e-6 ordinary logits
    would be so large that their exponentials' rounding leaves fp16's range."""
    import rl_fine_tuning_gb300 as rg
    P, f, ref = 1 << 20, ctypes.c_float, ctypes.byref
    s = rg.make_shape(1, 2, 64, 128, 1024)
    n = {op: rg.grpo_policy_workspace_bytes(s, op) for op in rg.HEAD_OPS}
    assert lib.grpo_logprobs(P, P, P, P, ref(s), f(T), P, n["logp"], P, None, P, None) == 2
    assert lib.grpo_logprobs_bwd(P, P, P, P, P, ref(s), f(T), f(1.0), 0, P, n["logp_grad"], P, P, P, P, None) == 2
    o = rg.clip_opts(temperature=T)
    assert lib.grpo_clip_loss_fwd(P, P, P, P, P, P, P, ref(s), ref(o), P, n["clip"], P, None, P, None) == 2
    assert lib.grpo_clip_loss_fwd_bwd(P, P, P, P, P, P, P, ref(s), ref(o), f(1.0), P, n["clip"], P, P, P, P, None, P,
                                      None) == 2
    # at the limits the other checks go on (a null pointer is what is wrong here)
    for ok in (1e20, 1e-6):
        assert lib.grpo_logprobs(None, P, P, P, ref(s), f(ok), P, n["logp"], P, None, P, None) == 1
        assert lib.grpo_logprobs_bwd(P, P, P, P, P, ref(s), f(ok), f(1.0), 0, P, n["logp_grad"], None, P, P, P, None) == 1
