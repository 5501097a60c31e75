"""Calls of the operators around the state update that are refused, or whose side effects
autograd has to see: host-side checks, and the same on the GPU where a launch is needed."""
import ctypes

import pytest
import torch

from kimi_delta_attention_20_b200 import _abi

A, B, C, D_ = (0x1000000 * (k + 1) for k in range(4))  # far apart, never dereferenced


@pytest.mark.parametrize("over", [dict(residual_out=D_), dict(residual_out=A), dict(residual_out=D_, gate=B), dict(residual_out=D_, scales=B)], ids=str)
def test_norm_refuses_a_sum_without_its_residual(over):
    """The sum is written where a residual is added; a call that asks for it without one would
    leave the buffer as it was."""
    a = _abi.RMSNormArgs(dtype=_abi.KDA_DTYPE_BF16, rows=8, D=64, x=A, eps=1e-6, y=C, **over)
    assert _abi.load().kda_rms_norm(ctypes.byref(a), None) == _abi.KDA_ERR_INVALID_ARGUMENT


# --------------------------------------------------------------------------- calls that have no gradients

def step_calls(dev):
    """(function, its tensors) of the forms without gradients; None: an argument left out."""
    import kimi_delta_attention_20_b200 as kda
    x, w, win, st = torch.zeros(2, 8, device=dev), torch.zeros(8, 4, device=dev), torch.zeros(2, 8, 4, device=dev), torch.zeros(2, 8, device=dev)
    return [(kda.causal_conv_step, [x, w, win]), (kda.gated_scan_step, [x, x.clone(), st]),
            (lambda a, b, c, d: kda.gated_scan_step(a, b, c, state_out=d), [x, x.clone(), st, st.clone()])]


def test_steps_refuse_to_drop_gradients():
    """Whichever tensor requires grad, and before anything else is looked at."""
    for f, args in step_calls("cpu"):
        for k in range(len(args)):
            leaf = [a.clone().requires_grad_(i == k) for i, a in enumerate(args)]
            with pytest.raises(NotImplementedError):
                f(*leaf)
            with torch.no_grad(), pytest.raises(ValueError):  # on the CPU
                f(*leaf)


@pytest.mark.gpu
def test_steps_of_weights_that_are_trained_run_without_recording():
    for f, args in step_calls("cuda"):
        want = [f(*args), *args]
        leaf = [a.clone().requires_grad_() for a in args]
        with torch.no_grad():
            f(*leaf)
        assert not want[0].requires_grad
