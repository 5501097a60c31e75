"""Calls of the operators around the state update that are refused, or whose side effects
autograd has to see: host-side checks, and the same on the GPU where a launch is needed."""
import ctypes

import pytest

from kimi_delta_attention_20_b200 import _abi

A, B, C, D_ = (0x1000000 * (k + 1) for k in range(4))  # far apart, never dereferenced


@pytest.mark.parametrize("over", [dict(residual_out=D_), dict(residual_out=A), dict(residual_out=D_, gate=B), dict(residual_out=D_, scales=B)], ids=str)
def test_norm_refuses_a_sum_without_its_residual(over):
    """The sum is written where a residual is added; a call that asks for it without one would
    leave the buffer as it was."""
    a = _abi.RMSNormArgs(dtype=_abi.KDA_DTYPE_BF16, rows=8, D=64, x=A, eps=1e-6, y=C, **over)
    assert _abi.load().kda_rms_norm(ctypes.byref(a), None) == _abi.KDA_ERR_INVALID_ARGUMENT
