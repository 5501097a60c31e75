"""Calls of the operators around the state update that are refused, or whose side effects
autograd has to see: host-side checks, and the same on the GPU where a launch is needed."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from kimi_delta_attention_20_b200 import _abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

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


def tangent_calls(dev):
    """Every function with the tensors that it reads."""
    import kimi_delta_attention_20_b200 as kda

    def z(*shape):
        return torch.zeros(shape, device=dev)

    H, D, K = 1, 32, 4
    C = 3 * H * D
    x, w, cw, win, st, S, beta = z(2, 6, C), z(C), z(C, K), z(2, C, K), z(2, C), z(2, H, D, D), z(2, 6, H)
    q, t = z(2, 6, H, D), z(2, H, D)
    return [
        (lambda a, b, c: kda.rms_norm(a, b, residual=c), [x, w, x]), (lambda a, b, c: kda.rms_norm(a, b, gate=c), [x, w, x]),
        (lambda a, b, c: kda.rms_norm_quant(a, b, residual=c), [x, w, x]), (lambda a, b, c, d: kda.rms_norm_bwd(a, b, c, gate=d), [x, x, w, x]),
        (lambda a, b, c: kda.rms_norm_bwd(a, b, dresidual=c), [x, x, x]),
        (lambda a, b, c: kda.causal_conv(a, b, initial_state=c), [x, cw, win]), (kda.causal_conv_step, [x[:, 0], cw, win]),
        (lambda a, b, c, d, e: kda.causal_conv_bwd(a, b, c, initial_state=d, dfinal_state=e), [x, cw, x, win, win]),
        (lambda a, b, c: kda.chunk_gated_scan(a, b, initial_state=c), [x, x, st]), (kda.gated_scan_step, [x[:, 0], x[:, 0], st]),
        (lambda a, b, c, d, e: kda.chunk_gated_scan_bwd(None, a, b, c, initial_state=d, dfinal_state=e), [x, x, x, st, st]),
        (lambda a, b, c, d, e, f: kda.chunk_kda(a, b, c, d, e, initial_state=f, use_qk_l2norm_in_kernel=True), [q, q, q, q, beta, S]),
        (kda.recurrent_step, [t, t, t, t, beta[:, 0], S]), (kda.decode_token, [x[:, 0].contiguous(), cw, win, t, beta[:, 0].contiguous(), S]),
        (lambda a, b, c, d, e, f, g: kda.chunk_kda_bwd(a, b, c, d, e, f, dfinal_state=g), [q, q, q, q, beta, q, S]),
    ]


def test_forward_mode_derivatives_are_refused():
    """A tangent on any input, which the outputs could not carry on; within a dual level, calls
    without tangents are what they were."""
    from torch.autograd import forward_ad
    with forward_ad.dual_level():
        for i, (f, args) in enumerate(tangent_calls("cpu")):
            for k in range(len(args)):
                dual = [forward_ad.make_dual(a, torch.ones_like(a)) if j == k else a for j, a in enumerate(args)]
                with pytest.raises(NotImplementedError):
                    f(*dual)
                    print("not refused:", i, k)
            with pytest.raises(ValueError):  # on the CPU
                f(*args)


# --------------------------------------------------------------------------- tensors that calls write

@pytest.mark.gpu
def test_written_tensors_count_as_changed():
    """Each call raises the version of what it writes of the caller's, and of nothing else."""
    import kimi_delta_attention_20_b200 as kda
    H, D, K = 1, 32, 4
    C = 3 * H * D

    def z(*shape, dtype=torch.float32):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    x, w, g = z(2, 6, C), z(C, K), z(2, 6, C)
    rows, q, k = z(2, C), z(2, H, D), z(1, 6, H, D)
    beta, kbeta = z(2, H), z(1, 6, H)
    calls = [  # function of the written tensors, those by name, and the tensors that are only read
        (lambda out: kda.rms_norm(x, out=out), dict(out=z(2, 6, C)), [x]),
        (lambda residual_out: kda.rms_norm(x, residual=g, residual_out=residual_out), dict(residual_out=z(2, 6, C)), [x, g]),
        (lambda out, scales_out: kda.rms_norm_quant(x, out=out, scales_out=scales_out),
         dict(out=z(2, 6, C, dtype=torch.float8_e4m3fn), scales_out=z(2, 6, 1)), [x]),
        (lambda out, final_state_out: kda.causal_conv(x, w, out=out, final_state_out=final_state_out, output_final_state=True),
         dict(out=z(2, 6, C), final_state_out=z(2, C, K)), [x, w]),
        (lambda conv_state, out: kda.causal_conv_step(rows, w, conv_state, out=out), dict(conv_state=z(2, C, K), out=z(2, C)), [rows, w]),
        (lambda out, final_state_out: kda.chunk_gated_scan(x, g, out=out, final_state_out=final_state_out, output_final_state=True),
         dict(out=z(2, 6, C), final_state_out=z(2, C)), [x, g]),
        (lambda state, out: kda.gated_scan_step(rows, rows, state, out=out), dict(state=z(2, C), out=z(2, C)), [rows]),
        (lambda state_out, s=z(2, C): kda.gated_scan_step(rows, rows, s, state_out=state_out), dict(state_out=z(2, C)), [rows]),
        (lambda conv_state, state, out: kda.decode_token(rows, w, conv_state, q, beta, state, out=out),
         dict(conv_state=z(2, C, K), state=z(2, H, D, D), out=z(2, H, D)), [rows, w, q, beta]),
        (lambda state, out: kda.recurrent_step(q, q, q, q, beta, state, out=out), dict(state=z(2, H, D, D), out=z(2, H, D)), [q, beta]),
        (lambda state_out, s=z(2, H, D, D): kda.recurrent_step(q, q, q, q, beta, s, state_out=state_out), dict(state_out=z(2, H, D, D)), [q]),
        (lambda out, final_state_out: kda.chunk_kda(k, k, k, k, kbeta, use_qk_l2norm_in_kernel=True, output_final_state=True, out=out,
                                                    final_state_out=final_state_out), dict(out=z(1, 6, H, D), final_state_out=z(1, H, D, D)), [k, kbeta]),
    ]
    for i, (f, written, read) in enumerate(calls):
        before, same = {n: t._version for n, t in written.items()}, [t._version for t in read]
        f(**written)
        assert all(t._version > before[n] for n, t in written.items()), i
        assert [t._version for t in read] == same, i
    state = z(2, C)
    s = torch.zeros_like(state)
    v = state._version
    kda.gated_scan_step(rows, rows, state, state_out=s)
    assert state._version == v  # only read
    with torch.inference_mode():  # tensors that have no version
        st = z(2, C)
        kda.gated_scan_step(z(2, C), z(2, C), st, out=z(2, C))
    kda.gated_scan_step(rows, rows, st)


@pytest.mark.gpu
def test_backward_notices_states_that_went_on():
    """A window, state or term that a backward pass needs and a later call overwrites."""
    import kimi_delta_attention_20_b200 as kda
    H, D, K = 1, 32, 4
    C = 3 * H * D

    def rnd(*shape):
        return torch.randn(*shape, generator=torch.Generator().manual_seed(sum(shape))).cuda()

    x, w, g = rnd(2, 6, C).requires_grad_(), rnd(C, K), -rnd(2, 6, C).abs()
    row, q, beta = rnd(2, C), rnd(2, H, D), rnd(2, H)
    win, st, S, term = rnd(2, C, K), rnd(2, C), rnd(2, H, D, D), rnd(2, 6, C)
    pairs = [
        (lambda: kda.causal_conv(x, w, initial_state=win)[0], lambda: kda.causal_conv_step(row, w, win)),
        (lambda: kda.causal_conv(x, w, initial_state=win)[0], lambda: kda.decode_token(row, w, win, -q.abs(), beta, S.clone())),
        (lambda: kda.chunk_gated_scan(x, g, initial_state=st)[0], lambda: kda.gated_scan_step(row, row, st)),
        (lambda: kda.chunk_gated_scan(x, g, initial_state=st)[0], lambda: kda.gated_scan_step(row, row, st.clone(), state_out=st)),
        (lambda: x * term, lambda: kda.rms_norm(g, residual=term, residual_out=term)),
        (lambda: x * term, lambda: kda.causal_conv(g, w, out=term)),
    ]
    for i, (forward, step) in enumerate(pairs):
        forward().sum().backward()  # nothing in between
        y = forward()
        step()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()


# --------------------------------------------------------------------------- import

def test_import_on_a_torch_without_cuda():
    """The binding loads where PyTorch was built without CUDA, and its functions then refuse
    their tensors by name."""
    code = ("import torch\n"
            "for n in [n for n in dir(torch._C) if n.startswith('_cuda_')]: delattr(torch._C, n)\n"
            "import kimi_delta_attention_20_b200 as kda\n"
            "try: kda.rms_norm(torch.zeros(2, 8))\n"
            "except ValueError as e: print('refused:', e)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "refused: x must be a CUDA tensor", r.stderr
