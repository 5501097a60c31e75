"""Python entry points of the operators around the state update of a layer: `rms_norm`,
`causal_conv` and `chunk_gated_scan`, with their backward and single-token forms.

As in `ops`, PyTorch supplies device memory and the current stream, and every step of the
computation runs in the library's CUDA kernels. Activations may be slices of a fused
projection: their channels have to be contiguous and their rows evenly spaced. Outputs are
contiguous. Each function returns its gradients' counterpart through autograd where an input
requires grad (the 8-bit norm and the single-token forms have none); forward-mode derivatives are
refused. Tensors of the caller's that a call writes count as changed in place, so a backward pass
that has saved one notices.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _abi
from .ops import _DTYPES, _no_tangents, _seqlens, _written

_F32 = _abi.KDA_DTYPE_F32
# of a device; what torch.cuda.current_stream wraps (a torch without CUDA has none, and no tensors to launch on)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _dev(name, t):
    """Device index of a CUDA tensor."""
    dev = t.get_device() if isinstance(t, torch.Tensor) else -1
    if dev < 0 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _same_dev(name, t, dev):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}")


def _dtype(name, t):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32 or bfloat16")
    return code


def _row_stride(t: torch.Tensor):
    """Distance between the rows (all but the last dimension) of ``t`` in elements, 0 where
    they are dense; None where the rows are not evenly spaced or their channels are apart."""
    if t.is_contiguous():
        return 0
    shape, stride = t.shape, t.stride()
    if shape[-1] > 1 and stride[-1] != 1:
        return None
    step = None  # of the rows collapsed so far
    rows = 1
    for n, s in zip(reversed(shape[:-1]), reversed(stride[:-1])):
        if n == 1:
            continue
        if step is None:
            step = s
        elif s != step * rows:
            return None
        rows *= n
    if step is None:
        return 0
    return step if step >= shape[-1] else None


def _act(name, t, like, dev):
    """(pointer, row stride) of an activation with the dtype, shape and device of ``like``."""
    if t is not like:
        _same_dev(name, t, dev)
        if t.dtype != like.dtype:
            raise ValueError(f"{name} must have dtype {like.dtype}")
        if t.shape != like.shape:
            raise ValueError(f"{name} must have shape {tuple(like.shape)}")
    stride = 0 if t.is_contiguous() else _row_stride(t)
    if stride is None:
        raise ValueError(f"{name} must have contiguous channels and evenly spaced rows")
    return t.data_ptr(), stride


def _cotangent(name, t, like, dev):
    """A cotangent as autograd hands it over: any strides, brought to dense rows if need be."""
    _same_dev(name, t, dev)
    if t.dtype != like.dtype:
        t = t.to(like.dtype)
    return t if _row_stride(t) is not None else t.contiguous()


def _state(name, t, shape, dev):
    """Pointer of a dense fp32 tensor, 0 for none."""
    if t is None:
        return 0
    _same_dev(name, t, dev)
    if t.dtype != torch.float32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {tuple(shape)}")
    return t.data_ptr()


def _out(name, t, like, dev):
    """The output buffer of activations: the caller's, checked, or a new one."""
    if t is None:
        return torch.empty_like(like) if like.is_contiguous() else torch.empty(like.shape, dtype=like.dtype, device=like.device)
    return _out_as(name, t, like.shape, like.dtype, like.device, dev)


def _out_as(name, t, shape, dtype, device, dev):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _same_dev(name, t, dev)
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    return t


def _ptr(t: Optional[torch.Tensor]):
    return 0 if t is None else t.data_ptr()


def _launch(call, packed, dev):
    """Queues a call on the current stream of its device."""
    if dev == torch.cuda.current_device():
        status = call.fn(packed, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = call.fn(packed, _raw_stream(dev))
    if status:
        _abi.check(status, call.name)


def _launch_scratch(call, fields, workspace, device, dev):
    """As _launch of the packed ``fields``, followed by the workspace that the call needs: the
    caller's, or a new one."""
    need = call.size(call.pack(*fields, 0, 0))
    if workspace is not None:
        _same_dev("workspace", workspace, dev)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        need = workspace.numel() * workspace.element_size()
    elif need:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    _launch(call, call.pack(*fields, _ptr(workspace), need), dev)


def _span(x, cu_seqlens, cu_seqlens_cpu, features):
    """(B, T, N, device offsets, host offsets) of [B, T, channels] activations."""
    if x.dim() != 3:
        raise ValueError(f"x must be [B, T, {features}]")
    B, T = x.shape[:2]
    if cu_seqlens is None:
        if cu_seqlens_cpu is not None:
            raise ValueError("cu_seqlens_cpu needs cu_seqlens")
        return B, T, B, None, None
    if B != 1:
        raise ValueError("cu_seqlens requires B == 1")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must hold N + 1 offsets")
    if cu_seqlens.is_cuda and cu_seqlens_cpu is None:
        if cu_seqlens.device != x.device:
            raise ValueError(f"cu_seqlens must be on {x.device}")
        dev, host = cu_seqlens.to(torch.int32).contiguous(), None
    else:
        dev, host = _seqlens(cu_seqlens, cu_seqlens_cpu, x.device)
    return B, T, cu_seqlens.numel() - 1, dev, host


def _wanted(want_final, final_state_out):
    if final_state_out is not None and not want_final:
        raise ValueError("final_state_out needs output_final_state")


def _recorded(*tensors):
    """Whether autograd records what is computed of the tensors (None: of none)."""
    if forward_ad._current_level >= 0:
        _no_tangents(*tensors)
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    return False


def _no_outs(**outs):
    for name, t in outs.items():
        if t is not None:
            raise ValueError(f"{name} cannot be used when gradients are recorded")


# --------------------------------------------------------------------------- RMS norm

def _weight(weight, x, dev):
    """(pointer, dtype code) of a norm weight."""
    if weight is None:
        return 0, _F32
    _same_dev("weight", weight, dev)
    if weight.shape != x.shape[-1:] or weight.dtype not in (torch.float32, x.dtype) or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous tensor of {x.shape[-1]} float32 or {x.dtype} values")
    return weight.data_ptr(), _DTYPES[weight.dtype]


def _norm_rows(tensors, like, dev):
    """(heads, [(pointer, stride) of each tensor or (0, 0)]): rows evenly spaced, or [.., heads, D]
    whose heads lie back to back and whose tokens are evenly spaced -- a slice of a fused projection."""
    rows, even = [], True
    for name, t in tensors:
        if t is None:
            rows.append((0, 0))
            continue
        if t is not like:
            _same_dev(name, t, dev)
            if t.dtype != like.dtype:
                raise ValueError(f"{name} must have dtype {like.dtype}")
            if t.shape != like.shape:
                raise ValueError(f"{name} must have shape {tuple(like.shape)}")
        stride = 0 if t.is_contiguous() else _row_stride(t)
        even = even and stride is not None
        rows.append((t.data_ptr(), stride))
    if even:
        return 1, rows
    H, D = like.shape[-2:] if like.dim() > 1 else (1, like.shape[-1])
    for i, (name, t) in enumerate(tensors):
        if t is None:
            continue
        dense = (D == 1 or t.stride(-1) == 1) and (H == 1 or t.stride(-2) == D)
        stride = _row_stride(t.flatten(-2)) if t.dim() > 1 and dense else None
        if stride is None:
            raise ValueError(f"{name} must have contiguous channels and evenly spaced rows (or heads back to back in evenly spaced tokens)")
        rows[i] = (t.data_ptr(), stride)
    return H, rows


def _norm(x, weight, residual, gate, eps, residual_out, quant=None, out=None):
    """One forward call; quant: (group_size, pow2_scales, scales_out) for the 8-bit output.
    Returns (y, scales or None, s or None)."""
    call = _abi.call("kda_rms_norm")
    dev = _dev("x", x)
    dt = _dtype("x", x)
    if x.dim() < 1:
        raise ValueError("x must be [..., D]")
    given = [t for t in (out, residual_out, None if quant is None else quant[2]) if t is not None]
    D = x.shape[-1]
    wp, wdt = _weight(weight, x, dev)
    heads, ((xp, xs), (rp, rs), (gp, gs)) = _norm_rows((("x", x), ("residual", residual), ("gate", gate)), x, dev)
    if residual is not None:
        if gate is not None:
            raise ValueError("residual and gate cannot be combined")
        residual_out = _out("residual_out", residual_out, x, dev)
    elif residual_out is not None:
        raise ValueError("residual_out needs residual")
    group = pow2 = 0
    scales = None
    if quant is None:
        y = _out("out", out, x, dev)
    else:
        group, pow2, scales = quant
        if group not in (0, 32, 64, 128):
            raise ValueError("group_size must be 0 (the whole row), 32, 64 or 128")
        if out is None and x.is_contiguous():
            y = torch.empty_like(x, dtype=torch.float8_e4m3fn)
        else:
            y = _out_as("out", out, x.shape, torch.float8_e4m3fn, x.device, dev)
        shape = (*x.shape[:-1], -(-D // group) if group else 1)
        scales = _out_as("scales_out", scales, shape, torch.float32, x.device, dev)
    _launch(call, call.pack(dt, wdt, x.numel() // D if D else 0, heads, D, xp, xs, rp, rs, gp, gs, wp, eps, y.data_ptr(),
                            _ptr(residual_out), _ptr(scales), group, int(pow2)), dev)
    if given:
        _written(*given)
    return y, scales, residual_out


def _rms_norm_fwd(x, weight, residual, gate, eps, out=None, residual_out=None):
    y, _, s = _norm(x, weight, residual, gate, eps, residual_out, out=out)
    return y if residual is None else (y, s)


class _RMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, gate, eps):
        r = _rms_norm_fwd(x, weight, residual, gate, eps)
        ctx.eps = eps
        ctx.save_for_backward(x if residual is None else r[1], weight, gate)
        ctx.has_residual = residual is not None
        return r

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dresidual=None):
        s, weight, gate = ctx.saved_tensors
        dx, dgate, dw = rms_norm_bwd(s, dy, weight, gate=gate, dresidual=dresidual, eps=ctx.eps,
                                     want_dweight=ctx.needs_input_grad[1])
        return dx, dw, dx if ctx.has_residual else None, dgate, None


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, *, residual: Optional[torch.Tensor] = None,
             gate: Optional[torch.Tensor] = None, eps: float = 1e-6, out: Optional[torch.Tensor] = None,
             residual_out: Optional[torch.Tensor] = None):
    """Root-mean-square norm over the last dimension:
    ``s = x (+ residual)``, ``y = s / sqrt(mean(s^2) + eps) * weight * sigmoid(gate)``
    (a residual or a gate, not both).

    x, residual, gate: [..., D] float32 or bfloat16, D up to 16384; weight: [D] float32 or x's
    dtype, or None. ``gate`` is the output gate of a KDA layer (page
    "atlas_core/kimi_k3/kda.rs", `full_rank_output_gate`) for whole sequences: x [B, T, H, Dv]
    is normed per head. Returns y, or with ``residual`` (y, s): the norm is of the float32
    sum, s is the sum in x's dtype (written to ``residual_out`` if given, which may be
    ``residual`` or ``x`` itself). Gradients flow to x, weight, residual and gate.
    """
    if _recorded(x, weight, residual, gate):
        _no_outs(out=out, residual_out=residual_out)
        return _RMSNorm.apply(x, weight, residual, gate, eps)
    return _rms_norm_fwd(x, weight, residual, gate, eps, out, residual_out)


def rms_norm_quant(x: torch.Tensor, weight: Optional[torch.Tensor] = None, *, residual: Optional[torch.Tensor] = None,
                   gate: Optional[torch.Tensor] = None, eps: float = 1e-6, group_size: int = 0,
                   pow2_scales: bool = False, out: Optional[torch.Tensor] = None,
                   scales_out: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None):
    """``rms_norm`` with the output in 8 bits for an 8-bit product: (q, scales), or with
    ``residual`` (q, scales, s), where q [..., D] is float8_e4m3fn and scales [..., groups]
    float32, y = q * scale. ``group_size`` channels (32, 64 or 128, or 0: the whole row) share
    the scale max(max|y| / 448, 2^-100), with ``pow2_scales`` rounded up to a power of two.
    No gradients: inputs that require grad are refused.
    """
    if _recorded(x, weight, residual, gate):
        raise NotImplementedError("rms_norm_quant has no gradients; use rms_norm")
    q, scales, s = _norm(x, weight, residual, gate, eps, residual_out, (group_size, pow2_scales, scales_out), out)
    return (q, scales) if residual is None else (q, scales, s)


def rms_norm_bwd(x: torch.Tensor, dy: torch.Tensor, weight: Optional[torch.Tensor] = None, *,
                 gate: Optional[torch.Tensor] = None, dresidual: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 want_dweight: bool = True, workspace: Optional[torch.Tensor] = None):
    """Gradients of ``rms_norm``: (dx, dgate or None, dweight or None) from the cotangent ``dy``
    of y. x is what was normed: with a residual, the sum s that the forward returned; dx is
    then the gradient of both terms, and ``dresidual``, the cotangent of s, is added to it.
    """
    _no_tangents(x, dy, weight, gate, dresidual)
    call = _abi.call("kda_rms_norm_bwd")
    dev = _dev("x", x)
    dt = _dtype("x", x)
    D = x.shape[-1]
    wp, wdt = _weight(weight, x, dev)
    if gate is not None and dresidual is not None:
        raise ValueError("dresidual and gate cannot be combined")
    # cotangents come with any strides; dense ones go with every layout of x and gate
    dy = _cotangent("dy", dy, x, dev)
    if dresidual is not None:
        dresidual = _cotangent("dresidual", dresidual, x, dev)
    if any(t is not None and _row_stride(t) is None for t in (x, gate)):
        dy = dy.contiguous()
        dresidual = dresidual if dresidual is None else dresidual.contiguous()
    heads, ((xp, xs), (dp, ds), (gp, gs), (rp, rs)) = _norm_rows((("x", x), ("dy", dy), ("gate", gate), ("dresidual", dresidual)), x, dev)
    dgate = dw = None
    if gate is not None:
        dgate = _out("dgate", None, x, dev)
    dx = _out("dx", None, x, dev)
    if weight is not None and want_dweight:
        dw = torch.empty_like(weight)
    _launch_scratch(call, (dt, wdt, x.numel() // D if D else 0, heads, D, xp, xs, dp, ds, gp, gs, rp, rs, wp, eps, dx.data_ptr(),
                           _ptr(dgate), _ptr(dw)), workspace, x.device, dev)
    return dx, dgate, dw


# --------------------------------------------------------------------------- causal convolution

def _conv_weight(conv_w, x, dev):
    _same_dev("conv_w", conv_w, dev)
    if conv_w.dtype != torch.float32 or conv_w.dim() != 2 or conv_w.shape[0] != x.shape[-1] or not conv_w.is_contiguous():
        raise ValueError(f"conv_w must be a contiguous float32 tensor [{x.shape[-1]}, K]")
    return conv_w.shape[1]


def _causal_conv_fwd(x, conv_w, initial_state, want_final, cu_seqlens, cu_seqlens_cpu, out=None, final_state_out=None):
    call = _abi.call("kda_causal_conv")
    dev = _dev("x", x)
    dt = _dtype("x", x)
    B, T, N, cu, cu_host = _span(x, cu_seqlens, cu_seqlens_cpu, "C")
    C, K = x.shape[2], _conv_weight(conv_w, x, dev)
    xp, xs = _act("x", x, x, dev)
    s0 = _state("initial_state", initial_state, (N, C, K), dev)
    y = _out("out", out, x, dev)
    _wanted(want_final, final_state_out)
    fs = _out_as("final_state_out", final_state_out, (N, C, K), torch.float32, x.device, dev) if want_final else None
    _launch(call, call.pack(dt, B, T, C, K, xp, xs, conv_w.data_ptr(), s0, _ptr(fs), y.data_ptr(), _ptr(cu), _ptr(cu_host), N), dev)
    if out is not None or final_state_out is not None:
        _written(out, final_state_out)
    return y, fs, cu, cu_host


class _CausalConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, conv_w, initial_state, want_final, cu_seqlens, cu_seqlens_cpu):
        y, fs, cu, cu_host = _causal_conv_fwd(x, conv_w, initial_state, want_final, cu_seqlens, cu_seqlens_cpu)
        ctx.save_for_backward(x, conv_w, initial_state, cu, cu_host)
        ctx.set_materialize_grads(False)
        return y, fs

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dfs):
        x, conv_w, s0, cu, cu_host = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
        dx, dw, ds0 = causal_conv_bwd(
            x, conv_w, dy, initial_state=s0, dfinal_state=dfs, cu_seqlens=cu, cu_seqlens_cpu=cu_host,
            want_dconv_w=ctx.needs_input_grad[1], want_dinitial_state=s0 is not None and ctx.needs_input_grad[2])
        return dx, dw, ds0, None, None, None


def causal_conv(x: torch.Tensor, conv_w: torch.Tensor, *, initial_state: Optional[torch.Tensor] = None,
                output_final_state: bool = False, cu_seqlens: Optional[torch.Tensor] = None,
                cu_seqlens_cpu: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                final_state_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Causal depthwise convolution + SiLU over whole sequences: the convolution of
    ``decode_token`` for prompts and training (page "atlas_core/kimi_k3/kda.rs", `conv_update`).

    x: [B, T, C] float32 or bfloat16; conv_w: [C, K] float32, K in 1..8, oldest tap first;
    initial_state: [N, C, K] float32 windows in the layout of ``decode_token``'s conv_state
    (None: zeros). ``cu_seqlens`` (int32, [N+1], B == 1) packs N sequences, on the CPU or, for
    calls that are captured or must not wait, on the device; ``cu_seqlens_cpu``, its host copy,
    is validated when given. Returns (y [B, T, C], final windows [N, C, K] or None);
    ``decode_token`` and ``causal_conv_step`` continue from the windows. Gradients flow to x,
    conv_w and initial_state.
    """
    if _recorded(x, conv_w, initial_state):
        _no_outs(out=out, final_state_out=final_state_out)
        return _CausalConv.apply(x, conv_w, initial_state, output_final_state, cu_seqlens, cu_seqlens_cpu)
    return _causal_conv_fwd(x, conv_w, initial_state, output_final_state, cu_seqlens, cu_seqlens_cpu, out, final_state_out)[:2]


def causal_conv_step(x: torch.Tensor, conv_w: torch.Tensor, conv_state: torch.Tensor, *,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of N sequences: x [N, C], conv_w [C, K] float32, conv_state [N, C, K] float32,
    updated IN PLACE (shifted one slot, x last). Returns silu(w . window) [N, C]. No gradients:
    inputs and states that require grad are refused while gradients are recorded.
    """
    if _recorded(x, conv_w, conv_state):
        raise NotImplementedError("causal_conv_step has no gradients; use causal_conv")
    call = _abi.call("kda_causal_conv_step")
    dev = _dev("x", x)
    dt = _dtype("x", x)
    if x.dim() != 2:
        raise ValueError("x must be [N, C]")
    N, C = x.shape
    K = _conv_weight(conv_w, x, dev)
    xp, xs = _act("x", x, x, dev)
    if conv_state is None:
        raise ValueError("conv_state is required")
    s = _state("conv_state", conv_state, (N, C, K), dev)
    y = _out("out", out, x, dev)
    _launch(call, call.pack(dt, N, C, K, xp, xs, conv_w.data_ptr(), s, y.data_ptr()), dev)
    _written(conv_state, out)
    return y


def causal_conv_bwd(x: torch.Tensor, conv_w: torch.Tensor, dy: torch.Tensor, *,
                    initial_state: Optional[torch.Tensor] = None, dfinal_state: Optional[torch.Tensor] = None,
                    cu_seqlens: Optional[torch.Tensor] = None, cu_seqlens_cpu: Optional[torch.Tensor] = None,
                    want_dconv_w: bool = True, want_dinitial_state: Optional[bool] = None,
                    workspace: Optional[torch.Tensor] = None):
    """Gradients of ``causal_conv``: (dx, dconv_w or None, dinitial_state or None) from the
    cotangents ``dy`` of y and, optionally, ``dfinal_state`` [N, C, K] float32 of the final
    windows. dinitial_state comes with an initial_state unless asked for otherwise.
    """
    _no_tangents(x, conv_w, dy, initial_state, dfinal_state)
    call = _abi.call("kda_causal_conv_bwd")
    dev = _dev("x", x)
    dt = _dtype("x", x)
    B, T, N, cu, cu_host = _span(x, cu_seqlens, cu_seqlens_cpu, "C")
    C, K = x.shape[2], _conv_weight(conv_w, x, dev)
    xp, xs = _act("x", x, x, dev)
    dy = _cotangent("dy", dy, x, dev)
    dp, dst = _act("dy", dy, x, dev)
    s0 = _state("initial_state", initial_state, (N, C, K), dev)
    if dfinal_state is not None:
        dfinal_state = dfinal_state.contiguous()
    dsT = _state("dfinal_state", dfinal_state, (N, C, K), dev)
    if want_dinitial_state is None:
        want_dinitial_state = initial_state is not None
    dx = _out("dx", None, x, dev)
    dw = torch.empty_like(conv_w) if want_dconv_w else None
    ds0 = torch.empty((N, C, K), dtype=torch.float32, device=x.device) if want_dinitial_state else None
    _launch_scratch(call, (dt, B, T, C, K, xp, xs, dp, dst, conv_w.data_ptr(), s0, dsT, dx.data_ptr(), _ptr(dw), _ptr(ds0), _ptr(cu),
                           _ptr(cu_host), N), workspace, x.device, dev)
    return dx, dw, ds0


# --------------------------------------------------------------------------- gated scan

def _scan_gate(sigmoid, lower_bound):
    """(gate form, has bound, bound)"""
    if lower_bound is None:
        return (_abi.KDA_SCAN_GATE_SIGMOID if sigmoid else _abi.KDA_SCAN_GATE_LOG), 0, 0.0
    if sigmoid:
        raise ValueError("lower_bound applies to the log-decay form only")
    if not lower_bound < 0:
        raise ValueError("lower_bound must be negative")
    return _abi.KDA_SCAN_GATE_LOG, 1, float(lower_bound)


def _gated_scan_fwd(x, g, initial_state, want_final, sigmoid, lower_bound, cu_seqlens, cu_seqlens_cpu, out=None,
                    final_state_out=None, workspace=None):
    call = _abi.call("kda_gated_scan")
    dev = _dev("x", x)
    dt = _dtype("x", x)
    gate, has_lb, lb = _scan_gate(sigmoid, lower_bound)
    B, T, N, cu, cu_host = _span(x, cu_seqlens, cu_seqlens_cpu, "D")
    D = x.shape[2]
    xp, xs = _act("x", x, x, dev)
    gp, gs = _act("g", g, x, dev)
    s0 = _state("initial_state", initial_state, (N, D), dev)
    h = _out("out", out, x, dev)
    _wanted(want_final, final_state_out)
    fs = _out_as("final_state_out", final_state_out, (N, D), torch.float32, x.device, dev) if want_final else None
    _launch_scratch(call, (dt, gate, B, T, D, xp, xs, gp, gs, h.data_ptr(), s0, _ptr(fs), _ptr(cu), _ptr(cu_host), N, has_lb, lb),
                    workspace, x.device, dev)
    if out is not None or final_state_out is not None:
        _written(out, final_state_out)
    return h, fs, cu, cu_host


class _GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, g, initial_state, want_final, sigmoid, lower_bound, cu_seqlens, cu_seqlens_cpu):
        h, fs, cu, cu_host = _gated_scan_fwd(x, g, initial_state, want_final, sigmoid, lower_bound, cu_seqlens, cu_seqlens_cpu)
        ctx.save_for_backward(x if sigmoid else None, g, h, initial_state, cu, cu_host)
        ctx.gate = sigmoid, lower_bound
        ctx.set_materialize_grads(False)
        return h, fs

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dfs):
        x, g, h, s0, cu, cu_host = ctx.saved_tensors
        if dh is None:
            dh = torch.zeros(h.shape, dtype=h.dtype, device=h.device)
        dx, dg, ds0 = chunk_gated_scan_bwd(
            x, g, h, dh, initial_state=s0, dfinal_state=dfs, use_gate_sigmoid_in_kernel=ctx.gate[0],
            lower_bound=ctx.gate[1], cu_seqlens=cu, cu_seqlens_cpu=cu_host,
            want_dinitial_state=s0 is not None and ctx.needs_input_grad[2])
        return dx, dg, ds0, None, None, None, None, None


def chunk_gated_scan(x: torch.Tensor, g: torch.Tensor, *, initial_state: Optional[torch.Tensor] = None,
                     output_final_state: bool = False, use_gate_sigmoid_in_kernel: bool = False,
                     lower_bound: Optional[float] = None, cu_seqlens: Optional[torch.Tensor] = None,
                     cu_seqlens_cpu: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                     final_state_out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gated linear recurrence per channel over whole sequences, the elementwise companion of
    ``chunk_kda``: ``h_t = a_t h_{t-1} + x_t``, with ``a = exp(max(g, lower_bound))`` of the
    log-decay g (<= 0); or, with ``use_gate_sigmoid_in_kernel``, of the gate's logit g
    ``a = sigmoid(g)`` and ``h_t = a_t h_{t-1} + (1 - a_t) x_t``.

    x, g: [B, T, D] float32 or bfloat16; initial_state: [N, D] float32 (None: zeros).
    ``cu_seqlens`` as in ``causal_conv``. The state is carried in float32; h is rounded to x's
    dtype as it is written. Returns (h [B, T, D], final state [N, D] float32 or None).
    Gradients flow to x, g and initial_state. A ``workspace`` passed in belongs to one call at
    a time (captured graphs that may overlap need one each).
    """
    if _recorded(x, g, initial_state):
        _no_outs(out=out, final_state_out=final_state_out, workspace=workspace)
        return _GatedScan.apply(x, g, initial_state, output_final_state, use_gate_sigmoid_in_kernel, lower_bound,
                                cu_seqlens, cu_seqlens_cpu)
    return _gated_scan_fwd(x, g, initial_state, output_final_state, use_gate_sigmoid_in_kernel, lower_bound, cu_seqlens,
                           cu_seqlens_cpu, out, final_state_out, workspace)[:2]


def gated_scan_step(x: torch.Tensor, g: torch.Tensor, state: torch.Tensor, *, use_gate_sigmoid_in_kernel: bool = False,
                    lower_bound: Optional[float] = None, out: Optional[torch.Tensor] = None,
                    state_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of N sequences: x, g [N, D]; state [N, D] float32, updated IN PLACE, or only
    read when ``state_out`` (a second buffer, disjoint from it) receives the new state. Gate
    arguments as in ``chunk_gated_scan``. Returns h [N, D]. No gradients: inputs and states that
    require grad are refused while gradients are recorded.
    """
    if _recorded(x, g, state, state_out):
        raise NotImplementedError("gated_scan_step has no gradients; use chunk_gated_scan")
    call = _abi.call("kda_gated_scan_step")
    dev = _dev("x", x)
    dt = _dtype("x", x)
    gate, has_lb, lb = _scan_gate(use_gate_sigmoid_in_kernel, lower_bound)
    if x.dim() != 2:
        raise ValueError("x must be [N, D]")
    N, D = x.shape
    xp, xs = _act("x", x, x, dev)
    gp, gs = _act("g", g, x, dev)
    if state is None:
        raise ValueError("state is required")
    s, so = _state("state", state, (N, D), dev), _state("state_out", state_out, (N, D), dev)
    h = _out("out", out, x, dev)
    _launch(call, call.pack(dt, gate, N, D, xp, xs, gp, gs, s, so, h.data_ptr(), has_lb, lb), dev)
    _written(state if state_out is None else state_out, out)
    return h


def chunk_gated_scan_bwd(x: Optional[torch.Tensor], g: torch.Tensor, h: torch.Tensor, dout: torch.Tensor, *,
                         initial_state: Optional[torch.Tensor] = None, dfinal_state: Optional[torch.Tensor] = None,
                         use_gate_sigmoid_in_kernel: bool = False, lower_bound: Optional[float] = None,
                         cu_seqlens: Optional[torch.Tensor] = None, cu_seqlens_cpu: Optional[torch.Tensor] = None,
                         want_dinitial_state: Optional[bool] = None, workspace: Optional[torch.Tensor] = None):
    """Gradients of ``chunk_gated_scan``: (dx, dg, dinitial_state or None) from the cotangents
    ``dout`` of h and, optionally, ``dfinal_state`` [N, D] float32. h is the forward's output;
    x is needed with ``use_gate_sigmoid_in_kernel`` only (None otherwise). dg is zero where
    the lower bound is taken (g < lower_bound). dinitial_state comes with an initial_state
    unless asked for otherwise.
    """
    _no_tangents(x, g, h, dout, initial_state, dfinal_state)
    call = _abi.call("kda_gated_scan_bwd")
    dev = _dev("g", g)
    dt = _dtype("g", g)
    gate, has_lb, lb = _scan_gate(use_gate_sigmoid_in_kernel, lower_bound)
    if use_gate_sigmoid_in_kernel and x is None:
        raise ValueError("x is required with use_gate_sigmoid_in_kernel")
    B, T, N, cu, cu_host = _span(g, cu_seqlens, cu_seqlens_cpu, "D")
    D = g.shape[2]
    xp, xs = _act("x", x, g, dev) if use_gate_sigmoid_in_kernel else (0, 0)
    gp, gs = _act("g", g, g, dev)
    hp, hs = _act("h", h, g, dev)
    dout = _cotangent("dout", dout, g, dev)
    dp, dst = _act("dout", dout, g, dev)
    s0 = _state("initial_state", initial_state, (N, D), dev)
    if dfinal_state is not None:
        dfinal_state = dfinal_state.contiguous()
    dsT = _state("dfinal_state", dfinal_state, (N, D), dev)
    if want_dinitial_state is None:
        want_dinitial_state = initial_state is not None
    dx, dg = _out("dx", None, g, dev), _out("dg", None, g, dev)
    ds0 = torch.empty((N, D), dtype=torch.float32, device=g.device) if want_dinitial_state else None
    _launch_scratch(call, (dt, gate, B, T, D, xp, xs, gp, gs, hp, hs, dp, dst, s0, dsT, dx.data_ptr(), dg.data_ptr(), _ptr(ds0), _ptr(cu),
                           _ptr(cu_host), N, has_lb, lb), workspace, g.device, dev)
    return dx, dg, ds0
