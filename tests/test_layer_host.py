"""Host-side checks of the operators around the state update that need no GPU: the argument
structs' layout, what the C entry points refuse before anything is launched, what the
Python functions refuse, and the 64-bit forms that the GPU tests compare with, against
finite differences and the oracle."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import layer_ref as ref
import oracle
from kimi_delta_attention_20_b200 import _abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = _abi.KDA_ERR_INVALID_ARGUMENT, _abi.KDA_ERR_UNSUPPORTED, _abi.KDA_ERR_WORKSPACE
F32, BF16 = _abi.KDA_DTYPE_F32, _abi.KDA_DTYPE_BF16
A, B, C, D_, E, F, G, H = (0x1000000 * (k + 1) for k in range(8))  # far apart, never dereferenced

STRUCTS = {"kda_rms_norm_args": _abi.RMSNormArgs, "kda_rms_norm_bwd_args": _abi.RMSNormBwdArgs, "kda_conv_args": _abi.ConvArgs,
           "kda_conv_step_args": _abi.ConvStepArgs, "kda_conv_bwd_args": _abi.ConvBwdArgs, "kda_scan_args": _abi.ScanArgs,
           "kda_scan_step_args": _abi.ScanStepArgs, "kda_scan_bwd_args": _abi.ScanBwdArgs}


def test_structs_match_header_layout(tmp_path):
    """The ctypes mirrors and the packed bytes have the layout that the C compiler gives."""
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "kda.h"', "int main(void) {"]
    for name, cls in STRUCTS.items():
        lines.append(f'printf("{name} sizeof %zu\\n", sizeof({name}));')
        lines += [f'printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0; }"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    for line in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        name, field, at = line.split()
        cls = STRUCTS[name]
        assert int(at) == (ctypes.sizeof(cls) if field == "sizeof" else getattr(cls, field).offset), line
    for cls in STRUCTS.values():
        values = [k + 1 for k in range(len(cls._fields_))]
        packed = _abi._packer(cls)(*values)
        assert len(packed) == ctypes.sizeof(cls)
        mirror = cls.from_buffer_copy(packed)
        assert [getattr(mirror, f) for f, _ in cls._fields_] == values


def norm_args(**over):
    a = _abi.RMSNormArgs(dtype=BF16, weight_dtype=F32, rows=8, D=64, x=A, weight=B, eps=1e-6, y=C)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def norm_bwd_args(**over):
    a = _abi.RMSNormBwdArgs(dtype=BF16, weight_dtype=F32, rows=8, D=64, x=A, dy=B, weight=C, eps=1e-6, dx=D_, dweight=E, workspace=F,
                            workspace_bytes=1 << 20)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def conv_args(**over):
    a = _abi.ConvArgs(dtype=BF16, B=1, T=10, C=64, K=4, x=A, conv_w=B, y=C, N=1)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def conv_bwd_args(**over):
    a = _abi.ConvBwdArgs(dtype=BF16, B=1, T=10, C=64, K=4, x=A, dy=B, conv_w=C, dx=D_, dconv_w=E, N=1, workspace=F, workspace_bytes=1 << 20)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def conv_step_args(**over):
    a = _abi.ConvStepArgs(dtype=BF16, N=2, C=64, K=4, x=A, conv_w=B, conv_state=C, y=D_)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def scan_args(**over):
    a = _abi.ScanArgs(dtype=BF16, gate=0, B=1, T=10, D=64, x=A, g=B, h=C, N=1)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def scan_bwd_args(**over):
    a = _abi.ScanBwdArgs(dtype=BF16, gate=0, B=1, T=10, D=64, g=A, h=B, dout=C, dx=D_, dg=E, N=1)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def scan_step_args(**over):
    a = _abi.ScanStepArgs(dtype=BF16, gate=0, N=2, D=64, x=A, g=B, state=C, h=D_)
    for k, v in over.items():
        setattr(a, k, v)
    return a


MAKE = {"kda_rms_norm": norm_args, "kda_rms_norm_bwd": norm_bwd_args, "kda_causal_conv": conv_args, "kda_causal_conv_bwd": conv_bwd_args,
        "kda_causal_conv_step": conv_step_args, "kda_gated_scan": scan_args, "kda_gated_scan_bwd": scan_bwd_args,
        "kda_gated_scan_step": scan_step_args}


@pytest.mark.parametrize("fn,over,want", [
    ("kda_rms_norm", dict(dtype=7), INVALID),
    ("kda_rms_norm", dict(weight_dtype=BF16, dtype=F32), INVALID),
    ("kda_rms_norm", dict(rows=-1), INVALID),
    ("kda_rms_norm", dict(D=0), INVALID),
    ("kda_rms_norm", dict(D=16385), UNSUPPORTED),
    ("kda_rms_norm", dict(rows=1 << 40), INVALID),
    ("kda_rms_norm", dict(heads=-1), INVALID),
    ("kda_rms_norm", dict(heads=3), INVALID),                                # 8 rows are no whole tokens
    ("kda_rms_norm", dict(heads=4, x_stride=255), INVALID),                  # tokens closer than their heads
    ("kda_rms_norm", dict(eps=-1.0), INVALID),
    ("kda_rms_norm", dict(eps=float("nan")), INVALID),
    ("kda_rms_norm", dict(x=None), INVALID),
    ("kda_rms_norm", dict(y=None), INVALID),
    ("kda_rms_norm", dict(x=A + 1), INVALID),
    ("kda_rms_norm", dict(weight=B + 2), INVALID),
    ("kda_rms_norm", dict(x_stride=63), INVALID),
    ("kda_rms_norm", dict(x_stride=-64), INVALID),
    ("kda_rms_norm", dict(y=A), INVALID),                                    # y over x
    ("kda_rms_norm", dict(y=A + 8 * 64 * 2 - 2), INVALID),                   # over its last element
    ("kda_rms_norm", dict(residual=D_, gate=E), UNSUPPORTED),
    ("kda_rms_norm", dict(residual=D_, residual_out=D_ + 64), INVALID),      # partly over the residual
    ("kda_rms_norm", dict(residual=D_, residual_stride=65, residual_out=D_), INVALID),
    ("kda_rms_norm", dict(residual=D_, residual_out=C), INVALID),            # over y
    ("kda_rms_norm", dict(scales=D_, group_size=48), UNSUPPORTED),
    ("kda_rms_norm", dict(scales=D_ + 2), INVALID),
    ("kda_rms_norm_bwd", dict(dy=None), INVALID),
    ("kda_rms_norm_bwd", dict(dx=A), INVALID),
    ("kda_rms_norm_bwd", dict(gate=G), INVALID),                             # its gradient has no place
    ("kda_rms_norm_bwd", dict(dgate=G), INVALID),                            # a gradient without its gate
    ("kda_rms_norm_bwd", dict(gate=G, dgate=H, dresidual=0x10), UNSUPPORTED),
    ("kda_rms_norm_bwd", dict(weight=None), INVALID),
    ("kda_rms_norm_bwd", dict(workspace=None), WORKSPACE),
    ("kda_rms_norm_bwd", dict(workspace_bytes=16), WORKSPACE),
    ("kda_rms_norm_bwd", dict(workspace=F + 4), WORKSPACE),
    ("kda_causal_conv", dict(K=0), UNSUPPORTED),
    ("kda_causal_conv", dict(K=9), UNSUPPORTED),
    ("kda_causal_conv", dict(C=0), INVALID),
    ("kda_causal_conv", dict(B=0), INVALID),
    ("kda_causal_conv", dict(T=-1), INVALID),
    ("kda_causal_conv", dict(B=1 << 16, T=1 << 16, N=1 << 16), INVALID),     # rows beyond 32 bits
    ("kda_causal_conv", dict(N=2), INVALID),
    ("kda_causal_conv", dict(B=2, N=2, cu_seqlens=D_), INVALID),
    ("kda_causal_conv", dict(cu_seqlens=D_, N=0), INVALID),
    ("kda_causal_conv", dict(cu_seqlens=D_ + 2), INVALID),
    ("kda_causal_conv", dict(conv_w=None), INVALID),
    ("kda_causal_conv", dict(y=None), INVALID),
    ("kda_causal_conv", dict(y=A), INVALID),
    ("kda_causal_conv", dict(initial_state=D_, final_state=D_), INVALID),
    ("kda_causal_conv", dict(x_stride=10), INVALID),
    ("kda_causal_conv_bwd", dict(dy=None), INVALID),
    ("kda_causal_conv_bwd", dict(dx=B), INVALID),
    ("kda_causal_conv_bwd", dict(workspace=None), WORKSPACE),
    ("kda_causal_conv_bwd", dict(workspace_bytes=100), WORKSPACE),
    ("kda_causal_conv_step", dict(N=-1), INVALID),
    ("kda_causal_conv_step", dict(conv_state=None), INVALID),
    ("kda_causal_conv_step", dict(y=A), INVALID),
    ("kda_causal_conv_step", dict(K=9), UNSUPPORTED),
    ("kda_gated_scan", dict(gate=2), INVALID),
    ("kda_gated_scan", dict(gate=1, has_lower_bound=1, lower_bound=-1.0), INVALID),
    ("kda_gated_scan", dict(has_lower_bound=1, lower_bound=0.0), INVALID),
    ("kda_gated_scan", dict(has_lower_bound=1, lower_bound=float("nan")), INVALID),
    ("kda_gated_scan", dict(D=0), INVALID),
    ("kda_gated_scan", dict(g=None), INVALID),
    ("kda_gated_scan", dict(h=A), INVALID),
    ("kda_gated_scan", dict(initial_state=D_, final_state=D_ + 128), INVALID),
    ("kda_gated_scan", dict(T=4096), WORKSPACE),                             # cut along time
    ("kda_gated_scan", dict(T=4096, workspace=D_ + 8, workspace_bytes=1 << 24), WORKSPACE),
    ("kda_gated_scan_bwd", dict(h=None), INVALID),
    ("kda_gated_scan_bwd", dict(gate=1), INVALID),                           # the sigmoid form reads x
    ("kda_gated_scan_bwd", dict(dg=D_), INVALID),                            # over dx
    ("kda_gated_scan_bwd", dict(T=4096), WORKSPACE),
    ("kda_gated_scan_step", dict(state=None), INVALID),
    ("kda_gated_scan_step", dict(state_out=C + 16), INVALID),                # partly over the state
    ("kda_gated_scan_step", dict(h=C), INVALID),
    ("kda_gated_scan_step", dict(state=C + 2), INVALID),
])
def test_entry_points_refuse(fn, over, want):
    lib = _abi.load()
    assert getattr(lib, fn)(ctypes.byref(MAKE[fn](**over)), None) == want
    assert getattr(lib, fn)(None, None) == INVALID


@pytest.mark.parametrize("fn,over", [
    ("kda_causal_conv", dict(C=(1 << 28) + 1)), ("kda_causal_conv_bwd", dict(C=1 << 30)), ("kda_causal_conv_step", dict(C=(1 << 31) - 1)),
    ("kda_gated_scan", dict(D=(1 << 28) + 1)), ("kda_gated_scan_bwd", dict(D=1 << 30)), ("kda_gated_scan_step", dict(D=(1 << 31) - 1)),
])
def test_entry_points_refuse_channels_beyond_their_range(fn, over):
    assert getattr(_abi.load(), fn)(ctypes.byref(MAKE[fn](**over)), None) == INVALID


@pytest.mark.parametrize("fn,over", [
    ("kda_rms_norm_bwd", dict(workspace=A)), ("kda_rms_norm_bwd", dict(workspace=E)), ("kda_causal_conv_bwd", dict(workspace=B)),
    ("kda_causal_conv_bwd", dict(workspace=D_ + 64)), ("kda_gated_scan", dict(T=4096, workspace=B, workspace_bytes=1 << 24)),
    ("kda_gated_scan", dict(T=4096, workspace=C - 16, workspace_bytes=1 << 24)),
    ("kda_gated_scan_bwd", dict(T=4096, workspace=B + 64, workspace_bytes=1 << 24)),
    ("kda_gated_scan_bwd", dict(T=4096, workspace=E, workspace_bytes=1 << 24)),
])
def test_entry_points_refuse_a_workspace_over_a_tensor(fn, over):
    assert getattr(_abi.load(), fn)(ctypes.byref(MAKE[fn](**over)), None) == INVALID


@pytest.mark.parametrize("fn", ["kda_causal_conv", "kda_causal_conv_bwd", "kda_gated_scan", "kda_gated_scan_bwd"])
@pytest.mark.parametrize("cu", [[1, 10], [0, 9], [0, 7, 5, 10]])
def test_entry_points_refuse_bad_offsets(fn, cu):
    lib = _abi.load()
    host = (ctypes.c_int32 * len(cu))(*cu)
    a = MAKE[fn](cu_seqlens=G, cu_seqlens_host=ctypes.addressof(host), N=len(cu) - 1)
    assert getattr(lib, fn)(ctypes.byref(a), None) == INVALID
    a = MAKE[fn](cu_seqlens_host=ctypes.addressof(host))  # a host copy of nothing
    assert getattr(lib, fn)(ctypes.byref(a), None) == INVALID


def test_empty_calls_launch_nothing():
    lib = _abi.load()
    before = lib.kda_launch_count()
    assert lib.kda_rms_norm(ctypes.byref(norm_args(rows=0, x=None, y=None)), None) == 0
    assert lib.kda_rms_norm_bwd(ctypes.byref(norm_bwd_args(rows=0, x=None, dy=None, dx=None, dweight=None)), None) == 0
    assert lib.kda_causal_conv(ctypes.byref(conv_args(T=0, x=None, y=None)), None) == 0
    assert lib.kda_causal_conv_step(ctypes.byref(conv_step_args(N=0, x=None)), None) == 0
    assert lib.kda_gated_scan(ctypes.byref(scan_args(T=0, x=None, g=None, h=None)), None) == 0
    assert lib.kda_gated_scan_step(ctypes.byref(scan_step_args(N=0, x=None)), None) == 0
    assert lib.kda_launch_count() == before


def test_workspace_sizes_read_shapes():
    lib = _abi.load()
    n = ctypes.c_size_t(7)
    assert lib.kda_rms_norm_bwd_workspace_size(ctypes.byref(norm_bwd_args(x=None, dy=None)), ctypes.byref(n)) == 0 and n.value > 0
    assert lib.kda_rms_norm_bwd_workspace_size(ctypes.byref(norm_bwd_args(dweight=None)), ctypes.byref(n)) == 0 and n.value == 0
    assert lib.kda_causal_conv_bwd_workspace_size(ctypes.byref(conv_bwd_args(x=None)), ctypes.byref(n)) == 0 and n.value >= 64 * 4 * 4
    assert lib.kda_gated_scan_workspace_size(ctypes.byref(scan_args()), ctypes.byref(n)) == 0 and n.value == 0
    assert lib.kda_gated_scan_workspace_size(ctypes.byref(scan_args(T=4096)), ctypes.byref(n)) == 0 and n.value > 0
    assert lib.kda_gated_scan_bwd_workspace_size(ctypes.byref(scan_bwd_args(T=4096)), ctypes.byref(n)) == 0 and n.value > 0
    for fn, a in (("kda_gated_scan", scan_args), ("kda_gated_scan_bwd", scan_bwd_args), ("kda_causal_conv_bwd", conv_bwd_args),
                  ("kda_rms_norm_bwd", norm_bwd_args)):
        assert getattr(lib, fn + "_workspace_size")(ctypes.byref(a()), None) == INVALID
        assert getattr(lib, fn + "_workspace_size")(None, ctypes.byref(n)) == INVALID


def test_python_functions_refuse_cpu_tensors():
    import kimi_delta_attention_20_b200 as kda
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    for call in (lambda: kda.rms_norm(x), lambda: kda.rms_norm_quant(x), lambda: kda.rms_norm_bwd(x, x), lambda: kda.causal_conv(x, w),
                 lambda: kda.causal_conv_bwd(x, w, x), lambda: kda.causal_conv_step(x[0], w, torch.zeros(4, 8, 4)),
                 lambda: kda.chunk_gated_scan(x, x), lambda: kda.chunk_gated_scan_bwd(None, x, x, x),
                 lambda: kda.gated_scan_step(x[0], x[0], torch.zeros(4, 8)), lambda: kda.rms_norm([1.0])):
        with pytest.raises((ValueError, AttributeError)):
            call()


def test_row_strides():
    from kimi_delta_attention_20_b200.layer_ops import _row_stride
    t = torch.zeros(2, 5, 40)
    assert _row_stride(t) == 0
    assert _row_stride(t[..., 3:20]) == 40
    assert _row_stride(t[0, :, :7]) == 40
    assert _row_stride(t[:, 2]) == 200 and _row_stride(t[:1, :3]) == 0
    assert _row_stride(t[:, :3]) is None           # rows of two batches, unevenly apart
    assert _row_stride(t[..., ::2]) is None        # channels apart
    assert _row_stride(t.transpose(1, 2)) is None
    assert _row_stride(torch.zeros(1, 1, 40).expand(2, 5, 40)) is None   # the same row again and again
    assert _row_stride(torch.zeros(3, 1)[:, 0:1]) == 0


# --------------------------------------------------------------------------- the 64-bit forms

def rnd(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def difference(f, args, k, cot, step=1e-6):
    """Central differences of sum(f * cot) for argument k."""
    g = torch.zeros_like(args[k])
    for i in range(g.numel()):
        ends = []
        for s in (step, -step):
            a = [t.clone() for t in args]
            a[k].view(-1)[i] += s
            ends.append(sum((o * c).sum() for o, c in zip(f(*a), cot)))
        g.view(-1)[i] = (ends[0] - ends[1]) / (2 * step)
    return g


def test_norm_reference_against_differences():
    x, w, gate, dy, dres = rnd(3, 7, seed=1), rnd(7, seed=2), rnd(3, 7, seed=3), rnd(3, 7, seed=4), rnd(3, 7, seed=5)
    dx, dg, dw, _, _ = ref.norm_grads(x, dy, w, gate)
    f = lambda x, w, g: (ref.norm(x, w, gate=g)[0],)  # noqa: E731
    for k, got in ((0, dx), (1, dw), (2, dg)):
        assert torch.allclose(got, difference(f, [x, w, gate], k, [dy]), atol=1e-7)
    dx, _, dw, _, _ = ref.norm_grads(x, dy, w, None, dres)
    assert torch.allclose(dx, difference(lambda x, w: ref.norm(x, w), [x, w], 0, [dy, dres]), atol=1e-7)


def test_conv_reference_is_the_oracle_token_by_token():
    K, C, T = 4, 5, 9
    x, w, s0 = rnd(T, C, seed=1), rnd(C, K, seed=2), rnd(1, C, K, seed=3)
    y, fin, _, _ = ref.conv(x, w, [T], s0)
    state = s0.numpy()
    for t in range(T):
        o, state = oracle.conv_update(state, x[t:t + 1].numpy(), w.numpy())
        np.testing.assert_allclose(y[t].numpy(), o[0], rtol=1e-12)
    np.testing.assert_array_equal(fin.numpy(), state)


def test_scan_reference_gradients_against_differences():
    lens = [3, 0, 2]
    T, D = sum(lens), 2
    x, g, s0 = rnd(T, D, seed=1), -rnd(T, D, seed=2).abs(), rnd(3, D, seed=3)
    dout, ds = rnd(T, D, seed=4), rnd(3, D, seed=5)
    for form in (dict(sigmoid=False, lower_bound=None), dict(sigmoid=False, lower_bound=-0.7), dict(sigmoid=True, lower_bound=None)):
        h, fin, _, _ = ref.scan(x, g, lens, s0, **form)
        assert torch.equal(fin[1], s0[1])
        dx, dg, d0, _, _, _ = ref.scan_grads(x, g, h, dout, lens, s0, ds, **form)
        f = lambda x, g, s: ref.scan(x, g, lens, s, **form)[:2]  # noqa: B023, E731
        for k, got in ((0, dx), (1, dg), (2, d0)):
            assert torch.allclose(got, difference(f, [x, g, s0], k, [dout, ds]), atol=1e-7)
