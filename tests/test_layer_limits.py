"""The operators around the state update at the ends of the ranges that the header gives: what
the entry points plan (CPU), and what the kernels then do (GPU)."""
import ctypes

import pytest
import torch

from kimi_delta_attention_20_b200 import _abi

ROWS = (1 << 31) - 4097  # the most rows of a call
DEV = "cuda"


def scan_bytes(T, dtype, cu, fn="kda_gated_scan"):
    args = (_abi.ScanArgs if fn == "kda_gated_scan" else _abi.ScanBwdArgs)(
        dtype=dtype, B=1, T=T, D=1, x=1 << 24, g=2 << 24, h=3 << 24, N=1, cu_seqlens=cu)
    n = ctypes.c_size_t()
    assert getattr(_abi.load(), fn + "_workspace_size")(ctypes.byref(args), ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("fn", ["kda_gated_scan", "kda_gated_scan_bwd"])
@pytest.mark.parametrize("cu", [None, 4 << 24], ids=["batch", "packed"])
@pytest.mark.parametrize("dtype", [_abi.KDA_DTYPE_F32, _abi.KDA_DTYPE_BF16])
def test_scan_of_the_most_rows_is_cut_as_one_of_fewer(dtype, cu, fn):
    """Pieces fill the GPU whatever the length, so the longest sequences need the workspace of
    somewhat shorter ones: 148 x 7 pieces."""
    want = scan_bytes(2_000_000_000, dtype, cu, fn)
    assert want > 0
    for T in (2_145_000_000, 2_146_000_000, 2_147_478_816, 2_147_478_817, ROWS):
        assert scan_bytes(T, dtype, cu, fn) == want


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
def test_scan_of_the_most_rows(packed):
    """Decays of one leave sums: every row of the longest sequence, its final state and its
    gradients are whole numbers that can be told beforehand."""
    import kimi_delta_attention_20_b200 as kda
    T, late = ROWS, ROWS - 1_000_001  # late: a row of the last piece
    span = dict(cu_seqlens=torch.tensor([0, T], dtype=torch.int32, device=DEV)) if packed else {}
    x, g, d = (torch.zeros(1, T, 1, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    x[0, 5], x[0, late] = 1, 2
    d[0, 7], d[0, T - 1] = 4, 8
    h, fin = kda.chunk_gated_scan(x, g, output_final_state=True, **span)
    assert (h[0, :5] == 0).all() and (h[0, 5:late] == 1).all() and (h[0, late:] == 3).all() and fin.item() == 3
    del x
    dx, dg, _ = kda.chunk_gated_scan_bwd(None, g, h, d, **span)
    del d, g
    assert (dx[0, :8] == 12).all() and (dx[0, 8:] == 8).all()
    # dg = d a h_{t-1}
    assert (dg[0, :6] == 0).all() and (dg[0, 6:8] == 12).all() and (dg[0, 8:late + 1] == 8).all() and (dg[0, late + 1:] == 24).all()
