"""Gradients of gates that are wide open or shut."""
import pytest
import torch

import layer_ref as ref
from layer_ref import U, half, within

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,D", [(5, 64), (7, 1023), (700, 512), (2000, 128), (4, 7000), (650, 5003), (3, 16384)])
def test_gradients_of_saturated_gates(M, D, dtype):
    """dgate = dy x r w p (1 - p) falls like exp(-|gate|) on both sides, and holds its digits there."""
    import kimi_delta_attention_20_b200 as kda
    gen = torch.Generator(device=DEV).manual_seed(D)
    x, dy = (torch.randn(M, D, generator=gen, device=DEV).to(dtype) for _ in range(2))
    gate = ((torch.rand(M, D, generator=gen, device=DEV) * 2 - 1) * 60).to(dtype)
    gate[0, 0], gate[1, 0], gate[2, 0] = 0.0, -0.0, 20.0
    w = 1 + 0.2 * torch.randn(D, generator=gen, device=DEV)
    dx, dgate, dw = kda.rms_norm_bwd(x, dy, w, gate=gate)
    rx, _, rw, mag, wmag = ref.norm_grads(x, dy, w, gate)
    # 1 - p as the sigmoid of -gate: by subtraction 64 bits lose it too, from a gate of 37 on
    y, _ = ref.norm(x, w)
    rg = dy.double() * y * torch.sigmoid(gate.double()) * torch.sigmoid(-gate.double())
    # what the norm leaves, twice; the exponential: 4 u, and 2 |gate| u for bf16, whose argument is rounded on its
    # way to the SFU; 1 + e, its reciprocal (2 u), two products and a subtraction
    k = (10 + 2 * gate.double().abs()) * U if dtype == torch.bfloat16 else 10 * U
    within("dgate", dgate, rg, rg.abs() * (half(dtype) + 2 * ref.norm_rel(D) + 2 * k) + 1e-37)
    within("dx", dx, rx, rx.abs() * half(dtype) + mag * (54 * U + 2 * ref.norm_rel(D) + 2 * k) + mag.amax(-1, keepdim=True) * 4 * U)
    within("dw", dw, rw, rw.abs() * half(w.dtype) + wmag * ((M + 8) * U + ref.norm_rel(D) + 130 * U))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [96, 5000])
def test_gates_at_the_ends(D, dtype):
    """Infinite gates are open or shut for good; a NaN stays in its row."""
    import kimi_delta_attention_20_b200 as kda
    x = torch.randn(4, D, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(dtype)
    gate = torch.zeros_like(x)
    gate[0], gate[1], gate[2, 5] = float("inf"), float("-inf"), float("nan")
    dx, dgate, _ = kda.rms_norm_bwd(x, x, gate=gate)
    plain, _, _ = kda.rms_norm_bwd(x, x)
    assert torch.equal(dx[0], plain[0]) and (dx[1] == 0).all() and (dgate[:2] == 0).all()
    assert dx[2].isnan().all() and dgate[2, 5].isnan() and dx[3].isfinite().all() and dgate[3].isfinite().all()
