"""The decay itself, as the states and gradients that are fp32 show it."""
import pytest
import torch

from layer_ref import U, within

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gates():
    """Every negative bf16 number of 2^-12 to 96, then the ends."""
    bits = torch.arange(0xb980, 0xc2c1, dtype=torch.int32)
    g = torch.cat(((bits << 16).view(torch.float32), torch.tensor([0.0, -0.0, -150.0, -3e38, float("-inf")])))
    return g.to(torch.bfloat16).to(DEV)


@pytest.mark.parametrize("lower_bound", [None, -5.0, -0.3])
@pytest.mark.parametrize("rows", [1, 2, 8, 300])
def test_decays_of_bf16_gates(rows, lower_bound):
    """With x = 0 and a state of 1 the final state is the product of the decays, and so is the
    state's gradient. The SFU's exponential of 2 is off by 2 steps (4 u), the rounding of a by
    u, and the split product by less than 1.6 u while a is a normal number; a lower bound that
    is no bf16 number rounds the product, by u of the exponent. Each row's product adds u."""
    import kimi_delta_attention_20_b200 as kda
    g1 = gates()
    D = g1.numel()
    # decays of several rows that come to that of one: the first row's alone, the others' gates 0
    at = rows // 2
    g = torch.zeros(1, rows, D, dtype=torch.bfloat16, device=DEV)
    g[0, at] = g1
    x = torch.zeros_like(g)
    one = torch.ones(1, D, device=DEV)
    kw = dict(lower_bound=lower_bound)
    h, fin = kda.chunk_gated_scan(x, g, initial_state=one, output_final_state=True, **kw)
    _, _, d0 = kda.chunk_gated_scan_bwd(None, g, h, x, initial_state=one, dfinal_state=one, **kw)
    e = g1.double() if lower_bound is None else g1.double().clamp_min(torch.tensor(lower_bound, dtype=torch.float32).item())
    want = torch.exp(e)
    # products with decays of exactly 1 round nothing; what is below the normal numbers may be 0
    k = 7 + (0 if lower_bound is None else -lower_bound)
    tol = want * k * U + 2.0 ** -126
    within("final", fin[0], want, tol)
    within("dinitial", d0[0], want, tol)
    if rows == 1:
        state = one.clone()
        kda.gated_scan_step(x[0], g[0], state, **kw)
        within("step", state[0], want, tol)
        # without a bound the end is reached: nothing of the state is left, not even as NaN
        if lower_bound is None:
            assert (fin[0, -3:] == 0).all() and (fin[0, -5:-3] == 1).all()


def test_a_constant_gate_over_a_long_memory():
    """Errors of one decay that lie the same way at every step: the state behind 4,096 rows of
    the same gate, in fp32, against the geometric sum."""
    import kimi_delta_attention_20_b200 as kda
    T = 4096
    g1 = gates()[:-5]
    g1 = g1[g1 > -8]
    g = g1.expand(1, T, -1).contiguous()
    x = torch.ones_like(g)
    _, fin = kda.chunk_gated_scan(x, g, output_final_state=True)
    a = torch.exp(g1.double())
    want = (1 - a ** T) / (1 - a)
    # a decay off by d moves the sum by d a times its slope, and so do products of decays where
    # rows are cut, by u a factor; every step rounds by u of what it holds
    slope = (want - T * a ** (T - 1)) / (1 - a)
    within("final", fin[0], want, 8 * U * a * slope + U * want * (1 + 2 * want))
