"""The 8-bit norm's quotient next to the borders of e4m3."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = 4096


def near_borders(group, seed):
    """Weights [D] whose groups' scales are any fp32 numbers, and whose other values are a
    scale times the middle of two neighbouring e4m3 values, or up to three fp32 steps off it."""
    gen = torch.Generator().manual_seed(seed)
    G = group or D
    w = torch.empty(D // G, G)
    top = 448 * torch.exp(4 * torch.rand(D // G, generator=gen) - 2)
    scale = top / 448
    for i in range(D // G):
        m, e = torch.randint(8, 16, (G,), generator=gen), torch.randint(-6, 8, (G,), generator=gen)
        v = scale[i] * ((m + 0.5) * torch.exp2(e.float() - 3))
        v = (v.view(torch.int32) + torch.randint(-3, 4, (G,), generator=gen).int()).view(torch.float32)
        w[i] = torch.where(v < top[i], v, top[i] / 2) * torch.where(torch.rand(G, generator=gen) < 0.5, -1, 1)
        w[i, int(torch.randint(0, G, (1,), generator=gen))] = top[i]
    return w.flatten()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [0, 1, 2])  # where rows begin: accesses of 16, 4 and 2 bytes
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("rows", [1, 700])
def test_quotients_are_rounded_once(rows, group, shift, dtype):
    """Rows of ones without eps have y = weight, so y and its scale are known to the bit, and
    with them the fp32 quotient and its nearest e4m3."""
    import kimi_delta_attention_20_b200 as kda
    x = torch.ones(rows, D + shift, dtype=dtype, device=DEV)[:, shift:]
    for seed in range(4):
        w = near_borders(group, seed).to(DEV)
        assert torch.equal(kda.rms_norm(torch.ones(1, D, device=DEV), w, eps=0.0)[0], w)
        q, sc = kda.rms_norm_quant(x, w, eps=0.0, group_size=group)
        # divisions of tensors on the CPU: on the GPU one by a number is a product with its reciprocal
        parts = w.cpu().view(-1, group or D)
        top = parts.abs().amax(-1)
        scale = top / torch.full_like(top, 448.0)
        assert torch.equal(sc.cpu(), scale.expand(rows, -1))
        want = (parts / scale[:, None]).flatten().to(torch.float8_e4m3fn).float()
        assert torch.equal(q.float().cpu(), want.expand(rows, -1))


def test_infinite_and_tiny_scales():
    """A group whose largest value is infinite holds zeros beside a NaN; one of the smallest
    values keeps the floor of the scale."""
    import kimi_delta_attention_20_b200 as kda
    x = torch.ones(3, 256, device=DEV)
    w = torch.ones(256, device=DEV)
    w[:64], w[5], w[64:128] = 3.0, float("inf"), 1e-36
    q, sc = kda.rms_norm_quant(x, w, eps=0.0, group_size=64)
    v = q.float()
    assert sc[:, 0].isinf().all() and v[:, 5].isnan().all() and (v[:, :5] == 0).all() and (v[:, 6:64] == 0).all()
    assert (sc[:, 1] == 2.0 ** -100).all() and (v[:, 64:128] == 0).all()
    assert (v[:, 128:] == 448).all()
