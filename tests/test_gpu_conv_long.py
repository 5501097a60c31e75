"""The convolution's steady state against the 64-bit form: pieces of more rows than its ring
holds, more slices of the weights' gradient than warps that join them, every window length
with every access width."""
import pytest
import torch

import layer_ref as ref
from layer_ref import U, half, within
from test_gpu_conv import linear, offsets

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.float32, torch.bfloat16]


def draw(*shape, dtype=torch.float32, seed, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV) * scale).to(dtype)


def check(lens, C, K, dtype, seed, windows=True, shift=0):
    import kimi_delta_attention_20_b200 as kda
    T, N = sum(lens), len(lens)
    x, dy = (draw(1, T, C + 8, dtype=dtype, seed=seed + i)[..., shift:shift + C] for i in range(2))
    w = draw(C, K, seed=seed + 2, scale=0.5)
    s0, ds = (draw(N, C, K, seed=seed + 3), draw(N, C, K, seed=seed + 4)) if windows else (None, None)
    span = offsets(lens)
    y, fin = kda.causal_conv(x, w, initial_state=s0, output_final_state=True, **span)
    X, W = x[0].double().requires_grad_(), w.double().requires_grad_()
    S = (torch.zeros(N, C, K, device=DEV) if s0 is None else s0).double().requires_grad_()
    yr, fr, z, mag = ref.conv(X, W, lens, S)
    az = z.detach().abs()
    mag = mag.detach()
    # z: (K + 1) u of its products' magnitudes, at a slope of at most 1.1; the sigmoid: 8 u, and for bf16 (the SFU's
    # exponential) 2 more and 2 |z| of its argument
    sfu = (2 + 2 * az) * U if dtype == torch.bfloat16 else 0
    within("y", y[0], yr.detach(), yr.detach().abs() * (half(dtype) + 8 * U + sfu) + 1.1 * (K + 1) * U * mag)
    assert torch.equal(fin.double(), fr.detach())
    dx, dw, d0 = kda.causal_conv_bwd(x, w, dy, initial_state=s0, dfinal_state=ds, **span)
    loss = (yr * dy[0].double()).sum()
    if ds is not None:
        loss = loss + (fr * ds.double()).sum()
    gx, gw, gs = torch.autograd.grad(loss, (X, W, S))
    # dz: the slope s (1 + z (1 - s)) is below 1.1, and its own slope below 1/2; its sigmoid's error counts |z| + 1.1 times
    d = dy[0].double().abs()
    e, big = d * (0.5 * (K + 1) * U * mag + 16 * U * (1.1 + az)), d * 1.1
    A, T0 = X.detach().abs().requires_grad_(), S.detach().abs().requires_grad_()
    V = torch.ones_like(W).requires_grad_()
    # magnitudes of the parts of each gradient, weighted by the error and by the size of dz
    lin = linear(A, W.detach().abs(), lens, T0)
    ex, e0 = torch.autograd.grad((lin * e).sum(), (A, T0), retain_graph=True)
    bx, b0 = torch.autograd.grad((lin * big).sum(), (A, T0))
    lin = linear(A.detach(), V, lens, T0.detach())
    ew, = torch.autograd.grad((lin * e).sum(), V, retain_graph=True)
    bw, = torch.autograd.grad((lin * big).sum(), V)
    within("dx", dx[0], gx, gx.abs() * half(dtype) + ex + (K + 3) * U * bx + 2 * U * gx.abs())
    # a walker adds its piece row after row (a piece is at least 32 rows, or what a full wave of 2,368 walkers leaves
    # it), a warp its share of the slices, then the 32 warps' sums follow
    units = -(-C // (128 if dtype == torch.bfloat16 else 64))
    piece = max(32, -(-T // max(1, 2368 // units)) + 7)
    n = min(T, piece) + -(-T // piece) // 32 + 1 + 32 + 2
    within("dw", dw, gw, ew + n * U * bw + 2 * U * gw.abs())
    if s0 is not None:
        within("ds0", d0, gs, e0 + (K + 3) * U * b0 + 2 * U * gs.abs())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [3, 4, 8])
@pytest.mark.parametrize("C", [10000, 10001, 10002, 10004])
def test_pieces_longer_than_the_ring(C, K, dtype):
    """72 to 136 rows a walker; the ring holds 24 (backward) and 48."""
    check([700, 0, 3, 1297], C, K, dtype, seed=C + K)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens", [[2000], [7, 1, 1100, 0, 1093]], ids=str)
def test_widest_channels(lens, dtype):
    """A few walkers for each unit of channels: pieces of several hundred rows."""
    check(lens, 30001 if len(lens) > 1 else 30000, 4, dtype, seed=5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [3, 4, 8])
@pytest.mark.parametrize("C", [1, 40, 130, 259])
def test_more_slices_than_warps(C, K, dtype):
    """Up to 157 slices of the weights' gradient."""
    check([2500, 1, 2499], C, K, dtype, seed=C + K)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [5, 6, 7])
@pytest.mark.parametrize("C,shift", [(1, 0), (264, 0), (260, 4), (258, 2), (257, 1), (264, 3)])
def test_other_window_lengths(C, shift, K, dtype):
    """The lengths between 4 and 8, by accesses of 16, 8, 4 and 2 bytes; sequences shorter than the window."""
    for lens in ([300], [0, 1, 2, 0, 3, 4, 5, 6, 7, 8, 127, 0, 1, 140, 0], [1] * 40):
        check(lens, C, K, dtype, seed=C + K + len(lens), shift=shift)
        check(lens, C, K, dtype, seed=C + K + len(lens), shift=shift, windows=False)
