"""Causal convolution + SiLU over packed sequences, its single token and its gradients
against the 64-bit form."""
import pytest
import torch

import layer_ref as ref
from layer_ref import U, half, within

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.float32, torch.bfloat16]
LENS = [[1], [3], [16], [17], [128], [129], [300], [0, 1, 2, 0, 3, 4, 127, 0, 1, 1, 140, 0], [5, 0, 0, 250], [64, 64, 64], [1] * 40, [0, 0]]


def draw(*shape, dtype, seed, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).to(DEV)


def offsets(lens):
    cu = torch.tensor(ref.bounds_of(lens), dtype=torch.int32)
    return dict(cu_seqlens=cu.to(DEV), cu_seqlens_cpu=cu)


def case(lens, C, K, dtype, seed, windows=True):
    T, N = sum(lens), len(lens)
    x, w = draw(T, C, dtype=dtype, seed=seed), draw(C, K, dtype=torch.float32, seed=seed + 1, scale=0.5)
    s0 = draw(N, C, K, dtype=torch.float32, seed=seed + 2) if windows else None
    return x, w, s0


def y_tol(z, mag, K, dtype):
    """z is off by (K + 1) u of its products' magnitudes, silu's slope is at most 1.1, and
    expf, its sum and a quotient follow."""
    y = (z * torch.sigmoid(z)).abs()
    return y * (half(dtype) + 8 * U) + 1.1 * (K + 1) * U * mag


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [4, 1, 2, 3, 8])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_conv(lens, K, dtype):
    import kimi_delta_attention_20_b200 as kda
    for C, windows in ((1, True), (6, False), (132, True), (259, False)):
        x, w, s0 = case(lens, C, K, dtype, seed=C + K, windows=windows)
        y, fin = kda.causal_conv(x[None], w, initial_state=s0, output_final_state=True, **offsets(lens))
        want, fin_ref, z, mag = ref.conv(x, w, lens, s0)
        within(f"y C{C}", y[0], want, y_tol(z, mag, K, dtype))
        # windows hold inputs: fp32 holds them exactly
        assert torch.equal(fin.double(), fin_ref)
        y2, none = kda.causal_conv(x[None], w, initial_state=s0, **offsets(lens))
        assert none is None and torch.equal(y, y2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [4, 1, 2, 3, 8])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_conv_gradients(lens, K, dtype):
    """dx, dw and the windows' gradients against 64-bit autograd of the plain form."""
    import kimi_delta_attention_20_b200 as kda
    for C, windows, final in ((1, True, True), (6, False, False), (132, True, False), (259, True, True)):
        x, w, s0 = case(lens, C, K, dtype, seed=C + K + 7, windows=windows)
        dy = draw(*x.shape, dtype=dtype, seed=C + 1)
        ds = draw(len(lens), C, K, dtype=torch.float32, seed=C + 2) if final else None
        dx, dw, d0 = kda.causal_conv_bwd(x[None], w, dy[None], initial_state=s0, dfinal_state=ds, **offsets(lens))
        X, W = x.double().requires_grad_(), w.double().requires_grad_()
        S = (torch.zeros(len(lens), C, K, device=DEV) if s0 is None else s0).double().requires_grad_()
        y, fin, z, mag = ref.conv(X, W, lens, S)
        loss = (y * dy.double()).sum()
        if final:
            loss = loss + (fin * ds.double()).sum()
        gx, gw, gs = torch.autograd.grad(loss, (X, W, S), allow_unused=True)
        gx, gw, gs = (torch.zeros_like(t) if g is None else g for g, t in ((gx, X), (gw, W), (gs, S)))
        # dz = dy s (1 + z (1 - s)): the bracket is at most 1.1 + |z| / 4 off s, slope in z at most 1/2;
        # summed magnitudes of the parts of dx (dw) bound their sums' roundings
        zd, md = z.detach(), mag.detach()
        e = dy.double().abs() * (0.5 * (K + 1) * U * md + 16 * U * (1.1 + zd.abs()))
        big = dy.double().abs() * 1.1
        ones = torch.ones_like(W)
        A = x.double().abs().requires_grad_()
        T0 = (torch.zeros_like(S) if s0 is None else s0.double().abs()).requires_grad_()
        lin = linear(A, w.double().abs(), lens, T0)
        ex, e0 = torch.autograd.grad((lin * e).sum(), (A, T0), retain_graph=True, allow_unused=True)
        bx, b0 = torch.autograd.grad((lin * big).sum(), (A, T0), retain_graph=True, allow_unused=True)
        ex, e0, bx, b0 = (torch.zeros_like(t) if v is None else v for v, t in ((ex, A), (e0, T0), (bx, A), (b0, T0)))
        within(f"dx C{C}", dx[0], gx, gx.abs() * half(dtype) + ex + (K + 3) * U * bx + 2 * U * gx.abs())
        Wv = ones.clone().requires_grad_()
        lin = linear(A.detach(), Wv, lens, T0.detach())
        ew, = torch.autograd.grad((lin * e).sum(), Wv, retain_graph=True, allow_unused=True) if sum(lens) else (torch.zeros_like(W),)
        bw, = torch.autograd.grad((lin * big).sum(), Wv, allow_unused=True) if sum(lens) else (torch.zeros_like(W),)
        # 16 rows a thread, then eight warps, then the blocks
        n = 16 + 8 + 8 + 2
        within(f"dw C{C}", dw, gw, ew + n * U * bw + 2 * U * gw.abs())
        if s0 is None:
            assert d0 is None
        else:
            within(f"ds0 C{C}", d0, gs, e0 + (K + 3) * U * b0 + 2 * U * gs.abs())


def linear(x, w, lens, s0):
    """sum_k w[k] in[t-K+1+k] alone."""
    K, out, at = w.shape[1], [], 0
    for n, T in enumerate(lens):
        rows = torch.cat((s0[n].t(), x[at:at + T]))
        out.append(sum((rows[1 + k:1 + k + T] * w[:, k] for k in range(K)), torch.zeros(T, w.shape[0], dtype=torch.float64, device=x.device)))
        at += T
    return torch.cat(out)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [4, 1, 3, 8])
def test_conv_step_continues_a_prompt(K, dtype):
    """A prompt's final windows, continued token by token, give the longer prompt's outputs."""
    import kimi_delta_attention_20_b200 as kda
    N, C, T, steps = 3, 70, 9, 6
    x = draw(N, T + steps, C, dtype=dtype, seed=K)
    w = draw(C, K, dtype=torch.float32, seed=3)
    y, _ = kda.causal_conv(x, w)
    y0, state = kda.causal_conv(x[:, :T].contiguous(), w, output_final_state=True)
    assert torch.equal(y0, y[:, :T])
    for t in range(steps):
        row = x[:, T + t]
        o = kda.causal_conv_step(row, w, state)
        assert torch.equal(o, y[:, T + t])
        full = torch.cat((torch.zeros(N, K, C, dtype=dtype, device=DEV), x[:, :T + t + 1]), 1)[:, -K:]
        assert torch.equal(state, full.transpose(1, 2).float())


def test_conv_matches_decode_token():
    """The windows of the fused decode token and of the prompt form are the same thing."""
    import kimi_delta_attention_20_b200 as kda
    N, H, D, K = 2, 2, 32, 4
    C = 3 * H * D
    x = draw(N, 6, C, dtype=torch.float32, seed=1)
    w = draw(C, K, dtype=torch.float32, seed=2)
    _, cs = kda.causal_conv(x[:, :5].contiguous(), w, output_final_state=True)
    _, full = kda.causal_conv(x, w, output_final_state=True)
    g, beta = -torch.rand(N, H, D, device=DEV), torch.zeros(N, H, device=DEV)
    kda.decode_token(x[:, 5].contiguous(), w, cs, g, beta, torch.zeros(N, H, D, D, device=DEV))
    assert torch.equal(cs, full)


def test_conv_reads_slices_and_keeps_sequences_apart():
    import kimi_delta_attention_20_b200 as kda
    lens, K = [40, 3, 90], 4
    T = sum(lens)
    fused = draw(1, T, 300, dtype=torch.bfloat16, seed=4)
    for lo, C in ((0, 128), (4, 96), (1, 77), (128, 172)):
        w, dy = draw(C, K, dtype=torch.float32, seed=5), draw(1, T, C, dtype=torch.bfloat16, seed=6)
        x = fused[..., lo:lo + C]
        a, b = (kda.causal_conv(t, w, output_final_state=True, **offsets(lens)) for t in (x, x.contiguous()))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        a, b = (kda.causal_conv_bwd(t, w, dy, **offsets(lens)) for t in (x, x.contiguous()))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # what is not finite in one sequence stays there
    C = 64
    w, x, dy = draw(C, K, dtype=torch.float32, seed=7), draw(1, T, C, dtype=torch.float32, seed=8), draw(1, T, C, dtype=torch.float32, seed=9)
    clean, cx = kda.causal_conv(x, w, **offsets(lens))[0], kda.causal_conv_bwd(x, w, dy, **offsets(lens))[0]
    x[0, 41] = float("nan")
    dirty, dx = kda.causal_conv(x, w, **offsets(lens))[0], kda.causal_conv_bwd(x, w, dy, **offsets(lens))[0]
    for sl in (slice(0, 40), slice(43, T)):
        assert torch.equal(clean[0, sl], dirty[0, sl]) and torch.equal(cx[0, sl], dx[0, sl])
    assert dirty[0, 41].isnan().all()


def test_conv_autograd_through_a_batch():
    import kimi_delta_attention_20_b200 as kda
    B, T, C, K = 3, 50, 20, 4
    x, w = draw(B, T, C, dtype=torch.float32, seed=1).requires_grad_(), draw(C, K, dtype=torch.float32, seed=2).requires_grad_()
    s0 = draw(B, C, K, dtype=torch.float32, seed=3).requires_grad_()
    y, fin = kda.causal_conv(x, w, initial_state=s0, output_final_state=True)
    (y.sin().sum() + (fin * fin).sum()).backward()
    X, W, S = (t.detach().double().requires_grad_() for t in (x, w, s0))
    yr, fr, _, _ = ref.conv(X.reshape(-1, C), W, [T] * B, S)
    (yr.sin().sum() + (fr * fr).sum()).backward()
    for n, a, b in (("x", x, X), ("w", w, W), ("s0", s0, S)):
        # fp32 throughout: each gradient is a short sum of products of numbers of order one
        within(n, a.grad, b.grad, 2e-5 * b.grad.abs().max())
