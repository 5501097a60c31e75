"""RMS norm (residual, output gate, 8-bit output) and its gradients against the 64-bit form."""
import pytest
import torch

import layer_ref as ref
from layer_ref import U, half, within

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.float32, torch.bfloat16]
# one channel, fewer than a run, a run and one, part of a warp, warp borders, odd widths, one row per CTA, several runs a thread
DIMS = [1, 3, 8, 9, 32, 64, 100, 128, 255, 256, 512, 520, 1000, 2048, 2049, 4096, 7000, 16384]


def draw(*shape, dtype, seed, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).to(DEV)


def weights(kind, D, dtype, seed):
    if kind == "none":
        return None
    return (1 + 0.2 * torch.randn(D, generator=torch.Generator().manual_seed(seed))).to(
        torch.float32 if kind == "f32" else dtype).to(DEV)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", DIMS)
def test_norm_with_residual_and_gate(D, dtype):
    import kimi_delta_attention_20_b200 as kda
    for rows, kind in ((1, "f32"), (5, "none"), (37, "same")):
        x, res, gate = (draw(rows, D, dtype=dtype, seed=D + rows + i, scale=s) for i, s in ((0, 1.0), (1, 3.0), (2, 2.0)))
        w = weights(kind, D, dtype, seed=D + 3)
        y = kda.rms_norm(x, w)
        want, _ = ref.norm(x, w)
        within(f"plain {rows}x{D}", y, want, want.abs() * (half(dtype) + ref.norm_rel(D)) + 1e-37)
        y, s = kda.rms_norm(x, w, residual=res)
        want, s_ref = ref.norm(x, w, residual=res)
        within(f"residual {rows}x{D}", y, want, want.abs() * (half(dtype) + ref.norm_rel(D)) + 1e-37)
        within(f"sum {rows}x{D}", s, s_ref, s_ref.abs() * (half(dtype) + U))
        y = kda.rms_norm(x, w, gate=gate)
        want, _ = ref.norm(x, w, gate=gate)
        within(f"gated {rows}x{D}", y, want, want.abs() * (half(dtype) + ref.norm_rel(D)) + 1e-37)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("D", [1, 31, 64, 96, 130, 512, 1000, 2048, 5000, 16384])
def test_quant(D, group, pow2, dtype):
    import kimi_delta_attention_20_b200 as kda
    rows = 7
    x, res = draw(rows, D, dtype=dtype, seed=D, scale=2.0), draw(rows, D, dtype=dtype, seed=D + 1)
    x[3] = 0
    res[3] = 0  # a row of zeros
    if D > 1:
        x[4, : D // 2] = 0
        res[4, : D // 2] = 0  # groups of zeros beside others
    w = weights("f32", D, dtype, seed=2)
    q, sc, s = kda.rms_norm_quant(x, w, residual=res, group_size=group, pow2_scales=pow2)
    y, s_ref = ref.norm(x, w, residual=res)
    G = group or D
    groups = -(-D // G)
    assert q.dtype == torch.float8_e4m3fn and q.shape == x.shape and sc.shape == (rows, groups)
    within("sum", s, s_ref, s_ref.abs() * (half(dtype) + U))
    rel = ref.norm_rel(D) + 4 * U
    top = torch.stack([p.abs().amax(-1) for p in y.split(G, -1)], -1)
    want = (top / 448).clamp_min(2.0 ** -100)
    if pow2:
        # a scale next to a power of two may fall on either side of it
        lo, hi = (torch.exp2(torch.ceil(torch.log2(want * (1 + e)))) for e in (-rel, rel))
        assert ((sc.double() == lo) | (sc.double() == hi)).all()
    else:
        within("scales", sc, want, want * rel)
    full = sc.double().repeat_interleave(G, -1)[:, :D]
    # half a step of e4m3: 2^-4 of the value, 2^-10 of the scale below its normal numbers
    back = q.float().double() * full
    within("values", back, y, y.abs() * (half(torch.float8_e4m3fn) + 2 * rel) + full * 2.0 ** -10)
    assert (q[3].float() == 0).all()


def test_quant_non_finite():
    """A NaN makes its row's norm NaN; infinities too where they meet. Other rows are untouched."""
    import kimi_delta_attention_20_b200 as kda
    x = draw(4, 256, dtype=torch.bfloat16, seed=5)
    clean = kda.rms_norm_quant(x, group_size=64)
    x[1, 7] = float("nan")
    q, sc = kda.rms_norm_quant(x, group_size=64)
    assert q[1].float().isnan().all() and sc[1].isnan().all()
    for r in (0, 2, 3):
        assert torch.equal(q[r].view(torch.uint8), clean[0][r].view(torch.uint8)) and torch.equal(sc[r], clean[1][r])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", DIMS)
def test_norm_gradients(D, dtype):
    import kimi_delta_attention_20_b200 as kda
    for rows, kind, gated in ((1, "f32", False), (6, "none", True), (301, "same", True), (1500 if D < 3000 else 400, "f32", False)):
        x, dy, gate, dres = (draw(rows, D, dtype=dtype, seed=D + rows + i) for i in range(4))
        w = weights(kind, D, dtype, seed=D)
        gate = gate if gated else None
        dres = None if gated else dres
        dx, dgate, dw = kda.rms_norm_bwd(x, dy, w, gate=gate, dresidual=dres)
        rx, rg, rw, mag, wmag = ref.norm_grads(x, dy, w, gate, dres)
        # dx: two terms, each off like y, and the sum of u s by (32 + 5 + 16 + 1) u of its magnitudes
        within(f"dx {rows}x{D}", dx, rx, rx.abs() * half(dtype) + mag * (54 * U + 2 * ref.norm_rel(D)))
        if gated:
            # 1 - sigmoid cancels: off by 6 u of 1
            p = torch.sigmoid(gate.double())
            slope = rg.abs() / (1 - p).clamp_min(1e-30)
            within(f"dgate {rows}x{D}", dgate, rg, rg.abs() * (half(dtype) + 2 * ref.norm_rel(D)) + slope * 6 * U)
        if w is None:
            assert dw is None
        else:
            # each thread adds its rows one after another, then the slices are joined
            n = rows + 8
            within(f"dw {rows}x{D}", dw, rw, rw.abs() * half(w.dtype) + wmag * (n * U + ref.norm_rel(D)))


@pytest.mark.parametrize("gated", [False, True])
def test_norm_autograd(gated):
    """Gradients through autograd against 64-bit autograd of the plain form, from a [B, T, H, D] slice."""
    import kimi_delta_attention_20_b200 as kda
    B, T, H, D = 2, 5, 3, 64
    fused = draw(B, T, 3 * H * D, dtype=torch.float32, seed=9)
    w = weights("f32", D, torch.float32, seed=10)
    leaves = {n: fused[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)).contiguous().requires_grad_() for i, n in enumerate(("x", "other"))}
    w.requires_grad_()
    dy, ds = draw(B, T, H, D, dtype=torch.float32, seed=11), draw(B, T, H, D, dtype=torch.float32, seed=12)
    kw = {"gate" if gated else "residual": leaves["other"]}
    r = kda.rms_norm(leaves["x"], w, **kw)
    loss = (r * dy).sum() if gated else (r[0] * dy).sum() + (r[1] * ds).sum()
    loss.backward()
    d = {n: t.detach().double().requires_grad_() for n, t in leaves.items()}
    wd = w.detach().double().requires_grad_()
    y, s = ref.norm(d["x"], wd, **{k: d["other"] for k in kw})
    ((y * dy.double()).sum() if gated else (y * dy.double()).sum() + (s * ds.double()).sum()).backward()
    for n in leaves:
        within(n, leaves[n].grad, d[n].grad, 2e-6 * d[n].grad.abs().max())
    within("w", w.grad, wd.grad, 2e-6 * wd.grad.abs().max())


def test_norm_rows_of_a_fused_projection_and_in_place_sum():
    """Slices are read in place, whatever their alignment; the sum may replace a term."""
    import kimi_delta_attention_20_b200 as kda
    fused = draw(4, 9, 700, dtype=torch.bfloat16, seed=1)
    for lo, D in ((0, 256), (8, 256), (1, 256), (3, 333), (130, 64)):
        x, g = fused[..., lo:lo + D], fused[..., lo + D:lo + 2 * D] if lo + 2 * D <= 700 else fused[..., :D]
        want = ref.norm(x, gate=g)[0]
        within("y", kda.rms_norm(x, gate=g), want, want.abs() * (half(x.dtype) + ref.norm_rel(D)))
        rx, _, _, mag, _ = ref.norm_grads(x, g)
        within("dx", kda.rms_norm_bwd(x, g)[0], rx, rx.abs() * half(x.dtype) + mag * (54 * U + 2 * ref.norm_rel(D)))
    x, res = draw(50, 640, dtype=torch.bfloat16, seed=2), draw(50, 640, dtype=torch.bfloat16, seed=3)
    y, s = kda.rms_norm(x, residual=res)
    for target in ("res", "x"):
        a, b = x.clone(), res.clone()
        y2, s2 = kda.rms_norm(a, residual=b, residual_out=b if target == "res" else a)
        assert s2.data_ptr() == (b if target == "res" else a).data_ptr()
        assert torch.equal(y2, y) and torch.equal(s2, s)


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_of_heads_in_a_fused_projection(dtype):
    """[B, T, H, D] views of slices, whose heads lie back to back and whose tokens do not."""
    import kimi_delta_attention_20_b200 as kda
    B, T, H, D = 2, 7, 3, 40
    fused = draw(B, T, 3 * H * D + 5, dtype=dtype, seed=1)
    x, g, r = (fused[..., k * H * D + 1:(k + 1) * H * D + 1].unflatten(-1, (H, D)) for k in range(3))
    w = weights("f32", D, dtype, seed=2)
    for kw in (dict(), dict(gate=g), dict(residual=r)):
        a, b = kda.rms_norm(x, w, **kw), kda.rms_norm(x.contiguous(), w, **{k: v.contiguous() for k, v in kw.items()})
        want = ref.norm(x, w, **kw)[0]
        within("y", a if torch.is_tensor(a) else a[0], want, want.abs() * (half(dtype) + ref.norm_rel(D)))
        if "residual" in kw:
            assert torch.equal(a[1], b[1])
    q, sc = kda.rms_norm_quant(x, w, gate=g, group_size=32)
    assert q.shape == x.shape and sc.shape == (B, T, H, 2)
    dx, dg, dw = kda.rms_norm_bwd(x, r, w, gate=g)
    rx, rg, rw, mag, wmag = ref.norm_grads(x, r, w, g)
    within("dx", dx, rx, rx.abs() * half(dtype) + mag * (54 * U + 2 * ref.norm_rel(D)))
    within("dw", dw, rw, rw.abs() * half(w.dtype) + wmag * (50 * U + ref.norm_rel(D)))
    with pytest.raises(ValueError):
        kda.rms_norm(fused[..., :H * D].unflatten(-1, (H, D)).transpose(1, 2))


def test_norm_autograd_of_heads_with_strided_cotangents():
    """Heads of a fused projection whose norm is one part of a concatenation: autograd hands
    back a slice whose heads do not lie back to back."""
    import kimi_delta_attention_20_b200 as kda
    B, T, H, D = 2, 5, 3, 24
    fused, w = draw(B, T, 2 * H * D, dtype=torch.float32, seed=1).requires_grad_(), weights("f32", D, torch.float32, seed=2)
    cot = draw(B, T, H, D + 9, dtype=torch.float32, seed=3)
    x, g = (fused[..., k * H * D:(k + 1) * H * D].unflatten(-1, (H, D)) for k in range(2))
    for kw in (dict(gate=g), dict(residual=g)):
        fused.grad = None
        r = kda.rms_norm(x, w, **kw)
        y, s = (r, None) if "gate" in kw else r
        loss = (torch.cat([y, torch.zeros(B, T, H, 9, device=DEV)], -1) * cot).sum()
        if s is not None:
            loss = loss + (torch.cat([torch.zeros(B, T, H, 9, device=DEV), s], -1) * cot).sum()
        loss.backward()
        dres = None if s is None else cot[..., 9:]
        rx, rg, _, mag, _ = ref.norm_grads((x if s is None else s).detach(), cot[..., :D], w, kw.get("gate"), dres)
        got = fused.grad.view(B, T, 2, H, D)
        tol = rx.abs() * half(torch.float32) + mag * (54 * U + 2 * ref.norm_rel(D))
        within("dx", got[:, :, 0], rx, tol)
        if s is not None:
            within("dresidual", got[:, :, 1], rx, tol)


def test_norm_empty_and_large_offsets():
    import kimi_delta_attention_20_b200 as kda
    x = torch.empty(0, 64, device=DEV)
    assert kda.rms_norm(x).shape == (0, 64)
    dx, _, dw = kda.rms_norm_bwd(x, x, torch.ones(64, device=DEV))
    assert dx.shape == (0, 64) and (dw == 0).all()
    # rows beyond 2^31 elements
    rows, D = (1 << 31) // 4096 + 3, 4096
    big = torch.zeros(rows, D, dtype=torch.bfloat16, device=DEV)
    big[-1] = draw(D, dtype=torch.bfloat16, seed=4)
    y = kda.rms_norm(big)
    within("last row", y[-1], ref.norm(big[-1])[0], ref.norm(big[-1])[0].abs() * (half(torch.bfloat16) + ref.norm_rel(D)))
    assert (y[-2] == 0).all()
