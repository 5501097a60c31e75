"""RMS norm of many rows against the 64-bit form: CTAs that walk several rows, the next one's
loads under way, with several runs of channels a thread and accesses of every width."""
import pytest
import torch

import layer_ref as ref
from layer_ref import U, half, within

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.float32, torch.bfloat16]
# 601: just enough rows for several runs a thread; else more than twice the rows that run at a time
SHAPES = [(64, 60000), (128, 40000), (257, 601), (257, 15000), (320, 601), (320, 15000), (511, 9000), (1023, 601), (1023, 6000),
          (2048, 601), (2048, 4000), (4096, 2500), (7000, 1500)]


def rows_of(M, D, dtype, seed, shift, scale=1.0):
    """Rows that begin `shift` elements behind a 16-byte boundary, with neighbours in between."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    pitch = D + shift + -(D + shift) % 8
    return (torch.randn(M, pitch, generator=gen, device=DEV) * scale).to(dtype)[:, shift:shift + D]


def weights(kind, D, dtype, seed):
    w = 1 + 0.2 * torch.randn(D, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)
    return None if kind == "none" else w if kind == "f32" else w.to(dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shift", [0, 1, 2])
@pytest.mark.parametrize("D,M", SHAPES)
def test_forward(D, M, shift, dtype):
    import kimi_delta_attention_20_b200 as kda
    x, res, gate = (rows_of(M, D, dtype, D + i, shift, s) for i, s in ((0, 1.0), (1, 3.0), (2, 2.0)))
    tol = half(dtype) + ref.norm_rel(D)
    for kind, kw in (("f32", {}), ("same", dict(residual=res)), ("f32", dict(gate=gate)), ("none", dict(gate=gate))):
        w = weights(kind, D, dtype, D)
        got = kda.rms_norm(x, w, **kw)
        y, s = ref.norm(x, w, **kw)
        within(f"y {list(kw)}", got[0] if "residual" in kw else got, y, y.abs() * tol + 1e-37)
        if "residual" in kw:
            within("sum", got[1], s, s.abs() * (half(dtype) + U))
            # the sum in the place of either term, while the next row is under way
            for k in (0, 1):
                terms = [x.contiguous(), res.contiguous()]
                if terms[k].data_ptr() == (x, res)[k].data_ptr():
                    terms[k] = terms[k].clone()
                again = kda.rms_norm(terms[0], w, residual=terms[1], residual_out=terms[k])
                assert torch.equal(again[1], got[1]) and again[1].data_ptr() == terms[k].data_ptr()
                within("y in place", again[0], y, y.abs() * tol + 1e-37)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shift", [0, 1, 2])
@pytest.mark.parametrize("D,M", SHAPES)
def test_quant(D, M, shift, dtype):
    import kimi_delta_attention_20_b200 as kda
    x, other = rows_of(M, D, dtype, D, shift, 2.0), rows_of(M, D, dtype, D + 1, shift)
    w = weights("f32", D, dtype, D)
    rel = ref.norm_rel(D) + 4 * U
    for group, pow2, kw in ((0, False, dict(residual=other)), (0, True, {}), (32, True, dict(residual=other)), (64, False, dict(gate=other)),
                            (128, False, dict(residual=other)), (128, True, {})):
        q, sc, *s = kda.rms_norm_quant(x, w, group_size=group, pow2_scales=pow2, **kw)
        y, s_ref = ref.norm(x, w, **kw)
        if s:
            within("sum", s[0], s_ref, s_ref.abs() * (half(dtype) + U))
        G = group or D
        want = (torch.stack([p.abs().amax(-1) for p in y.split(G, -1)], -1) / 448).clamp_min(2.0 ** -100)
        if pow2:  # next to a power of two it may fall on either side
            lo, hi = (torch.exp2(torch.ceil(torch.log2(want * (1 + e)))) for e in (-rel, rel))
            assert ((sc.double() == lo) | (sc.double() == hi)).all()
        else:
            within("scales", sc, want, want * rel)
        full = sc.double().repeat_interleave(G, -1)[:, :D]
        # half a step of e4m3: 2^-4 of the value, 2^-10 of the scale below its normal numbers
        within(f"values {group}", q.float().double() * full, y, y.abs() * (half(torch.float8_e4m3fn) + 2 * rel) + full * 2.0 ** -10)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shift", [0, 1, 2])
@pytest.mark.parametrize("D,M", SHAPES)
def test_gradients(D, M, shift, dtype):
    import kimi_delta_attention_20_b200 as kda
    x, dy, third = (rows_of(M, D, dtype, D + i, shift) for i in range(3))
    for kind, gated in (("f32", True), ("same", False)):
        w = weights(kind, D, dtype, D)
        gate, dres = (third, None) if gated else (None, third)
        dx, dgate, dw = kda.rms_norm_bwd(x, dy, w, gate=gate, dresidual=dres)
        rx, rg, rw, mag, wmag = ref.norm_grads(x, dy, w, gate, dres)
        # two terms, each off like y, and the sum of u s by (32 + 5 + 16 + 1) u of its magnitudes
        within("dx", dx, rx, rx.abs() * half(dtype) + mag * (54 * U + 2 * ref.norm_rel(D)))
        if gated:
            p = torch.sigmoid(gate.double())
            slope = rg.abs() / (1 - p).clamp_min(1e-30)  # 1 - sigmoid cancels: off by 6 u of 1
            within("dgate", dgate, rg, rg.abs() * (half(dtype) + 2 * ref.norm_rel(D)) + slope * 6 * U)
        # a thread adds its rows one after another, then the rows of a CTA and the slices are joined: M terms
        # and joins at the very most
        within("dw", dw, rw, rw.abs() * half(w.dtype) + wmag * ((M + 8) * U + ref.norm_rel(D)))
