"""Gated linear recurrence over packed sequences, its single token and its gradients
against the 64-bit form."""
import pytest
import torch

import layer_ref as ref
from layer_ref import U, half, within

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.float32, torch.bfloat16]
FORMS = [dict(sigmoid=False, lower_bound=None), dict(sigmoid=False, lower_bound=-0.5), dict(sigmoid=True, lower_bound=None)]
# within a chunk of rows, at its borders, over several; empty sequences at the ends and between
LENS = [[1], [31], [32], [33], [63], [64], [65], [200], [0, 1, 64, 3, 0, 130, 0], [64, 64, 0, 64], [1] * 70, [0, 0], [2, 0, 0, 700]]


def kwargs(form):
    return dict(use_gate_sigmoid_in_kernel=form["sigmoid"], lower_bound=form["lower_bound"])


def draw(*shape, dtype, seed, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).to(DEV)


def gates(T, D, sigmoid, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    if sigmoid:
        g = torch.randn(T, D, generator=gen) + 3 * torch.rand(D, generator=gen)
    else:
        g = -torch.exp(6 * torch.rand(D, generator=gen) - 5) * torch.nn.functional.softplus(torch.randn(T, D, generator=gen))
    return g.to(dtype).to(DEV)


def offsets(lens):
    cu = torch.tensor(ref.bounds_of(lens), dtype=torch.int32)
    return dict(cu_seqlens=cu.to(DEV), cu_seqlens_cpu=cu)


def check_scan(lens, D, dtype, form, seed, states=True, span=None):
    import kimi_delta_attention_20_b200 as kda
    T, N = sum(lens), len(lens)
    span = offsets(lens) if span is None else span
    shape = (1, T, D) if span else (N, lens[0], D)
    x, g = draw(T, D, dtype=dtype, seed=seed), gates(T, D, form["sigmoid"], dtype, seed + 1)
    s0 = draw(N, D, dtype=torch.float32, seed=seed + 2) if states else None
    h, fin = kda.chunk_gated_scan(x.view(shape), g.view(shape), initial_state=s0, output_final_state=True, **kwargs(form), **span)
    h_ref, f_ref, e, fe = ref.scan(x, g, lens, s0, **form)
    within("h", h.reshape(T, D), h_ref, h_ref.abs() * half(dtype) + e * 1.01 + 1e-38)
    within("final", fin, f_ref, fe + U * f_ref.abs())
    dout = draw(T, D, dtype=dtype, seed=seed + 3)
    ds = draw(N, D, dtype=torch.float32, seed=seed + 4) if states else None
    dx, dg, d0 = kda.chunk_gated_scan_bwd(x.view(shape), g.view(shape), h, dout.view(shape), initial_state=s0, dfinal_state=ds,
                                          **kwargs(form), **span)
    rx, rg, r0, ex, eg, e0 = ref.scan_grads(x, g, h.reshape(T, D), dout, lens, s0, ds, **form)
    within("dx", dx.reshape(T, D), rx, rx.abs() * half(dtype) + ex * 1.01 + 1e-38)
    within("dg", dg.reshape(T, D), rg, rg.abs() * half(dtype) + eg * 1.01 + 1e-38)
    if states:
        within("ds0", d0, r0, e0 + U * r0.abs())
    else:
        assert d0 is None


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("form", FORMS, ids=str)
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_scan_packed(lens, form, dtype):
    for D, states in ((1, True), (6, False), (132, True), (259, True)):
        check_scan(lens, D, dtype, form, seed=D + len(lens), states=states)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("form", FORMS, ids=str)
@pytest.mark.parametrize("N,T", [(1, 1), (3, 64), (5, 1), (2, 129), (3, 32)])
def test_scan_batch(N, T, form, dtype):
    check_scan([T] * N, 20, dtype, form, seed=N + T, span={})


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens,D", [([5000], 4), ([4700, 0, 300], 130), ([2500], 1000), ([700], 2600), ([300, 40], 20000), ([150], 39000),
                                    ([300, 200, 100, 257], 8448), ([300, 200, 100, 257], 17024),
                                    ([300, 200, 100, 257], 8450), ([300, 200, 100, 257], 8452)])
def test_scan_cut_along_time(lens, D, dtype):
    """Sequences cut into many pieces, few, or none, with lanes of 8 and of 4 bytes."""
    check_scan(lens, D, dtype, FORMS[0], seed=D)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("form", [FORMS[0], FORMS[2]], ids=str)
@pytest.mark.parametrize("lens,D", [([20000], 4), ([9000, 0, 1, 8063, 64, 3000], 41)], ids=str)
def test_scan_cut_into_many_pieces(lens, D, form, dtype):
    """More pieces than a walker composes the maps of itself."""
    check_scan(lens, D, dtype, form, seed=D)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,T,D", [(1, 3000, 20), (3, 500, 260), (4, 300, 8448), (1000, 2, 64), (300, 7, 1024)])
def test_scan_cut_of_a_batch(N, T, D, dtype):
    check_scan([T] * N, D, dtype, FORMS[2], seed=N + T, span={})


@pytest.mark.parametrize("lens", [[40, 0, 600, 1, 1, 1, 300], [0, 0, 900], [700, 0]], ids=str)
def test_scan_with_offsets_on_the_device_alone(lens):
    cu = torch.tensor(ref.bounds_of(lens), dtype=torch.int64, device=DEV)
    for D in (16, 77, 4000):
        check_scan(lens, D, torch.bfloat16, FORMS[0], seed=D, span=dict(cu_seqlens=cu))


def test_scan_repeats_bit_for_bit():
    """What is joined, and in which order, does not depend on timing."""
    import kimi_delta_attention_20_b200 as kda
    T, D = 20000, 300
    x, g = draw(1, T, D, dtype=torch.float32, seed=1), gates(T, D, False, torch.float32, 2)[None]
    h, f = kda.chunk_gated_scan(x, g, output_final_state=True)
    b = kda.chunk_gated_scan_bwd(None, g, h, x)
    busy = torch.randn(4096, 4096, device=DEV)
    other = torch.cuda.Stream()
    for k in range(6):
        if k % 2:
            with torch.cuda.stream(other):
                for _ in range(4):
                    busy @ busy
        h2, f2 = kda.chunk_gated_scan(x, g, output_final_state=True)
        b2 = kda.chunk_gated_scan_bwd(None, g, h, x)
        assert torch.equal(h, h2) and torch.equal(f, f2) and torch.equal(b[0], b2[0]) and torch.equal(b[1], b2[1])


def test_scan_keeps_sequences_apart():
    """What is not finite in one sequence stays there, forwards and backwards, within a chunk
    of rows and across chunks; hard resets (g = -inf) drop what came before."""
    import kimi_delta_attention_20_b200 as kda
    lens = [40, 3, 90, 300]
    T, D = sum(lens), 70
    x, g = draw(1, T, D, dtype=torch.float32, seed=1), gates(T, D, False, torch.float32, 2)[None]
    dout = draw(1, T, D, dtype=torch.float32, seed=3)
    h = kda.chunk_gated_scan(x, g, **offsets(lens))[0]
    dx = kda.chunk_gated_scan_bwd(None, g, h, dout, **offsets(lens))[0]
    for bad in (float("inf"), float("nan")):
        x2, d2 = x.clone(), dout.clone()
        x2[0, 41] = bad
        d2[0, 41] = bad
        h2 = kda.chunk_gated_scan(x2, g, **offsets(lens))[0]
        dx2 = kda.chunk_gated_scan_bwd(None, g, h, d2, **offsets(lens))[0]
        assert not h2[0, 41].isfinite().any()
        for sl in (slice(0, 40), slice(43, T)):
            assert torch.equal(h[0, sl], h2[0, sl]) and torch.equal(dx[0, sl], dx2[0, sl])
    g3 = g.clone()
    g3[0, 200] = float("-inf")
    h3 = kda.chunk_gated_scan(x, g3, **offsets(lens))[0]
    assert torch.equal(h3[0, 200], x[0, 200]) and h3.isfinite().all()


def test_scan_reads_slices():
    import kimi_delta_attention_20_b200 as kda
    T = 150
    fused = -draw(2, T, 600, dtype=torch.bfloat16, seed=4).abs()
    for lo, D in ((0, 128), (4, 96), (1, 77), (128, 172)):
        x, g = fused[..., lo:lo + D], fused[..., lo + D:lo + 2 * D]
        a, b = kda.chunk_gated_scan(x, g)[0], kda.chunk_gated_scan(x.contiguous(), g.contiguous())[0]
        assert torch.equal(a, b)
        a, b = (kda.chunk_gated_scan_bwd(p, q, a, r, use_gate_sigmoid_in_kernel=True) for p, q, r in ((x, g, x), (x.contiguous(), g.contiguous(), x.contiguous())))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("form", FORMS, ids=str)
@pytest.mark.parametrize("D", [1, 7, 128, 1000])
def test_scan_step_continues_a_prompt(D, form, dtype):
    import kimi_delta_attention_20_b200 as kda
    N, T, steps = 3, 70, 4
    x, g = draw(N, T + steps, D, dtype=dtype, seed=D), gates(N * (T + steps), D, form["sigmoid"], dtype, D).view(N, T + steps, D)
    full, _ = kda.chunk_gated_scan(x, g, **kwargs(form))
    _, state = kda.chunk_gated_scan(x[:, :T].contiguous(), g[:, :T].contiguous(), output_final_state=True, **kwargs(form))
    spare = torch.empty_like(state)
    for t in range(T, T + steps):
        keep = state.clone()
        o2 = kda.gated_scan_step(x[:, t], g[:, t], state, state_out=spare, **kwargs(form))
        assert torch.equal(state, keep)
        o = kda.gated_scan_step(x[:, t], g[:, t], state, **kwargs(form))
        assert torch.equal(o, o2) and torch.equal(state, spare)
        h_ref, f_ref, e, fe = ref.scan(x[:, t], g[:, t], [1] * N, keep, **form)
        within("state", state, f_ref, fe + U * f_ref.abs())
        within("h", o, f_ref, f_ref.abs() * half(dtype) + fe * 1.01 + 1e-38)
        if dtype == torch.float32:  # the prompt walked the same tokens
            within("prompt", o, full[:, t].double(), 1e-4 * full[:, t].abs().max())


def test_scan_autograd():
    """Through autograd against 64-bit autograd of the plain form, h rounded to fp32."""
    import kimi_delta_attention_20_b200 as kda
    lens, D = [100, 0, 33], 12
    T = sum(lens)
    for form in FORMS:
        x, g = draw(1, T, D, dtype=torch.float32, seed=1).requires_grad_(), gates(T, D, form["sigmoid"], torch.float32, 2)[None].requires_grad_()
        s0 = draw(3, D, dtype=torch.float32, seed=3).requires_grad_()
        h, fin = kda.chunk_gated_scan(x, g, initial_state=s0, output_final_state=True, **kwargs(form), **offsets(lens))
        (h.sin().sum() + (fin * fin).sum()).backward()
        X, G, S = (t.detach().double().requires_grad_() for t in (x, g, s0))
        hr, fr, _, _ = ref.scan(X[0], G[0], lens, S, **form)
        (hr.sin().sum() + (fr * fr).sum()).backward()
        for n, a, b in (("x", x, X), ("g", g, G), ("s0", s0, S)):
            # runs of at most 100 steps, each off by some 20 u of what it carries
            within(n, a.grad, b.grad, 100 * 30 * U * b.grad.abs().max())
