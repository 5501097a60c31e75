"""The operators around the state update run together, as a layer uses them: prompts and
decoding, training, other streams, captured graphs, and calls that the functions refuse."""
import pytest
import torch

import layer_ref as ref
from layer_ref import within

pytestmark = pytest.mark.gpu
DEV = "cuda"


def draw(*shape, dtype=torch.float32, seed=0, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).to(DEV)


def offsets(lens):
    cu = torch.tensor(ref.bounds_of(lens), dtype=torch.int32)
    return dict(cu_seqlens=cu.to(DEV), cu_seqlens_cpu=cu)


class KDALayer:
    """norm (+ residual) -> fused projection -> convolution -> chunk_kda -> gated norm -> projection."""

    def __init__(self, model, H, D, K=4, dtype=torch.float32):
        self.H, self.D, self.dtype = H, D, dtype
        self.C = 3 * H * D
        self.w_norm = 1 + draw(model, seed=1, scale=0.1)
        # q | k | v | decay | output gate | beta
        self.w_in = draw(model, 5 * H * D + H, dtype=dtype, seed=2, scale=model ** -0.5)
        self.w_conv = draw(self.C, K, seed=3, scale=0.5)
        self.w_out = draw(H * D, model, dtype=dtype, seed=4, scale=(H * D) ** -0.5)

    def project(self, x, residual):
        import kimi_delta_attention_20_b200 as kda
        y, s = kda.rms_norm(x, self.w_norm, residual=residual)
        p = y @ self.w_in
        H, D = self.H, self.D
        qkv, g, gate, beta = p.split((self.C, H * D, H * D, H), -1)
        g = -torch.nn.functional.softplus(g.float()).to(self.dtype).unflatten(-1, (H, D))
        return s, qkv, g.contiguous(), gate.unflatten(-1, (H, D)), beta.contiguous()

    def prompt(self, x, residual, lens, conv_state=None, state=None):
        import kimi_delta_attention_20_b200 as kda
        s, qkv, g, gate, beta = self.project(x, residual)
        span = offsets(lens)
        qkv, conv_state = kda.causal_conv(qkv, self.w_conv, initial_state=conv_state, output_final_state=True, **span)
        q, k, v = (t.unflatten(-1, (self.H, self.D)).contiguous() for t in qkv.chunk(3, -1))
        o, state = kda.chunk_kda(q, k, v, g, beta, use_qk_l2norm_in_kernel=True, initial_state=state, output_final_state=True, **span)
        o = kda.rms_norm(o, gate=gate)
        return s + o.flatten(-2) @ self.w_out, conv_state, state

    def token(self, x, residual, conv_state, state):
        import kimi_delta_attention_20_b200 as kda
        s, qkv, g, gate, beta = self.project(x, residual)
        o = kda.decode_token(qkv.contiguous(), self.w_conv, conv_state, g, beta, state, g_out=gate.contiguous())
        return s + o.flatten(-2) @ self.w_out


def test_kda_layer_prompt_then_tokens_equals_the_longer_prompt():
    """Packed prompts through the layer, continued by the fused decode token, against the same
    tokens as longer prompts; and a prompt cut in two, with windows and states handed on."""
    layer = KDALayer(model=96, H=2, D=64)
    lens, steps = [37, 5], 3
    full = [draw(n + steps, 96, seed=10 + i) for i, n in enumerate(lens)]
    res = [draw(n + steps, 96, seed=20 + i) for i, n in enumerate(lens)]
    pack = lambda ts, a, b: torch.cat([t[a(n):b(n)] for t, n in zip(ts, lens)])[None]  # noqa: E731
    want, _, _ = layer.prompt(pack(full, lambda n: 0, lambda n: n + steps), pack(res, lambda n: 0, lambda n: n + steps), [n + steps for n in lens])
    got, cs, S = layer.prompt(pack(full, lambda n: 0, lambda n: n), pack(res, lambda n: 0, lambda n: n), lens)
    at = ref.bounds_of([n + steps for n in lens])
    # the chunk forward's bar for fp32 is 1e-4 of the scale; the norm before and after it divides by numbers of order one
    tol = 4e-4 * want.abs().max()
    for i, n in enumerate(lens):
        within(f"prompt {i}", got[0, ref.bounds_of(lens)[i]:ref.bounds_of(lens)[i + 1]], want[0, at[i]:at[i] + n], tol)
    first, cs1, S1 = layer.prompt(pack(full, lambda n: 0, lambda n: 4), pack(res, lambda n: 0, lambda n: 4), [4, 4])
    _, cs2, S2 = layer.prompt(pack(full, lambda n: 4, lambda n: n), pack(res, lambda n: 4, lambda n: n), [n - 4 for n in lens], cs1, S1)
    within("windows", cs2, cs, 1e-5 * cs.abs().max())
    within("states", S2, S, 2e-4 * S.abs().max())
    for t in range(steps):
        x = torch.stack([f[n + t] for f, n in zip(full, lens)])
        r = torch.stack([f[n + t] for f, n in zip(res, lens)])
        o = layer.token(x, r, cs, S)
        within(f"token {t}", o, torch.stack([want[0, at[i] + n + t] for i, n in enumerate(lens)]), tol)


def scan_layer(x, res, p, step=None, dbl=False, lens=None):
    """norm (+ residual) -> projection -> convolution -> gated scan -> gated norm. `step`: the
    windows and states of a decoding step, updated in place; dbl: the 64-bit form."""
    import kimi_delta_attention_20_b200 as kda
    D = p["conv"].shape[0]
    if dbl:
        y, s = ref.norm(x, p["w"], residual=res)
        u, g, z = (y @ p["proj"]).split(D, -1)
        c = ref.conv(u[0], p["conv"], lens)[0]
        h = ref.scan(c, g[0], lens, sigmoid=True)[0]
        return ref.norm(h, gate=z[0])[0], s
    y, s = kda.rms_norm(x, p["w"], residual=res)
    u, g, z = (y @ p["proj"]).split(D, -1)
    if step is not None:
        c = kda.causal_conv_step(u, p["conv"], step[0])
        h = kda.gated_scan_step(c, g, step[1], use_gate_sigmoid_in_kernel=True)
        return kda.rms_norm(h, gate=z), s
    span = offsets(lens)
    c, cs = kda.causal_conv(u, p["conv"], output_final_state=True, **span)
    h, st = kda.chunk_gated_scan(c, g, use_gate_sigmoid_in_kernel=True, output_final_state=True, **span)
    return kda.rms_norm(h, gate=z), s, cs, st


def scan_params(model, D):
    return {"w": 1 + draw(model, seed=1, scale=0.1), "proj": draw(model, 3 * D, seed=2, scale=model ** -0.5), "conv": draw(D, 4, seed=3, scale=0.5)}


def test_scan_layer_prompt_then_tokens():
    lens, steps, model, D = [50, 3], 4, 40, 72
    p = scan_params(model, D)
    x, r = draw(1, sum(lens) + 2 * steps, model, seed=5), draw(1, sum(lens) + 2 * steps, model, seed=6)
    full = [n + steps for n in lens]
    want = scan_layer(x, r, p, lens=full)[0]
    at = ref.bounds_of(full)
    keep = torch.cat([torch.arange(at[i], at[i] + n) for i, n in enumerate(lens)]).to(DEV)
    got, _, cs, st = scan_layer(x[:, keep], r[:, keep], p, lens=lens)
    # the same arithmetic up to the order of fp32 sums in the projection
    within("prompt", got[0], want[0, keep], 1e-4 * want.abs().max())
    for t in range(steps):
        rows = torch.tensor([at[i] + n + t for i, n in enumerate(lens)], device=DEV)
        o, _ = scan_layer(x[0, rows], r[0, rows], p, step=(cs, st))
        within(f"token {t}", o, want[0, rows], 1e-4 * want.abs().max())


def test_scan_layer_gradients():
    """All gradients of the layer against 64-bit autograd of the plain forms."""
    lens, model, D = [70, 1, 0, 29], 24, 36
    T = sum(lens)
    p = scan_params(model, D)
    x, r = draw(1, T, model, seed=5), draw(1, T, model, seed=6)
    dy, ds = draw(1, T, D, seed=7), draw(1, T, model, seed=8)
    leaves = {**p, "x": x, "r": r}
    lo = {k: v.clone().requires_grad_() for k, v in leaves.items()}
    hi = {k: v.double().requires_grad_() for k, v in leaves.items()}
    o = scan_layer(lo["x"], lo["r"], lo, lens=lens)
    ((o[0] * dy).sum() + (o[1] * ds).sum()).backward()
    y, s = scan_layer(hi["x"], hi["r"], hi, lens=lens, dbl=True)
    ((y * dy[0].double()).sum() + (s * ds.double()).sum()).backward()
    for k in leaves:
        # fp32 chains of four operators and a product, gradients summed over 100 rows
        within(k, lo[k].grad, hi[k].grad, 2e-4 * hi[k].grad.abs().max())


def calls(p):
    """One call of everything, on tensors of the current stream: outputs, gradients, updated states."""
    import kimi_delta_attention_20_b200 as kda
    x, g, w, cw, dy = p["x"], p["g"], p["w"], p["cw"], p["dy"]
    y, s = kda.rms_norm(x, w, residual=dy)
    q, sc = kda.rms_norm_quant(x, w, group_size=32)
    out = [y, s, q.view(torch.uint8), sc, *kda.rms_norm_bwd(x, dy, w, gate=g)]
    c, cs = kda.causal_conv(x, cw, output_final_state=True)
    out += [c, cs, *kda.causal_conv_bwd(x, cw, dy, initial_state=cs)]
    h, f = kda.chunk_gated_scan(x, g, output_final_state=True, lower_bound=-3.0)
    out += [h, f, *kda.chunk_gated_scan_bwd(None, g, h, dy, initial_state=f, dfinal_state=f, lower_bound=-3.0)]
    st, win = f.clone(), cs.clone()
    out += [kda.gated_scan_step(x[:, 0], g[:, 0], st), st, kda.causal_conv_step(x[:, 0], cw, win), win]
    return [t for t in out if t is not None]


def call_params(seed, B=2, T=700, D=96, dtype=torch.bfloat16):
    return {"x": draw(B, T, D, dtype=dtype, seed=seed), "g": -draw(B, T, D, dtype=dtype, seed=seed + 1).abs(), "w": draw(D, seed=seed + 2),
            "cw": draw(D, 4, seed=seed + 3), "dy": draw(B, T, D, dtype=dtype, seed=seed + 4)}


def same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_on_another_stream():
    """Work queued on a side stream, behind work that delays it, is the default stream's."""
    p = call_params(1)
    want = calls(p)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device=DEV)
    with torch.cuda.stream(side):
        for _ in range(10):
            busy = busy @ busy * 1e-4
        late = {k: v.clone() for k, v in p.items()}  # ready behind the products only
        got = calls(late)
    side.synchronize()
    assert same(want, got)


def test_two_captured_graphs():
    """Two graphs of the same calls, replayed at the same time on two streams and again with
    other inputs, give each its own results."""
    ps = [call_params(10), call_params(20)]
    news = [call_params(30), call_params(40)]
    want = [calls(p) for p in ps]
    again = [calls(p) for p in news]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in ps]
    for p in ps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(calls(p))
        graphs.append(g)
    for expect, inputs in ((want, None), (again, news)):
        if inputs:
            for p, n in zip(ps, inputs):
                for k in p:
                    p[k].copy_(n[k])
        torch.cuda.synchronize()
        for _ in range(3):
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for e, o in zip(expect, outs):
            assert same(e, o)


def test_captured_training_step():
    """Forward and backward through autograd captured into one graph and replayed."""
    import kimi_delta_attention_20_b200 as kda
    p = call_params(50, dtype=torch.float32)
    leaves = {k: p[k].detach().clone().requires_grad_() for k in ("x", "g", "w", "cw")}

    def step():
        y, s = kda.rms_norm(leaves["x"], leaves["w"], residual=leaves["g"])
        c, _ = kda.causal_conv(y, leaves["cw"])
        h, _ = kda.chunk_gated_scan(c, leaves["g"], use_gate_sigmoid_in_kernel=True)
        return torch.autograd.grad((h * p["dy"]).sum() + s.sum(), list(leaves.values()))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    g.replay()
    torch.cuda.synchronize()
    assert same(want, got)


def test_functions_refuse():
    """What does not fit is refused by name, before anything is launched."""
    import kimi_delta_attention_20_b200 as kda
    from kimi_delta_attention_20_b200._abi import KDAError
    x, w, cw = draw(2, 6, 16), draw(16), draw(16, 4)
    bad = [
        lambda: kda.rms_norm(x.half()), lambda: kda.rms_norm(x, w[:8]), lambda: kda.rms_norm(x, w.bfloat16()),
        lambda: kda.rms_norm(x, residual=x.bfloat16()), lambda: kda.rms_norm(x, residual=x[:1]), lambda: kda.rms_norm(x, residual=x, gate=x),
        lambda: kda.rms_norm(x, gate=x.cpu()), lambda: kda.rms_norm(x.transpose(1, 2)), lambda: kda.rms_norm(x, out=x[:1]),
        lambda: kda.rms_norm(x, residual_out=x.clone()), lambda: kda.rms_norm(x[:1].expand(2, 6, 16)[:, :, ::2]),
        lambda: kda.rms_norm_quant(x, group_size=16), lambda: kda.rms_norm_quant(x, out=torch.empty_like(x)),
        lambda: kda.rms_norm_bwd(x, x[:1]), lambda: kda.rms_norm_bwd(x, x, gate=x, dresidual=x),
        lambda: kda.causal_conv(x[0], cw), lambda: kda.causal_conv(x, cw.bfloat16()), lambda: kda.causal_conv(x, cw[:8]),
        lambda: kda.causal_conv(x, cw, initial_state=torch.zeros(2, 16, 3, device=DEV)), lambda: kda.causal_conv(x, cw, cu_seqlens=torch.tensor([0, 12])),
        lambda: kda.causal_conv(x[:1], cw, cu_seqlens=torch.tensor([6])), lambda: kda.causal_conv(x[:1], cw, cu_seqlens_cpu=torch.tensor([0, 6])),
        lambda: kda.causal_conv_step(x, cw, torch.zeros(2, 16, 4, device=DEV)), lambda: kda.causal_conv_step(x[:, 0], cw, None),
        lambda: kda.chunk_gated_scan(x, x[:1]), lambda: kda.chunk_gated_scan(x, x, lower_bound=1.0),
        lambda: kda.chunk_gated_scan(x, x, lower_bound=-1.0, use_gate_sigmoid_in_kernel=True),
        lambda: kda.chunk_gated_scan(x, x, initial_state=torch.zeros(2, 16, device=DEV, dtype=torch.bfloat16)),
        lambda: kda.chunk_gated_scan_bwd(None, x, x, x, use_gate_sigmoid_in_kernel=True), lambda: kda.gated_scan_step(x, x, x),
        lambda: kda.gated_scan_step(x[:, 0], x[:, 0], None),
        lambda: kda.causal_conv(x, cw, final_state_out=torch.empty(2, 16, 4, device=DEV)),
        lambda: kda.chunk_gated_scan(x, x, final_state_out=torch.empty(2, 16, device=DEV)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("not refused:", i)
    leaf = x.clone().requires_grad_()
    with pytest.raises(NotImplementedError):
        kda.rms_norm_quant(leaf)
    for f in (lambda: kda.rms_norm(leaf, out=torch.empty_like(x)), lambda: kda.causal_conv(leaf, cw, out=torch.empty_like(x)),
              lambda: kda.chunk_gated_scan(leaf, x, final_state_out=torch.empty(2, 16, device=DEV))):
        with pytest.raises(ValueError):
            f()
    # the library's own refusals: outputs over inputs, offsets that do not fit, windows and rows out of range
    for f in (lambda: kda.rms_norm(x, out=x), lambda: kda.causal_conv(x, cw, out=x), lambda: kda.chunk_gated_scan(x, x, out=x),
              lambda: kda.causal_conv(x[:1], cw, cu_seqlens=torch.tensor([0, 5])), lambda: kda.causal_conv(x, draw(16, 9)),
              lambda: kda.rms_norm(draw(2, 20000))):
        with pytest.raises(KDAError):
            f()


@pytest.mark.parametrize("cu", [[0, 700, 300, 900, 1000], [0, -5, 2000, 100, 1000], [1000, 900, 300, 100, 0], [7, 7, 7, 7, 7]], ids=str)
@pytest.mark.parametrize("D", [40, 77, 40000])
def test_offsets_that_are_not_what_the_host_was_told(cu, D):
    """Offsets on the device may hold anything, whether the host's copy orders the work or
    none: no access leaves the buffers, and calls that follow are as they were."""
    import kimi_delta_attention_20_b200 as kda
    T, N, K = 1000, 4, 4
    host = torch.tensor([0, 240, 500, 760, 1000], dtype=torch.int32)
    good, odd = host.to(DEV), torch.tensor(cu, dtype=torch.int32, device=DEV)
    x, g, w = draw(1, T, D, dtype=torch.bfloat16, seed=1), -draw(1, T, D, dtype=torch.bfloat16, seed=2).abs(), draw(D, K, seed=3)
    s0, c0 = draw(N, D, seed=4), draw(N, D, K, seed=5)

    def run(dev, cpu):
        kw = dict(cu_seqlens=dev, cu_seqlens_cpu=cpu)
        h, f = kda.chunk_gated_scan(x, g, initial_state=s0, output_final_state=True, **kw)
        y, win = kda.causal_conv(x, w, initial_state=c0, output_final_state=True, **kw)
        return (h, f, y, win, *kda.chunk_gated_scan_bwd(None, g, h, x, initial_state=s0, dfinal_state=s0, **kw),
                *kda.causal_conv_bwd(x, w, x, initial_state=c0, dfinal_state=c0, **kw))

    want = run(good, host)
    run(odd, host)
    run(odd, None)
    torch.cuda.synchronize()
    assert same(want, run(good, host))


def test_offsets_changed_before_the_backward_are_noticed():
    import kimi_delta_attention_20_b200 as kda
    cu = torch.tensor([0, 3, 8], dtype=torch.int32, device=DEV)
    x = draw(1, 8, 16, seed=1).requires_grad_()
    for call in (lambda: kda.chunk_gated_scan(x, -x.detach().abs(), cu_seqlens=cu)[0], lambda: kda.causal_conv(x, draw(16, 4), cu_seqlens=cu)[0]):
        y = call()
        cu[1] = 4
        with pytest.raises(RuntimeError):
            y.sum().backward()


def test_elements_beyond_32_bits():
    """The last rows of tensors of over 2^31 elements, behind rows of zeros, are those of a
    call of these rows alone."""
    import kimi_delta_attention_20_b200 as kda
    T, C, K, n = 65600, 32776, 4, 5
    w, tail = draw(C, K, seed=1), draw(1, n, C, dtype=torch.bfloat16, seed=2)
    tail_g, tail_d = -draw(1, n, C, dtype=torch.bfloat16, seed=3).abs(), draw(1, n, C, dtype=torch.bfloat16, seed=4)
    x, g, d = (torch.zeros(1, T, C, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    x[:, -n:], g[:, -n:], d[:, -n:] = tail, tail_g, tail_d

    def run(x, g, d):
        h, _ = kda.chunk_gated_scan(x, g)
        outs = [h, kda.causal_conv(x, w)[0], *kda.chunk_gated_scan_bwd(None, g, h, d)[:2], kda.causal_conv_bwd(x, w, d, want_dconv_w=False)[0]]
        first = [t[:, :-n].abs().max().item() for t in outs] if x.shape[1] > n else []
        return [t[:, -n:].clone() for t in outs], first

    want, _ = run(tail, tail_g, tail_d)
    got, first = run(x, g, d)
    assert same(want, got) and first[:2] == [0.0, 0.0]


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two devices")
def test_on_another_device():
    p = call_params(60)
    want = calls(p)
    there = {k: v.to("cuda:1") for k, v in p.items()}
    got = calls(there)
    torch.cuda.synchronize(1)
    assert torch.cuda.current_device() == 0 and all(t.get_device() == 1 for t in got)
    assert same(want, [t.to("cuda:0") for t in got])
