"""Cases, plain forms and exact values of the operators around the recurrence of a layer.

Three operators, each with its backward pass and, where a serving loop needs one, its
single-token form:

  norm   root-mean-square norm: with the residual's addition, with a sigmoid output gate,
         with the output in 8 bits (e4m3) and its scales; backward
  conv   causal depthwise convolution + SiLU over packed sequences, its single token, backward
  scan   gated linear recurrence h_t = a_t h_{t-1} + x_t per channel over packed sequences,
         its single token, backward

`run` computes a pass in elementary torch operations, or with `own` set by the calls that a
user makes of the library. `exact` gives the same in 64 bits, token after token where the
operator is defined that way.
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
SCALE_FLOOR = 2.0 ** -100
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------- cases

def _norm(name, form, rows, dim, dtype="bf16", group=0, pow2=False, weight="f32"):
    return {"name": name, "op": "norm", "form": form, "rows": rows, "dim": dim, "dtype": dtype, "group": group,
            "pow2": pow2, "weight": weight}


def _conv(name, form, lens, dim, dtype="bf16", width=4, state=False):
    return {"name": name, "op": "conv", "form": form, "lens": lens, "dim": dim, "dtype": dtype, "width": width,
            "state": state}


def _scan(name, form, lens, dim, dtype="bf16", gate="log", bound=0.0, state=False):
    return {"name": name, "op": "scan", "form": form, "lens": lens, "dim": dim, "dtype": dtype, "gate": gate,
            "bound": bound, "state": state}


def listed():
    return [
        # one decode step of 64 sequences: the norm before an 8-bit projection, latency counts
        _norm("norm_quant_decode", "add_quant", 64, 2048, group=128),
        # a long prompt batch before an 8-bit projection, one scale per token
        _norm("norm_quant_prefill", "add_quant", 16384, 4096),
        # output norm of a prompt, per head: 8192 tokens x 96 heads of 128
        _norm("norm_gated_prefill", "gated", 8192 * 96, 128, weight="none"),
        # training step of the layer norm at an odd width, fp32
        _norm("norm_bwd_odd", "add_bwd", 8191, 2047, dtype="f32"),
        # output norm of a training batch, 32 x 2048 tokens x 8 heads of 64
        _norm("norm_gated_bwd", "gated_bwd", 32 * 2048 * 8, 64),
        # the q, k, v channels of 16 heads of 128 over a ragged prompt batch with carried windows
        _conv("conv_prefill", "fwd", "1,2500,63,4096,0,1532", 6144, state=True),
        # training batch 32 x 2048 of the 8-head layer (keys 32, values 64)
        _conv("conv_bwd", "bwd", "32*2048", 1024),
        # four packed long sequences at the width of 96 heads of 128
        _scan("scan_prefill", "fwd", "4096,8192,12288,7168", 12288, bound=-5.0, state=True),
        # one very long sequence with few channels, an odd number of them, fp32
        _scan("scan_long", "fwd", "131072", 257, dtype="f32"),
        # training batch at the width of 16 heads of 128, sigmoid gate
        _scan("scan_bwd", "bwd", "4*2048", 2048, gate="sigmoid"),
        # the backward of a ragged packed batch with states, odd width
        _scan("scan_bwd_ragged", "bwd", "777,1,3000,0,64,4350", 1023, bound=-5.0, state=True),
        # one decode step of 64 sequences at the width of 96 heads of 128
        _scan("scan_step", "step", "64*1", 12288, state=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(rng, most):
    """Sequence lengths with at most `most` tokens in all: one sequence, a rectangular batch, or a ragged one."""
    kind = rng.choice(("one", "batch", "ragged"))
    total = _log(rng, 1, most)
    if kind == "one":
        return str(total)
    n = min(total, _log(rng, 2, 64))
    if kind == "batch":
        return "%d*%d" % (n, max(1, total // n))
    cuts = sorted(rng.randrange(total + 1) for _ in range(n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    op = rng.choice(("norm", "conv", "scan"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if op == "norm":
        form = rng.choice(("add", "add_quant", "gated", "add_bwd", "gated_bwd"))
        dim = _log(rng, 16, 16384)
        dim = dim if rng.random() < 0.4 else max(8, dim // 8 * 8)
        rows = _log(rng, 1, max(1, min(1 << 20, (48 << 20) // dim)))
        quant = form == "add_quant"
        return _norm("", form, rows, dim, dtype, rng.choice((0, 32, 64, 128)) if quant else 0,
                     quant and rng.random() < 0.3, rng.choice(("f32", "same", "none")))
    dim = _log(rng, 16, 12288)
    dim = dim if rng.random() < 0.4 else max(4, dim // 4 * 4)
    form = rng.choice(("fwd", "fwd", "bwd", "bwd", "step"))
    if form == "step":
        lens = "%d*1" % _log(rng, 1, 256)
    else:
        lens = _lens(rng, max(1, min(131072, (48 << 20) // dim)))
    if op == "conv":
        return _conv("", form, lens, dim, dtype, rng.choice((4, 4, 4, 2, 3, 8)), rng.random() < 0.5)
    gate = rng.choice(("log", "sigmoid"))
    bound = -5.0 if gate == "log" and rng.random() < 0.5 else 0.0
    return _scan("", form, lens, dim, dtype, gate, bound, rng.random() < 0.5)


def _lengths(case):
    text = case["lens"]
    if "*" in text:
        n, t = text.split("*")
        return [int(t)] * int(n), True
    lens = [int(t) for t in text.split(",")]
    return lens, len(lens) == 1


# --------------------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dtype)

    s = dict(case)
    D = case["dim"]
    if case["op"] == "norm":
        M = case["rows"]
        s["x"] = normal(M, D)
        s["w"] = None
        if case["weight"] != "none":
            s["w"] = (1 + torch.randn(D, generator=gen, device=dev) * 0.1).to(dt if case["weight"] == "same" else torch.float32)
        if case["form"] in ("add", "add_quant"):
            s["res"] = normal(M, D)
        if case["form"] in ("gated", "gated_bwd"):
            s["gate"] = normal(M, D)
        if case["form"] in ("add_bwd", "gated_bwd"):
            s["dy"] = normal(M, D)
        if case["form"] == "add_bwd":
            s["dres"] = normal(M, D)
        return s

    lens, even = _lengths(case)
    N, T = len(lens), sum(lens)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    # the offsets on the device and their host copy, as a serving loop keeps them; None for a rectangular batch
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    s["cu_arg"], s["cu_host"] = (None, None) if even else (s["cu"], torch.tensor(cu, dtype=torch.int32))
    shape = (N, lens[0], D) if even else (1, T, D)
    if case["form"] == "step":
        shape = (N, D)
    s["x"] = normal(*shape)
    if case["op"] == "conv":
        K = case["width"]
        s["w"] = normal(D, K, dtype=torch.float32, scale=0.5)
        # windows hold past inputs, so their values are of the input's type
        s["s0"] = normal(N, D, K).float() if case["state"] or case["form"] == "step" else None
        if case["form"] == "bwd":
            s["dy"] = normal(*shape)
            s["ds"] = normal(N, D, K, dtype=torch.float32) if case["state"] else None
        return s
    if case["gate"] == "sigmoid":  # memories of a few to a few hundred tokens
        g = torch.randn(shape, generator=gen, device=dev) + torch.rand(D, generator=gen, device=dev) * 4
    else:  # log-decays -rate softplus(N(0, 1)), rates per channel over three decades
        rate = torch.exp(torch.rand(D, generator=gen, device=dev) * 6.5 - 6)
        g = -rate * torch.log1p(torch.exp(torch.randn(shape, generator=gen, device=dev)))
    s["g"] = g.to(dt)
    del g
    s["s0"] = normal(N, D, dtype=torch.float32) if case["state"] or case["form"] == "step" else None
    if case["form"] == "bwd":
        s["h"] = _plain_scan(s)[0]  # what the forward pass left behind
        s["dy"] = normal(*shape)
        s["ds"] = normal(N, D, dtype=torch.float32) if case["state"] else None
    return s


# --------------------------------------------------------------------------- plain forms

def _plain_norm(s):
    x = s["x"].float()
    dt = s["x"].dtype
    if s.get("res") is not None:
        x = x + s["res"].float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    y = x * r
    if s["w"] is not None:
        y = y * s["w"].float()
    if s["form"] == "gated":
        return (y * torch.sigmoid(s["gate"].float())).to(dt)
    if s["form"] == "add":
        return y.to(dt), x.to(dt)
    D = s["dim"]
    G = s["group"] or D
    pad = -D % G
    yg = torch.nn.functional.pad(y, (0, pad)).unflatten(-1, (-1, G))
    scale = (yg.abs().amax(-1) / E4M3_MAX).clamp_min(SCALE_FLOOR)
    if s["pow2"]:
        scale = torch.exp2(torch.ceil(torch.log2(scale)))
    q = (yg / scale[..., None]).flatten(-2)[..., :D].to(torch.float8_e4m3fn)
    return q, scale, x.to(dt)


def _plain_norm_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    dt = s["x"].dtype
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r
    nw = n if s["w"] is None else n * s["w"].float()
    gated = s["form"] == "gated_bwd"
    dgate = None
    dn = dy
    if gated:
        sg = torch.sigmoid(s["gate"].float())
        dgate = (dy * nw * sg * (1 - sg)).to(dt)
        dn = dy * sg
    dw = None
    if s["w"] is not None:
        dw = (dn * n).sum(0).to(s["w"].dtype)
        dn = dn * s["w"].float()
    dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    if not gated:
        dx = dx + s["dres"].float()
    return dx.to(dt), dgate, dw


def _rows(s):
    """Sequence of every packed token, and the number of tokens."""
    T = s["x"].numel() // s["dim"]
    t = torch.arange(T, device=s["x"].device)
    return torch.searchsorted(s["cu"][1:].long(), t, right=True), t


def _windows(s):
    """Every sequence behind its window: rows [T + N K, C], the first row of each token's window, rows of the windows."""
    K, N, D = s["width"], s["cu"].numel() - 1, s["dim"]
    seq, t = _rows(s)
    x = s["x"].float().reshape(-1, D)
    E = x.new_zeros(x.shape[0] + N * K, D)
    first = (s["cu"][:-1].long() + K * torch.arange(N, device=x.device))[:, None] + torch.arange(K, device=x.device)
    if s["s0"] is not None:
        E[first] = s["s0"].transpose(1, 2)
    E[t + (seq + 1) * K] = x
    return E, t + seq * K + 1, first, s["cu"][1:].long()[:, None] - s["cu"][:-1].long()[:, None] + first


def _plain_conv(s):
    if s["form"] == "step":
        s["s0"].copy_(torch.cat((s["s0"][..., 1:], s["x"].float()[..., None]), -1))
        z = (s["s0"] * s["w"]).sum(-1)
        return (z * torch.sigmoid(z)).to(s["x"].dtype), s["s0"]
    K = s["width"]
    E, start, _, last = _windows(s)
    z = (E.unfold(0, K, 1)[start] * s["w"]).sum(-1)
    y = (z * torch.sigmoid(z)).to(s["x"].dtype).reshape(s["x"].shape)
    return y, E[last].transpose(1, 2).contiguous()


def _plain_conv_bwd(s):
    K, D = s["width"], s["dim"]
    E, start, first, last = _windows(s)
    W = E.unfold(0, K, 1)[start]
    z = (W * s["w"]).sum(-1)
    sg = torch.sigmoid(z)
    dz = s["dy"].float().reshape(-1, D) * sg * (1 + z * (1 - sg))
    dw = (dz[..., None] * W).sum(0, dtype=torch.float64).float()  # long sums
    P = dz.new_zeros(E.shape[0] + K - 1, D)
    P[start + K - 1] = dz
    dE = (P.unfold(0, K, 1) * s["w"].flip(-1)).sum(-1)
    seq, t = _rows(s)
    if s["ds"] is not None:
        dE.index_put_((last,), s["ds"].transpose(1, 2), accumulate=True)
    dx = dE[t + (seq + 1) * K].to(s["x"].dtype).reshape(s["x"].shape)
    return dx, dw, dE[first].transpose(1, 2).contiguous() if s["s0"] is not None else None


def _halves(a, x):
    """h_t = a_t h_{t-1} + x_t along the first axis from h = 0: pairs of steps are joined, the half-length recurrence
    gives every second h, and one more step the others."""
    n = a.shape[0]
    if n <= 1:
        return x
    m = n // 2 * 2
    odd = _halves(a[0:m:2] * a[1:m:2], x[0:m:2] * a[1:m:2] + x[1:m:2])
    h = torch.empty_like(x)
    h[0] = x[0]
    h[1::2] = odd
    h[2::2] = a[2::2] * odd[: (n - 1) // 2] + x[2::2]
    return h


def _decay(s):
    g = s["g"].float().reshape(-1, s["dim"])
    if s["gate"] == "sigmoid":
        return torch.sigmoid(g)
    return torch.exp(g.clamp_min(s["bound"]) if s["bound"] else g)


def _plain_scan(s):
    D, dt = s["dim"], s["x"].dtype
    x = s["x"].float().reshape(-1, D)
    a = _decay(s)
    if s["gate"] == "sigmoid":
        x = torch.sigmoid(-s["g"].float().reshape(-1, D)) * x
    if s["form"] == "step":
        s["s0"].copy_(a * s["s0"] + x)
        return s["s0"].to(dt), s["s0"]
    lo, hi = s["cu"][:-1].long(), s["cu"][1:].long()
    full = hi > lo
    at, N = lo[full], len(lo)
    if s["s0"] is not None:
        x = x.index_add(0, at, a[at] * s["s0"][full])
    a = a.index_fill(0, at, 0.0)
    h = _halves(a, x)
    fin = s["s0"].clone() if s["s0"] is not None else h.new_zeros(N, D)
    fin[full] = h[hi[full] - 1]
    return h.to(dt).reshape(s["x"].shape), fin


def _plain_scan_bwd(s):
    D, dt = s["dim"], s["x"].dtype
    a = _decay(s)
    h = s["h"].float().reshape(-1, D)
    d = s["dy"].float().reshape(-1, D)
    lo, hi = s["cu"][:-1].long(), s["cu"][1:].long()
    full = hi > lo
    first, last = lo[full], hi[full] - 1
    if s["ds"] is not None:
        d = d.index_add(0, last, s["ds"][full])
    # the cotangent runs backwards: d_t += a_{t+1} d_{t+1} inside a sequence
    nxt = torch.cat((a[1:], a[:1])).index_fill(0, last, 0.0)
    d = _halves(nxt.flip(0), d.flip(0)).flip(0)
    prev = torch.cat((h[:1], h[:-1]))
    prev[first] = s["s0"][full] if s["s0"] is not None else 0.0
    d0 = None
    if s["s0"] is not None:
        d0 = s["ds"].clone() if s["ds"] is not None else torch.zeros_like(s["s0"])
        d0[full] = a[first] * d[first]
    if s["gate"] == "sigmoid":
        b = torch.sigmoid(-s["g"].float().reshape(-1, D))
        dx = b * d
        dg = d * (prev - s["x"].float().reshape(-1, D)) * a * b
    else:
        dx = d
        dg = d * a * prev
        if s["bound"]:
            dg = dg * (s["g"].float().reshape(-1, D) >= s["bound"])
    return dx.to(dt).reshape(s["x"].shape), dg.to(dt).reshape(s["x"].shape), d0


# --------------------------------------------------------------------------- one pass

def run(s):
    if own:
        return _own(s)
    if s["op"] == "norm":
        return _plain_norm_bwd(s) if s["form"].endswith("bwd") else _plain_norm(s)
    if s["op"] == "conv":
        return _plain_conv_bwd(s) if s["form"] == "bwd" else _plain_conv(s)
    return _plain_scan_bwd(s) if s["form"] == "bwd" else _plain_scan(s)


def _own(s):
    import kimi_delta_attention_20_b200 as kda

    op, form = s["op"], s["form"]
    if op == "norm":
        if form == "add":
            return kda.rms_norm(s["x"], s["w"], residual=s["res"], eps=EPS)
        if form == "add_quant":
            return kda.rms_norm_quant(s["x"], s["w"], residual=s["res"], eps=EPS, group_size=s["group"],
                                      pow2_scales=s["pow2"])
        if form == "gated":
            return kda.rms_norm(s["x"], s["w"], gate=s["gate"], eps=EPS)
        return kda.rms_norm_bwd(s["x"], s["dy"], s["w"], gate=s.get("gate"), dresidual=s.get("dres"), eps=EPS)
    if op == "conv":
        if form == "step":
            return kda.causal_conv_step(s["x"], s["w"], s["s0"]), s["s0"]
        kw = dict(initial_state=s["s0"], cu_seqlens=s["cu_arg"], cu_seqlens_cpu=s["cu_host"])
        if form == "fwd":
            return kda.causal_conv(s["x"], s["w"], output_final_state=True, **kw)
        return kda.causal_conv_bwd(s["x"], s["w"], s["dy"], dfinal_state=s["ds"], **kw)
    kw = dict(use_gate_sigmoid_in_kernel=s["gate"] == "sigmoid", lower_bound=s["bound"] or None)
    if form == "step":
        return kda.gated_scan_step(s["x"], s["g"], s["s0"], **kw), s["s0"]
    kw |= dict(initial_state=s["s0"], cu_seqlens=s["cu_arg"], cu_seqlens_cpu=s["cu_host"])
    if form == "fwd":
        return kda.chunk_gated_scan(s["x"], s["g"], output_final_state=True, **kw)
    return kda.chunk_gated_scan_bwd(s["x"], s["g"], s["h"], s["dy"], dfinal_state=s["ds"], **kw)


# --------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    esz = 2 if case["dtype"] == "bf16" else 4
    D, form = case["dim"], case["form"]
    if case["op"] == "norm":
        el = case["rows"] * D
        wb = 0 if case["weight"] == "none" else D * (esz if case["weight"] == "same" else 4)
        groups = case["rows"] * -(-D // (case["group"] or D))
        by = {"add": 4 * esz * el + wb, "add_quant": (3 * esz + 1) * el + 4 * groups + wb, "gated": 3 * esz * el + wb,
              "add_bwd": 4 * esz * el + 2 * wb, "gated_bwd": 5 * esz * el + 2 * wb}[form]
        return {"bytes": by, "flops": el * (14 if form.endswith("bwd") else 8)}
    lens, _ = _lengths(case)
    N, T = len(lens), sum(lens)
    el = T * D
    st = 4 * N * D
    if case["op"] == "conv":
        K = case["width"]
        st *= K
        w = 4 * D * K
        if form == "step":
            return {"bytes": 2 * esz * el + 2 * st + w, "flops": el * (2 * K + 6)}
        if form == "fwd":
            return {"bytes": 2 * esz * el + w + st * (2 if case["state"] else 1), "flops": el * (2 * K + 6)}
        return {"bytes": 3 * esz * el + 2 * w + st * (3 if case["state"] else 0), "flops": el * (6 * K + 12)}
    if form == "step":
        return {"bytes": 3 * esz * el + 2 * st, "flops": el * 8}
    if form == "fwd":
        return {"bytes": 3 * esz * el + st * (2 if case["state"] else 1), "flops": el * 8}
    tensors = 6 if case["gate"] == "sigmoid" else 5  # the sigmoid form reads x too
    return {"bytes": tensors * esz * el + st * (3 if case["state"] else 0), "flops": el * 12}


# --------------------------------------------------------------------------- 64 bits

def _round_e4m3(v):
    """The nearest value of e4m3 (4 exponent bits, bias 7, 3 mantissa bits, at most 448), ties to even."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -20))).clamp_min(-6.0)
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_norm(s):
    x = s["x"].double()
    w = torch.ones((), dtype=torch.float64, device=x.device) if s["w"] is None else s["w"].double()
    form = s["form"]
    if form in ("add", "add_quant"):
        x = x + s["res"].double()
    ms = x.square().sum(-1, keepdim=True) / s["dim"] + EPS
    if form == "gated":
        return x * w / (ms.sqrt() * (1 + torch.exp(-s["gate"].double())))
    if form == "add":
        return x * w / ms.sqrt(), x
    if form == "add_quant":
        y = x * w / ms.sqrt()
        qs, scales = [], []
        for part in y.split(s["group"] or s["dim"], -1):
            sc = (part.abs().max(-1, keepdim=True).values / E4M3_MAX).clamp_min(SCALE_FLOOR)
            if s["pow2"]:
                m, e = torch.frexp(sc)  # sc = m 2^e, m in [1/2, 1)
                sc = torch.exp2((e - (m == 0.5).to(e.dtype)).double())
            scales.append(sc)
            qs.append(_round_e4m3(part / sc))
        return torch.cat(qs, -1), torch.cat(scales, -1), x
    # gradients: y_i = x_i w_i p_i / sqrt(ms), d ms / d x_j = 2 x_j / D
    dy = s["dy"].double()
    p = torch.ones_like(x) if form == "add_bwd" else 1 / (1 + torch.exp(-s["gate"].double()))
    root = ms.sqrt()
    inner = (dy * w * p * x).sum(-1, keepdim=True)
    dx = dy * w * p / root - x * inner / (s["dim"] * ms * root)
    if form == "add_bwd":
        dx = dx + s["dres"].double()
    dgate = None if form == "add_bwd" else dy * x * w / root * p * (1 - p)
    return dx, dgate, None if s["w"] is None else (dy * x * p / root).sum(0)


def _spans(case):
    """(first token, length, sequences) of each run of sequences that can be walked side by side."""
    lens, even = _lengths(case)
    if even:
        return [(0, lens[0], len(lens))]
    at, spans = 0, []
    for n in lens:
        spans.append((at, n, 1))
        at += n
    return spans


def _exact_conv(s, case):
    D, K, form = s["dim"], s["width"], s["form"]
    w = s["w"].double()
    x = s["x"].double().reshape(-1, D)
    N = len(_lengths(case)[0])
    s0 = torch.zeros(N, D, K, dtype=torch.float64, device=x.device) if s["s0"] is None else s["s0"].double()
    ys, fins, dxs, d0s = [], [], [], []
    dw = torch.zeros_like(w)
    n0 = 0
    for at, T, B in _spans(case):
        hist = torch.cat((s0[n0:n0 + B].transpose(1, 2), x[at:at + T * B].reshape(B, T, D)), 1)  # [B, K + T, D]
        z = torch.zeros(B, T, D, dtype=torch.float64, device=x.device)
        for i in range(K):
            z += hist[:, 1 + i:1 + i + T] * w[:, i]
        sg = 1 / (1 + torch.exp(-z))
        if form != "bwd":
            ys.append((z * sg).reshape(-1, D))
            fins.append(hist[:, T:].transpose(1, 2))
        else:
            dz = s["dy"].double().reshape(-1, D)[at:at + T * B].reshape(B, T, D) * (sg + z * sg * (1 - sg))
            dh = torch.zeros_like(hist)
            for i in range(K):
                dh[:, 1 + i:1 + i + T] += dz * w[:, i]
                dw[:, i] += (dz * hist[:, 1 + i:1 + i + T]).sum((0, 1))
            if s["ds"] is not None:
                dh[:, T:] += s["ds"][n0:n0 + B].double().transpose(1, 2)
            dxs.append(dh[:, K:].reshape(-1, D))
            d0s.append(dh[:, :K].transpose(1, 2))
        n0 += B
    if form == "bwd":
        return torch.cat(dxs).reshape(s["x"].shape), dw, torch.cat(d0s) if s["s0"] is not None else None
    return torch.cat(ys).reshape(s["x"].shape), torch.cat(fins)


def _exact_scan(s, case):
    D, form = s["dim"], s["form"]
    g = s["g"].reshape(-1, D)
    x = s["x"].reshape(-1, D)
    N = len(_lengths(case)[0])
    s0 = torch.zeros(N, D, dtype=torch.float64, device=x.device) if s["s0"] is None else s["s0"].double()

    def gate(rows):  # a, and the weight of x
        v = rows.double()
        if s["gate"] == "sigmoid":
            return 1 / (1 + torch.exp(-v)), 1 / (1 + torch.exp(v))
        return torch.exp(torch.clamp(v, min=s["bound"]) if s["bound"] else v), None

    outs, fins, n0 = [], [], 0
    dgs, d0s = [], []
    for at, T, B in _spans(case):
        gs, xs = (v[at:at + T * B].reshape(B, T, D).transpose(0, 1) for v in (g, x))
        if form != "bwd":
            h, o = s0[n0:n0 + B].clone(), torch.empty(T, B, D, dtype=torch.float64, device=x.device)
            for t0 in range(0, T, 4096):  # stretches, so that the 64-bit copies stay small
                a, b = gate(gs[t0:t0 + 4096])
                v = xs[t0:t0 + 4096].double() if b is None else b * xs[t0:t0 + 4096].double()
                for i in range(a.shape[0]):
                    torch.addcmul(v[i], a[i], h, out=o[t0 + i])
                    h = o[t0 + i]
            outs.append(o.transpose(0, 1).reshape(-1, D))
            fins.append(h.clone())
        else:
            dy = s["dy"].reshape(-1, D)[at:at + T * B].reshape(B, T, D).transpose(0, 1).double()
            hs = s["h"].reshape(-1, D)[at:at + T * B].reshape(B, T, D).transpose(0, 1).double()
            a, b = gate(gs)
            c = torch.zeros(B, D, dtype=torch.float64, device=x.device) if s["ds"] is None else s["ds"][n0:n0 + B].double()
            d = torch.empty_like(dy)
            for t in range(T - 1, -1, -1):
                torch.add(dy[t], c, out=d[t])
                c = a[t] * d[t]
            prev = torch.cat((s0[n0:n0 + B][None], hs[:-1])) if T else hs
            if s["gate"] == "sigmoid":
                dx, dg = b * d, d * (prev - xs.double()) * a * b
            else:
                dx, dg = d, d * prev * a
                if s["bound"]:
                    dg = torch.where(gs.double() < s["bound"], torch.zeros_like(dg), dg)
            outs.append(dx.transpose(0, 1).reshape(-1, D))
            dgs.append(dg.transpose(0, 1).reshape(-1, D))
            d0s.append(c)
        n0 += B
    if form == "bwd":
        return (torch.cat(outs).reshape(s["x"].shape), torch.cat(dgs).reshape(s["x"].shape),
                torch.cat(d0s) if s["s0"] is not None else None)
    return torch.cat(outs).reshape(s["x"].shape), torch.cat(fins)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "conv":
        return _exact_conv(s, case)
    return _exact_scan(s, case)
