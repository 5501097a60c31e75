"""Plain 64-bit forms of the operators around the state update (RMS norm, causal
convolution, gated scan), token after token, and bounds on what fp32 arithmetic and the
rounding of the outputs may be off from them.

u = 2^-24 is half a step of fp32; `half(dtype)` half a step of an output type, relative.
The bounds count roundings: a sum of n products held in fp32 is off by at most
(n + 1) u times the sum of the products' magnitudes, CUDA's expf by 2 steps (4 u), a
division, root or product by 1 u each.
"""
import torch

U = 2.0 ** -24


def half(dtype):
    return torch.finfo(dtype).eps / 2


def bounds_of(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def within(name, got, want, tol):
    """Every element of got is within tol (elementwise) of want; what is not finite agrees."""
    got, want = got.double(), want.double()
    assert got.shape == want.shape, f"{name}: {tuple(got.shape)} and {tuple(want.shape)}"
    if not got.numel():
        return
    tol = torch.as_tensor(tol, dtype=torch.float64, device=got.device).expand_as(want)
    off = (got - want).abs()
    bad = ~(off <= tol)
    if bad.any():
        i = int((off / tol.clamp_min(1e-300)).nan_to_num(nan=1e300, posinf=1e300).argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off; at {i}: {got.flatten()[i].item():.9g}, "
                             f"want {want.flatten()[i].item():.9g}, tolerance {tol.flatten()[i].item():.3g}")


# --------------------------------------------------------------------------- RMS norm

def norm(x, weight=None, residual=None, gate=None, eps=1e-6):
    """(y, s) in 64 bits."""
    s = x.double()
    if residual is not None:
        s = s + residual.double()
    y = s / (s.square().mean(-1, keepdim=True) + eps).sqrt()
    if weight is not None:
        y = y * weight.double()
    if gate is not None:
        y = y * torch.sigmoid(gate.double())
    return y, s


def norm_rel(D):
    """What fp32 leaves of y, relative: each thread sums at most 32 squares and the row's
    threads are joined by a tree and at most 16 more terms, so the sum of squares is off by
    at most (32 + 5 + 16 + 1) u (its root by half of that); the sum x + residual, the mean,
    the added eps, the root, the reciprocal, two products, expf, its sum and a quotient
    follow. For bf16 the gate's exponential is the SFU's, 2^(-gate log2 e): off by 4 u and, from
    the rounding of its argument, 2 |gate| u, where |gate| stays below 10."""
    return 27 * U + 14 * U + 24 * U


def norm_grads(x, dy, weight=None, gate=None, dresidual=None, eps=1e-6):
    """(dx, dgate, dweight) from the written-out derivative, in 64 bits."""
    s, d = x.double(), dy.double()
    D = s.shape[-1]
    w = torch.ones((), dtype=torch.float64, device=s.device) if weight is None else weight.double()
    p = torch.ones_like(s) if gate is None else torch.sigmoid(gate.double())
    r = 1 / (s.square().mean(-1, keepdim=True) + eps).sqrt()
    u = d * w * p
    dx = r * (u - s * r * r * (u * s).sum(-1, keepdim=True) / D)
    mag = r * (u.abs() + s.abs() * r * r * (u * s).abs().sum(-1, keepdim=True) / D)
    if dresidual is not None:
        dx = dx + dresidual.double()
        mag = mag + dresidual.double().abs()
    dgate = None if gate is None else d * s * r * w * p * (1 - p)
    flat = (d * s * r * p).reshape(-1, D)
    return dx, dgate, flat.sum(0), mag, flat.abs().sum(0)


# --------------------------------------------------------------------------- causal convolution

def conv(x, w, lens, s0=None):
    """(y [T, C], final windows [N, C, K], z, sum |w in|) of packed rows x [T, C], 64 bits."""
    x, w = x.double(), w.double()
    C, K = w.shape
    ys, zs, mags, fins = [], [], [], []
    at = 0
    for n, T in enumerate(lens):
        win = torch.zeros(K, C, dtype=torch.float64, device=x.device) if s0 is None else s0[n].double().t()
        rows = torch.cat((win, x[at:at + T]))
        z = sum((rows[1 + k:1 + k + T] * w[:, k] for k in range(K)), torch.zeros(T, C, dtype=torch.float64, device=x.device))
        mags.append(sum((rows[1 + k:1 + k + T].abs() * w[:, k].abs() for k in range(K)), torch.zeros_like(z)))
        zs.append(z)
        ys.append(z * torch.sigmoid(z))
        fins.append(rows[T:].t())
        at += T
    return torch.cat(ys), torch.stack(fins), torch.cat(zs), torch.cat(mags)


# --------------------------------------------------------------------------- gated scan

def decay(g, sigmoid, lower_bound):
    g = g.double()
    if sigmoid:
        return torch.sigmoid(g), torch.sigmoid(-g)
    if lower_bound is not None:
        g = g.clamp_min(lower_bound)
    return torch.exp(g), torch.ones_like(g)


def decay_rel(g):
    """What fp32 leaves of a and of 1 - a, relative: expf is off by 4 u; the SFU's exponential,
    taken for bf16, by 4 u and 2 |g| u from the rounding of its argument g log2 e. A sum, a
    quotient, the weighting of x and the product of a run's a follow (8 u)."""
    return (12 + 2 * g.double().abs()) * U


def scan(x, g, lens, s0=None, sigmoid=False, lower_bound=None):
    """(h [T, D], final states [N, D], bound on h's fp32 error, the same of the states)."""
    a, b = decay(g, sigmoid, lower_bound)
    k = decay_rel(g)
    v = b * x.double()
    D = x.shape[1]
    hs, es, fins, fes = [], [], [], []
    at = 0
    for n, T in enumerate(lens):
        h = torch.zeros(D, dtype=torch.float64, device=x.device) if s0 is None else s0[n].double()
        m, e = h.abs(), torch.zeros_like(h)
        for t in range(at, at + T):
            e = a[t] * (e + k[t] * m) + k[t] * v[t].abs()
            h = a[t] * h + v[t]
            m = a[t] * m + v[t].abs()
            e = e + 2 * U * m
            hs.append(h)
            es.append(e)
        fins.append(h)
        fes.append(e)
        at += T
    empty = x.new_zeros(0, D, dtype=torch.float64)
    return (torch.stack(hs) if hs else empty, torch.stack(fins), torch.stack(es) if es else empty, torch.stack(fes))


def scan_grads(x, g, h, dout, lens, s0=None, dsT=None, sigmoid=False, lower_bound=None):
    """(dx, dg, ds0) from the written-out derivative with h as given, and bounds on the fp32
    error of each."""
    a, b = decay(g, sigmoid, lower_bound)
    r = decay_rel(g)
    T_, D = g.shape
    dx, dg, ex, eg = (torch.zeros(T_, D, dtype=torch.float64, device=g.device) for _ in range(4))
    d0, e0 = [], []
    at = 0
    for n, T in enumerate(lens):
        c = torch.zeros(D, dtype=torch.float64, device=g.device) if dsT is None else dsT[n].double()
        m, e = c.abs(), torch.zeros_like(c)
        for t in range(at + T - 1, at - 1, -1):
            d = dout[t].double() + c
            m = dout[t].double().abs() + m
            e = e + 2 * U * m
            if t > at:
                hp = h[t - 1].double()
            else:
                hp = torch.zeros_like(c) if s0 is None else s0[n].double()
            k = hp - x[t].double() if sigmoid else hp
            km = hp.abs() + x[t].double().abs() if sigmoid else hp.abs()
            dx[t] = b[t] * d
            ex[t] = b[t] * (e + r[t] * m)
            dg[t] = d * a[t] * b[t] * k
            eg[t] = a[t] * b[t] * km * (e + 2 * r[t] * m + 4 * U * m)
            if lower_bound is not None:
                below = g[t].double() < lower_bound
                dg[t][below] = 0
            c = a[t] * d
            e = a[t] * (e + r[t] * m)
            m = a[t] * m
        d0.append(c)
        e0.append(e)
        at += T
    return dx, dg, torch.stack(d0), ex, eg, torch.stack(e0)
