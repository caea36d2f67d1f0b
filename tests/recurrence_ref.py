"""The gated channel recurrence, the 8-bit checkpoints and the norms around a block in 64 bits, from
their definitions, and how far an fp32 computation of the recurrence may be off (torch, any device).

Bounds of the recurrence.  An exponential or reciprocal is off by 2^-22 relative, and the exponent
e^A z by 2^-22 |e^A z|, so a gate's value by eps = 2^-22 (6 + |e^A z| + |i|); e^g - 1 and the input
term by eps relative too.  A token multiplies, adds and rounds the state: 2^-22 of the states before
and after it, products of several decays included.  Errors decay as the state does:
    E_t = e^{g_t} E_{t-1} + eps (|e^{g_t} - 1| |h_{t-1}| + |b_t|) + 2^-22 (|h_t| + |h_{t-1}|)
and the same backwards for l_t = dL/dh_t.  The gradients multiply a handful of such factors (4 eps
relative of each product's terms).  Where 1 - e^{2g} is below 1e-37, next to fp32's smallest normal
number 1.2e-38, its root m is taken as zero; so is a gate's value below 2^-126, where 1 - e^{2g} is
below 2 |g_min| 2^-126 (1.2e-37 for g_min = -5).  So m is off by at most the root of the larger of the
two, which every product with m (or with g / m, which is -m / 2 there) inherits.
e^g is one plus e^g - 1, off by 2^-24 too: within eps of itself down to e^-5, so for g_min >= -5.
"""
import torch

ULP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative


def _ranges(lengths):
    first = 0
    for n, ln in enumerate(lengths):
        yield n, first, first + ln
        first += ln


def recurrence(x, z, i, A, g_min, h0, lengths, dy=None, dh=None):
    """dict of (value, bound before its rounding) pairs: y, h, edges and, with dy, dx, dz, di, dA,
    dh0."""
    x, z, i, A = x.double(), z.double(), i.double(), A.double()
    T, D = x.shape
    N = len(lengths)
    rate = A.exp()
    u = rate * z
    sz, oz, si, oi = u.sigmoid(), (-u).sigmoid(), i.sigmoid(), (-i).sigmoid()
    g = g_min * sz
    a, c = g.exp(), torch.expm1(g)
    m = (-torch.expm1(2 * g)).sqrt()
    b = torch.where(m > 0, m * si * x, 0.0)
    eps = 2.0 ** -22 * (6 + u.abs().clamp(max=200) + i.abs().clamp(max=200))
    floor = max(1e-37, -2 * g_min * 2.0 ** -126) ** 0.5
    low = floor * torch.where(m > 0, (si * x).abs(), 0.0)
    zero = torch.zeros(N, D, dtype=torch.float64, device=x.device)
    h0 = zero if h0 is None else h0.double()
    h, before, E = torch.empty_like(x), torch.empty_like(x), torch.zeros_like(x)
    end, end_E = h0.clone(), zero.clone()
    for n, f, e in _ranges(lengths):
        s, err = h0[n], zero[n]
        for t in range(f, e):
            before[t] = s
            s = a[t] * s + b[t]
            err = a[t] * err + eps[t] * (c[t].abs() * before[t].abs() + b[t].abs()) + 2.0 ** -22 * (
                s.abs() + before[t].abs()) + low[t]
            h[t], E[t] = s, err
        end[n], end_E[n] = s, err
    before_E = torch.cat([torch.zeros_like(E[:1]), E[:-1]])
    out = dict(y=(h, E), h=(end, end_E), edges=(before[::8], before_E[::8]))
    if dy is None:
        return out
    dy = dy.double()
    dh = zero if dh is None else dh.double()
    lam, L = torch.empty_like(x), torch.empty_like(x)
    dh0, dh0_E = torch.empty_like(zero), zero.clone()
    for n, f, e in _ranges(lengths):
        s, err = dh[n], zero[n]
        for t in range(e - 1, f - 1, -1):
            was = s
            s = s + dy[t]
            err = err + 2.0 ** -22 * (s.abs() + was.abs())
            lam[t], L[t] = s, err
            s = a[t] * s
            err = a[t] * err + (eps[t] * c[t].abs() + 2.0 ** -22) * lam[t].abs()
        dh0[n], dh0_E[n] = s, err
    inv = torch.where(m > 0, 1 / m, 0.0)
    f = m * si
    out["dx"] = (lam * f, L * f + 4 * eps * (lam * f).abs() + floor * si * lam.abs())
    f = torch.where(m > 0, m * si * x * oi, 0.0)
    out["di"] = (lam * f, (L + 4 * eps * lam.abs()) * f.abs() + low * oi * lam.abs())
    k = rate * oz * g * a
    v = torch.where(m > 0, a * inv * si * x, 0.0)
    size = before.abs() + v.abs()
    dz = lam * k * (before - v)
    E_dz = k.abs() * (L * size + lam.abs() * (before_E + 6 * eps * size)) + (
        rate * oz * low * lam.abs())
    out["dz"] = (dz, E_dz)
    zz = torch.where(z.isinf(), 0.0, z)
    out["dA"] = ((dz * zz).sum(0), ((E_dz + (T / 64 + 80) * 2.0 ** -24 * dz.abs()) * zz.abs()).sum(0))
    out["dh0"] = (dh0, dh0_E)
    return out


def near(got, pair, name):
    """Within the bound and, for a rounded result, half a step of its type."""
    ref, E = pair
    if ref.numel() == 0:
        return
    d = (got.double() - ref).abs()
    tol = E * 1.01 + ULP[got.dtype] * (ref.abs() + E) + 1e-30
    worst = float((d - tol).max())
    assert bool((d <= tol).all()), (name, worst, float(d.max()))


def pack(x):
    """Codes [T, D] and exponents [groups, T] by trial of every exponent."""
    x = x.double()
    T, D = x.shape
    codes = torch.zeros(T, D, dtype=torch.int8, device=x.device)
    exps = torch.zeros(-(-D // 64), T, dtype=torch.int8, device=x.device)
    for j in range(exps.shape[0]):
        v = x[:, 64 * j:64 * j + 64]
        top = v.abs().amax(1)
        e = torch.full((T,), 121.0, dtype=torch.float64, device=x.device)
        for k in range(120, -128, -1):
            e = torch.where(top * 2.0 ** -k < 127.5, float(k), e)
        bad = ~torch.isfinite(v).all(1)
        q = (v * torch.exp2(-e)[:, None]).round().clamp(-127, 127)
        codes[:, 64 * j:64 * j + 64] = torch.where(bad[:, None], 0.0, q).to(torch.int8)
        exps[j] = torch.where(bad, -128.0, e).to(torch.int8)
    return codes, exps


def unpack(codes, exps):
    e = exps.double().t().repeat_interleave(64, dim=1)[:, :codes.shape[1]]
    v = codes.double() * torch.exp2(e)
    return torch.where(e == -128, float("nan"), v)


def block_norm(y, r, gate, scale, w_post, w_pre, post, eps):
    y, r = y.double(), r.double()

    def rms(t):
        return (t.square().mean(-1, keepdim=True) + eps).sqrt()

    n = y / rms(y) if post else y
    for w in (w_post, scale):
        n = n if w is None else n * w.double()
    n = n if gate is None else n * gate.double().sigmoid()
    r = r + n
    x = r / rms(r)
    return r, x if w_pre is None else x * w_pre.double()


def block_norm_gradients(y, r_out, dx, dr, gate, scale, w_post, w_pre, post, eps):
    """By differentiating the two halves in 64 bits: x' from r_out, and r' - r from y."""
    def leaf(t):
        return None if t is None else t.double().detach().clone().requires_grad_(True)

    ro, wp = leaf(r_out), leaf(w_pre)
    zero = torch.zeros_like(r_out, dtype=torch.float64)
    _, x = block_norm(zero, ro, None, None, None, wp, False, eps)
    out = {}
    grads = torch.autograd.grad(x, [t for t in (ro, wp) if t is not None], dx.double())
    G = grads[0] + (0.0 if dr is None else dr.double())
    out["dr"], out["dw_pre"] = G, grads[1] if wp is not None else None
    names = ["y", "gate", "scale", "w_post"]
    leaves = [leaf(t) for t in (y, gate, scale, w_post)]
    added, _ = block_norm(leaves[0], zero, *leaves[1:], None, post, eps)
    used = [(n, t) for n, t in zip(names, leaves) if t is not None]
    for (n, _), t in zip(used, torch.autograd.grad(added, [t for _, t in used], G)):
        out["d" + n] = t
    return {n: out.get(n) for n in ("dr", "dy", "dgate", "dscale", "dw_post", "dw_pre")}
