"""The per-head-decay linear attention and the query/key norm with rotation in 64 bits, from
their definitions, for the GPU tests (torch, any device)."""
import torch


def forward(q, k, v, g, S0, lengths):
    """o [T, H, dv] and the final states [N, H, dk, dv], token by token."""
    q, k, v = q.double(), k.double(), v.double()
    T, H, dk = q.shape
    a = g.double().expand(T, H).exp()
    o = torch.zeros_like(v)
    ends, t = [], 0
    for n, ln in enumerate(lengths):
        S = torch.zeros(H, dk, v.shape[2], dtype=torch.float64, device=q.device)
        if S0 is not None:
            S = S + S0[n].double()
        for t in range(t, t + ln) if ln else ():
            S = a[t][:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
            o[t] = torch.einsum("hk,hkv->hv", q[t], S)
        t = t + 1 if ln else t
        ends.append(S)
    return o, torch.stack(ends)


def gradients(q, k, v, g, do, S0, dS, lengths):
    """dq, dk, dv, dg, dS0 by the recurrence and its reverse; the decay's gradient from
    <dL/dS_t, e^{g_t} S_{t-1}>."""
    q, k, v, do = q.double(), k.double(), v.double(), do.double()
    T, H, dk = q.shape
    dv = v.shape[2]
    a = g.double().expand(T, H).exp()
    out = dict(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v),
               dg=torch.zeros(T, H, dtype=torch.float64, device=q.device))
    dS0, first = [], 0
    for n, ln in enumerate(lengths):
        S = torch.zeros(H, dk, dv, dtype=torch.float64, device=q.device)
        if S0 is not None:
            S = S + S0[n].double()
        decayed = []
        for t in range(first, first + ln):
            S = a[t][:, None, None] * S
            decayed.append(S)
            S = S + k[t][:, :, None] * v[t][:, None, :]
            out["dq"][t] = torch.einsum("hkv,hv->hk", S, do[t])
        D = torch.zeros_like(S) if dS is None else dS[n].double().clone()
        for t in range(first + ln - 1, first - 1, -1):
            D = D + q[t][:, :, None] * do[t][:, None, :]
            out["dk"][t] = torch.einsum("hkv,hv->hk", D, v[t])
            out["dv"][t] = torch.einsum("hkv,hk->hv", D, k[t])
            out["dg"][t] = (D * decayed[t - first]).sum((-1, -2))
            D = a[t][:, None, None] * D
        dS0.append(D)
        first += ln
    out["dS0"] = torch.stack(dS0)
    if g.dim() == 1:
        out["dg"] = out["dg"].sum(0)
    return out


def rotation(cos_sin, pos, d, interleaved):
    """[T, d, d] rotation matrices."""
    T, rot = pos.numel(), 0 if cos_sin is None else cos_sin.shape[1]
    R = torch.eye(d, dtype=torch.float64, device=pos.device).repeat(T, 1, 1)
    for p in range(rot // 2):
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + rot // 2)
        c, s = cos_sin[pos.long(), p].double(), cos_sin[pos.long(), rot // 2 + p].double()
        R[:, i, i], R[:, i, j], R[:, j, i], R[:, j, j] = c, -s, s, c
    return R


def norm(x, w, eps, R):
    x = x.double()
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    if w is not None:
        y = y * w.double()
    return torch.einsum("tij,thj->thi", R, y)


def norm_gradients(x, dy, w, eps, R):
    """dx and dw by differentiating norm() in 64 bits."""
    x = x.double().requires_grad_(True)
    w = (torch.ones(x.shape[-1], device=x.device) if w is None else w).double().detach().clone()
    w.requires_grad_(True)
    norm(x, w, eps, R).backward(dy.double())
    return x.grad, w.grad
