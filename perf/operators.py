"""Cases for the per-head-decay linear attention and the query/key norm with position rotation:
their inputs, their plain forms in elementary torch operations and their definitions in 64 bits.

Linear attention with one decay a token and head (the state is dk x dv for each sequence and head):
    S_t = e^{g_t} S_{t-1} + k_t v_t^T        o_t = S_t^T q_t
"fwd" is a whole packed batch of prompts, "bwd" its gradients, "step" one token of many requests
whose states live in a pool.  "norm" is the RMS norm of every query and key head followed by the
rotation of its first channels by the token's position, "norm_bwd" its gradients.

own = False computes the plain forms; own = True calls the library's entry points.
"""
import math
import random

import torch

own = False

CHUNK = 128  # tokens a chunk of the plain form


# ------------------------------------------------------------------ cases --

def _lengths(seed, n, lo, hi):
    r = random.Random(seed)
    return ",".join(str(int(round(math.exp(r.uniform(math.log(lo), math.log(hi))))))
                    for _ in range(n))


def listed():
    return [
        # prefill of one long document: the state is carried over 65,536 tokens, 32 chains only
        dict(name="fwd_long_prompt", op="fwd", lengths="65536", H=32, dk=128, dv=128,
             dtype="bf16", per_token=True, state=False, fused=False),
        # prefill of a batch of requests of very different lengths that continue cached states,
        # the values still a view of the fused projection's output
        dict(name="fwd_packed_prompts", op="fwd", lengths=_lengths(5, 24, 16, 8192), H=16, dk=128,
             dv=128, dtype="bf16", per_token=True, state=True, fused=True),
        # a few short chat turns of a small model: latency
        dict(name="fwd_short_turns", op="fwd", lengths="1,37,150,64", H=4, dk=64, dv=64,
             dtype="bf16", per_token=True, state=True, fused=False),
        # evaluation in fp32 with one fixed decay for each head
        dict(name="fwd_f32_fixed_decay", op="fwd", lengths="2048,1531", H=8, dk=64, dv=128,
             dtype="f32", per_token=False, state=True, fused=False),
        # training on one long document
        dict(name="bwd_long_document", op="bwd", lengths="65536", H=16, dk=128, dv=128,
             dtype="bf16", per_token=True, state=False, fused=False),
        # training on packed documents, the states passed on from an earlier segment
        dict(name="bwd_packed_documents", op="bwd", lengths="700,1,2049,96,1300", H=8, dk=128,
             dv=64, dtype="bf16", per_token=True, state=True, fused=False),
        # a decode step of a full batch: states in a pool, a few rows of the batch unused
        dict(name="step_full_batch", op="step", N=256, pool=320, unused=3, H=32, dk=128, dv=128,
             dtype="bf16", per_token=True, fused=True),
        # a decode step of a few requests: latency
        dict(name="step_few", op="step", N=3, pool=8, unused=0, H=16, dk=128, dv=128,
             dtype="bf16", per_token=True, fused=False),
        # norm and rotation of a prompt's queries and (fewer) keys, read from the fused projection
        dict(name="norm_prompt", op="norm", T=65536, Hq=32, Hk=8, d=128, rot=128,
             interleaved=False, dtype="bf16", weight=True, fused=True),
        # the same for a decode step's batch, half of the channels rotated, pairs side by side
        dict(name="norm_step", op="norm", T=64, Hq=32, Hk=8, d=128, rot=64, interleaved=True,
             dtype="bf16", weight=True, fused=True),
        # its gradients in training, as many key heads as query heads
        dict(name="norm_bwd_document", op="norm_bwd", T=32768, Hq=16, Hk=16, d=128, rot=64,
             interleaved=False, dtype="bf16", weight=True, fused=False),
        # a small model's gradients in fp32 at an odd length
        dict(name="norm_bwd_f32", op="norm_bwd", T=4097, Hq=8, Hk=2, d=64, rot=64,
             interleaved=True, dtype="f32", weight=True, fused=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_lengths(rng, tokens, most):
    n = _log_int(rng, 1, most)
    cuts = sorted(rng.randint(0, tokens) for _ in range(n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [tokens]))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "norm", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("fwd", "bwd"):
        H = rng.choice([1, 2, 4, 5, 8, 16, 32])
        most = ((1 << 21) if op == "fwd" else (1 << 20)) // H
        if dtype == "f32":
            most //= 16
        return dict(op=op, lengths=_draw_lengths(rng, _log_int(rng, 1, min(65536, most)), 24),
                    H=H, dk=rng.choice([64, 128]), dv=rng.choice([64, 128]), dtype=dtype,
                    per_token=rng.random() < 0.7, state=rng.random() < 0.6,
                    fused=rng.random() < 0.4)
    if op == "step":
        N, H = _log_int(rng, 1, 256), rng.choice([2, 8, 12, 16, 32])
        return dict(op=op, N=N, pool=N + rng.randint(0, 64), unused=rng.randint(0, N // 4), H=H,
                    dk=rng.choice([64, 128]), dv=rng.choice([64, 128]), dtype=dtype,
                    per_token=rng.random() < 0.7, fused=rng.random() < 0.4)
    d = rng.choice([64, 128])
    Hq = rng.choice([1, 4, 8, 16, 32])
    Hk = rng.choice([h for h in (1, 2, 4, 8, 16, 32) if h <= Hq])
    return dict(op=op, T=_log_int(rng, 1, 65536 if op == "norm" else 16384), Hq=Hq, Hk=Hk, d=d,
                rot=rng.choice([0, 32, d // 2, d]), interleaved=rng.random() < 0.5, dtype=dtype,
                weight=rng.random() < 0.8, fused=rng.random() < 0.5)


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] in ("fwd", "bwd"):
        lens = [int(x) for x in c["lengths"].split(",")]
        T, N, H, dk, dv = sum(lens), len(lens), c["H"], c["dk"], c["dv"]
        g = 4 * H * (T if c["per_token"] else 1)
        S = 4 * N * H * dk * dv
        if c["op"] == "fwd":
            return dict(bytes=T * H * (2 * dk + 2 * dv) * e + g + S * (2 if c["state"] else 1),
                        flops=4.0 * T * H * dk * dv)
        return dict(bytes=T * H * (4 * dk + 3 * dv) * e + 2 * g + S * (3 if c["state"] else 0),
                    flops=10.0 * T * H * dk * dv)
    if c["op"] == "step":
        n, H, dk, dv = c["N"] - c["unused"], c["H"], c["dk"], c["dv"]
        return dict(bytes=n * H * (8 * dk * dv + (2 * dk + 2 * dv) * e + 4),
                    flops=5.0 * n * H * dk * dv)
    rows = c["T"] * (c["Hq"] + c["Hk"])
    if c["op"] == "norm":
        return dict(bytes=rows * c["d"] * e * 2 + 4 * c["T"], flops=8.0 * rows * c["d"])
    return dict(bytes=rows * c["d"] * e * 3 + 4 * c["T"], flops=16.0 * rows * c["d"])


# ----------------------------------------------------------------- inputs --

def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32

    def normal(*shape, dtype=torch.float32, scale=1.0):
        x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
        return x.mul_(scale).to(dtype)

    s = dict(case=dict(c))
    if c["op"] in ("fwd", "bwd", "step"):
        H, dk, dv = c["H"], c["dk"], c["dv"]
        if c["op"] == "step":
            T = c["N"]
        else:
            s["lengths"] = [int(x) for x in c["lengths"].split(",")]
            T = sum(s["lengths"])
            cu = [0]
            for n in s["lengths"]:
                cu.append(cu[-1] + n)
            s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")

        def unit(x):  # heads of length 1, as the norm in front of the attention leaves them
            return (x / x.float().norm(dim=-1, keepdim=True)).to(dt)

        s["q"], s["k"] = unit(normal(T, H, dk)), unit(normal(T, H, dk))
        if c["fused"]:  # the values stay a view of the projection's output
            s["v"] = normal(T, H * (2 * dk + dv), dtype=dt)[:, 2 * H * dk:].unflatten(1, (H, dv))
        else:
            s["v"] = normal(T, H, dv, dtype=dt)
        # decays with time constants from about two tokens to some hundreds, head by head
        slope = torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H)
        s["g"] = (-slope * torch.nn.functional.softplus(normal(T, H)) if c["per_token"] else -slope)
        if c["op"] == "step":
            s["S"] = normal(c["pool"], H, dk, dv, scale=0.1)
            slots = torch.randperm(c["pool"], generator=gen, device="cuda")[:T].to(torch.int32)
            at = torch.randperm(T, generator=gen, device="cuda")[:c["unused"]]
            slots[at] = -1
            s["slots"] = slots
        else:
            N = len(s["lengths"])
            s["S0"] = normal(N, H, dk, dv, scale=0.1) if c["state"] else None
            if c["op"] == "bwd":
                s["do"] = normal(T, H, dv, dtype=dt)
                s["dS"] = normal(N, H, dk, dv, scale=0.1) if c["state"] else None
        return s

    T, Hq, Hk, d, rot = c["T"], c["Hq"], c["Hk"], c["d"], c["rot"]
    if c["fused"]:  # queries, keys and values side by side, as one projection writes them
        x = normal(T, (Hq + 2 * Hk) * d, dtype=dt, scale=2.0)
        s["q"] = x[:, :Hq * d].unflatten(1, (Hq, d))
        s["k"] = x[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d))
    else:
        s["q"], s["k"] = (normal(T, h, d, dtype=dt, scale=2.0) for h in (Hq, Hk))
    s["wq"], s["wk"] = ((normal(d, scale=0.2).add_(1.0) for _ in range(2)) if c["weight"]
                        else (None, None))
    P = 65536
    s["pos"] = torch.randint(0, P, (T,), generator=gen, device="cuda", dtype=torch.int32)
    if rot:
        f = torch.exp(torch.arange(rot // 2, device="cuda", dtype=torch.float64)
                      * (-2.0 * math.log(1e4) / rot))
        a = torch.arange(P, device="cuda", dtype=torch.float64)[:, None] * f
        s["cos_sin"] = torch.cat([a.cos(), a.sin()], 1).float()
    else:
        s["cos_sin"] = None
    if c["op"] == "norm_bwd":
        s["dyq"], s["dyk"] = normal(T, Hq, d, dtype=dt), normal(T, Hk, d, dtype=dt)
    return s


# ------------------------------------------------------------ plain forms --

def _segments(x):
    """[..., n] -> [..., n, n]: the sum of x over (j, i], for i >= j (a running sum of its own
    for every j, so that nothing large cancels)."""
    n = x.shape[-1]
    low = torch.ones(n, n, dtype=torch.bool, device=x.device).tril(-1)
    return torch.where(low, x[..., :, None], 0.0).cumsum(-2)


def _plain_linear(q, k, v, g, S0, lengths):
    """o and the final states, chunk by chunk: products inside a chunk, the chunks' contributions
    to the states, and the states at the chunk starts as sums over the earlier chunks."""
    T, H, dk = q.shape
    dv, N, dev = v.shape[2], len(lengths), q.device
    q, k, v = q.float(), k.float(), v.float()
    g = g.float().expand(T, H)
    count = [-(-n // CHUNK) for n in lengths]
    NC = sum(count)
    ln = torch.tensor(lengths, device=dev)
    nc = torch.tensor(count, device=dev)
    seq = torch.repeat_interleave(torch.arange(N, device=dev), nc, output_size=NC)
    first = nc.cumsum(0) - nc
    row = (torch.arange(NC, device=dev) - first[seq])[:, None] * CHUNK + torch.arange(CHUNK,
                                                                                      device=dev)
    at = torch.where(row < ln[seq][:, None], row + (ln.cumsum(0) - ln)[seq][:, None], T)

    def chunks(x):  # [T, H, ...] -> [H, NC, CHUNK, ...], zeros past the sequence's end
        return torch.cat([x, x.new_zeros(1, *x.shape[1:])])[at].movedim(2, 0)

    Q, K, V, G = chunks(q), chunks(k), chunks(v), chunks(g)
    pair = _segments(G)                                             # [H, NC, C, C]
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    A = (Q @ K.transpose(-1, -2)) * torch.where(low, pair, -math.inf).exp()
    add = (K * pair[:, :, -1, :, None].exp()).transpose(-1, -2) @ V  # [H, NC, dk, dv]
    head = G.cumsum(-1)
    whole = head[:, :, -1]                                          # [H, NC]
    same = seq[:, None] == seq[None, :]
    before = same & torch.ones(NC, NC, dtype=torch.bool, device=dev).tril(-1)
    run = _segments(whole)                                          # (j, i], i >= j
    upto = torch.cat([torch.zeros_like(run[:, :1]), run[:, :-1]], 1)  # (j, i - 1]
    W = torch.where(before, upto, -math.inf).exp()
    start = (W @ add.flatten(2)).unflatten(2, (dk, dv))             # [H, NC, dk, dv]
    since = (before * whole[:, None, :]).sum(-1)                    # decay since the sequence began
    if S0 is not None:
        start = start + since.exp()[:, :, None, None] * S0.float().movedim(1, 0)[:, seq]
    o = A @ V + head.exp()[..., None] * (Q @ start)
    o = o.movedim(0, 2)[row < ln[seq][:, None]]                     # [T, H, dv]
    last = (first + nc - 1).clamp(min=0)
    end = whole.exp()[:, last, None, None] * start[:, last] + add[:, last]
    empty = (nc == 0)[:, None, None, None]
    S_out = torch.where(empty, 0.0 if S0 is None else S0.float(), end.movedim(0, 1))
    return o, S_out


def _plain_fwd(s):
    o, S = _plain_linear(s["q"], s["k"], s["v"], s["g"], s["S0"], s["lengths"])
    return dict(o=o.to(s["q"].dtype), S=S)


def _plain_bwd(s):
    """Gradients by differentiating the plain forward's elementary operations."""
    leaf = {n: s[n].detach().float().requires_grad_(True) for n in ("q", "k", "v", "g")}
    S0 = s["S0"]
    if S0 is not None:
        leaf["S0"] = S0 = S0.detach().clone().requires_grad_(True)
    o, S = _plain_linear(leaf["q"], leaf["k"], leaf["v"], leaf["g"], S0, s["lengths"])
    if s["dS"] is not None:
        torch.autograd.backward([o, S], [s["do"].float(), s["dS"]])
    else:
        o.backward(s["do"].float())
    dt = s["q"].dtype
    out = {"d" + n: leaf[n].grad.to(dt) for n in ("q", "k", "v")}
    out["dg"] = leaf["g"].grad
    if S0 is not None:
        out["dS0"] = S0.grad
    return out


def _plain_step(s):
    used = s["slots"] >= 0
    at = s["slots"].clamp(min=0).long()
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    g = s["g"].expand(q.shape[:2])
    S = g.exp()[..., None, None] * s["S"][at] + k[..., :, None] * v[..., None, :]
    o = (S * q[..., :, None]).sum(-2)
    s["S"][at[used]] = S[used]
    return dict(o=torch.where(used[:, None, None], o, 0.0).to(s["q"].dtype), S=s["S"])


def _pairs(x, rot, interleaved):
    """The two members of every rotated pair, and the channels that stay as they are."""
    r = x[..., :rot]
    if interleaved:
        return r[..., 0::2], r[..., 1::2], x[..., rot:]
    return r[..., :rot // 2], r[..., rot // 2:], x[..., rot:]


def _join(a, b, rest, interleaved):
    r = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1)


def _turn(x, s, sign):
    c = s["case"]
    if not c["rot"]:
        return x
    cs = s["cos_sin"].to(x.dtype)[s["pos"].long()][:, None, :]
    cos, sin = cs[..., :c["rot"] // 2], cs[..., c["rot"] // 2:] * sign
    a, b, rest = _pairs(x, c["rot"], c["interleaved"])
    return _join(a * cos - b * sin, a * sin + b * cos, rest, c["interleaved"])


EPS = 1e-6


def _normed(x, w):
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    return r, x * r, 1.0 if w is None else w


def _plain_norm(s):
    def one(n):
        _, hat, w = _normed(s[n].float(), s["w" + n])
        return _turn(hat * w, s, 1.0).to(s[n].dtype)

    return dict(q=one("q"), k=one("k"))


def _plain_norm_bwd(s):
    def one(n):
        r, hat, w = _normed(s[n].float(), s["w" + n])
        dy = _turn(s["dy" + n].float(), s, -1.0)
        out = {} if s["w" + n] is None else {"dw" + n: (dy * hat).sum((0, 1))}
        dy = dy * w
        dx = r * (dy - hat * (dy * hat).mean(-1, keepdim=True))
        return {**out, "d" + n: dx.to(s[n].dtype)}

    return {**one("q"), **one("k")}


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "norm": _plain_norm,
                "norm_bwd": _plain_norm_bwd}[op](s)
    from serving_kda_chunkwise_gb300 import kda
    if op == "fwd":
        o, S = kda.linear_fwd_chunked(s["q"], s["k"], s["v"], s["g"], S0=s["S0"],
                                      cu_seqlens=s["cu"])
        return dict(o=o, S=S)
    if op == "bwd":
        out = kda.linear_bwd(s["q"], s["k"], s["v"], s["g"], s["do"], S0=s["S0"], dS_out=s["dS"],
                             cu_seqlens=s["cu"], want_dS0=s["S0"] is not None)
        return {n: x for n, x in out.items() if x is not None}
    if op == "step":
        o = kda.linear_decode_step(s["q"], s["k"], s["v"], s["g"], s["S"], slots=s["slots"])
        return dict(o=o, S=s["S"])
    c = s["case"]
    if op == "norm":
        q, k = kda.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], eps=EPS, cos_sin=s["cos_sin"],
                                positions=s["pos"], interleaved=c["interleaved"])
        return dict(q=q, k=k)
    out = kda.qk_norm_rope_bwd(s["q"], s["k"], s["dyq"], s["dyk"], s["wq"], s["wk"], eps=EPS,
                               cos_sin=s["cos_sin"], positions=s["pos"],
                               interleaved=c["interleaved"])
    return {n: x for n, x in out.items() if x is not None}


def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""

    def by_length(lengths):
        """Sequences from the longest to the shortest, their first rows, and how many are longer
        than t for every t."""
        order = sorted(range(len(lengths)), key=lambda n: -lengths[n])
        first = [0]
        for n in lengths:
            first.append(first[-1] + n)
        active, m = [], len(order)
        for t in range(lengths[order[0]]):
            while lengths[order[m - 1]] <= t:
                m -= 1
            active.append(m)
        return order, torch.tensor([first[n] for n in order], device="cuda"), active

    def linear(s):
        """The recurrence token by token, and for the gradients its reverse."""
        c = s["case"]
        q, k, v = (s[n].double() for n in ("q", "k", "v"))
        T, H, dk = q.shape
        dv, N = v.shape[2], len(s["lengths"])
        g = s["g"].double().expand(T, H)
        a = g.exp()
        order, first, active = by_length(s["lengths"])
        back = torch.tensor(order, device="cuda")
        S = torch.zeros(N, H, dk, dv, dtype=torch.float64, device="cuda")
        if s["S0"] is not None:
            S += s["S0"].double()[back]
        do = s["do"].double() if c["op"] == "bwd" else None
        o, dq = torch.zeros_like(v), torch.zeros_like(q)
        for t, m in enumerate(active):
            at = first[:m] + t
            Sm = S[:m].mul_(a[at][:, :, None, None])
            Sm.add_(k[at][..., :, None] * v[at][..., None, :])
            if do is None:
                o[at] = (q[at][..., None, :] @ Sm)[..., 0, :]
            else:
                dq[at] = (Sm @ do[at][..., :, None])[..., 0]
        end = torch.empty_like(S)
        end[back] = S
        if do is None:
            return dict(o=o, S=end)
        D = torch.zeros_like(S)
        if s["dS"] is not None:
            D += s["dS"].double()[back]
            anchor = (S * D).sum((-1, -2))
        else:
            anchor = torch.zeros(N, H, dtype=torch.float64, device="cuda")
        dkk, dvv = torch.zeros_like(k), torch.zeros_like(v)
        for t in range(len(active) - 1, -1, -1):
            m = active[t]
            at = first[:m] + t
            Dm = D[:m]
            Dm.add_(q[at][..., :, None] * do[at][..., None, :])
            dkk[at] = (Dm @ v[at][..., :, None])[..., 0]
            dvv[at] = (k[at][..., None, :] @ Dm)[..., 0, :]
            Dm.mul_(a[at][:, :, None, None])
        # the loss depends on g_t through everything that crosses from before t to t or later
        each = (q * dq).sum(-1) - (k * dkk).sum(-1)
        dg = torch.empty_like(each)
        for i, n in enumerate(order):
            b = int(first[i])
            x = each[b:b + s["lengths"][n]]
            dg[b:b + s["lengths"][n]] = x.flip(0).cumsum(0).flip(0) + anchor[i]
        out = dict(dq=dq, dk=dkk, dv=dvv, dg=dg if c["per_token"] else dg.sum(0))
        if s["S0"] is not None:
            dS0 = torch.empty_like(D)
            dS0[back] = D
            out["dS0"] = dS0
        return out

    def step(s):
        S = s["S"].double()
        o = torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
        g = s["g"].double().expand(s["q"].shape[:2])
        for i, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                S[slot] = (S[slot] * g[i].exp()[:, None, None]
                           + torch.einsum("hk,hv->hkv", s["k"][i].double(), s["v"][i].double()))
                o[i] = torch.einsum("hk,hkv->hv", s["q"][i].double(), S[slot])
        return dict(o=o, S=S)

    def rotation(s):
        """The rotation of every token as a d x d matrix."""
        c = s["case"]
        d, rot = c["d"], c["rot"]
        R = torch.eye(d, dtype=torch.float64, device="cuda").repeat(c["T"], 1, 1)
        for p in range(rot // 2):
            i, j = (2 * p, 2 * p + 1) if c["interleaved"] else (p, p + rot // 2)
            cos = s["cos_sin"][s["pos"].long(), p].double()
            sin = s["cos_sin"][s["pos"].long(), rot // 2 + p].double()
            R[:, i, i], R[:, i, j], R[:, j, i], R[:, j, j] = cos, -sin, sin, cos
        return R

    def norm(s):
        """y = R diag(w) x / rms(x); its transposed derivative for the gradients."""
        c = s["case"]
        R, out = rotation(s), {}
        one = torch.ones(c["d"], dtype=torch.float64, device="cuda")
        for n in ("q", "k"):
            x = s[n].double()
            w = one if s["w" + n] is None else s["w" + n].double()
            rms = (x.square().sum(-1, keepdim=True) / c["d"] + EPS).sqrt()
            if c["op"] == "norm":
                out[n] = torch.einsum("tij,thj->thi", R, w * x / rms)
                continue
            u = torch.einsum("tij,thi->thj", R, s["dy" + n].double())
            if s["w" + n] is not None:
                out["dw" + n] = torch.einsum("thj,thj->j", u, x / rms)
            dot = (u * w * x).sum(-1, keepdim=True)
            out["d" + n] = u * w / rms - x * dot / (c["d"] * rms ** 3)
        return out

    c = case
    if "T" in c and c["T"] * c["d"] ** 2 * 8 > 12e9:
        return None
    s = prepare(case, seed)
    if c["op"] in ("fwd", "bwd"):
        return linear(s)
    return step(s) if c["op"] == "step" else norm(s)
