"""Cases for the gated recurrence of single channels, the 8-bit checkpoints of its inputs and the
norms around a block: their inputs, their plain forms in elementary torch operations and their
definitions in 64 bits.

Recurrence, per sequence and channel c, with s the logistic function (the state is one number):
    g_t = g_min s(e^{A_c} z_t)      h_t = e^{g_t} h_{t-1} + sqrt(1 - e^{2 g_t}) s(i_t) x_t
"fwd" is a packed batch of prompts, "train" a forward followed by its gradients, "bwd" the gradients
alone, "bwd8" the gradients from inputs that were kept in 8 bits, "step" one token of many requests
whose states live in a pool.
Checkpoints: 64 channels of a token share the smallest exponent e with max |x| 2^-e < 127.5, and
each is kept as the integer next to x 2^-e.  "keep" packs an activation and brings it back.
Norms around a block with output y and residual r:
    r' = r + scale s(gate) (w_post y / rms(y))      x' = w_pre r' / rms(r')
"norm" computes both, "norm_bwd" their gradients.

own = False computes the plain forms; own = True calls the library's entry points.
"""
import math
import random

import torch

own = False

G_MIN = -5.0
EPS = 1e-6
GROUP = 64  # channels that share an exponent


# ------------------------------------------------------------------ cases --

def _lengths(seed, n, lo, hi):
    r = random.Random(seed)
    return ",".join(str(int(round(math.exp(r.uniform(math.log(lo), math.log(hi))))))
                    for _ in range(n))


def listed():
    return [
        # prefill of one long document: every channel's state is carried over 65,536 tokens
        dict(name="fwd_long_prompt", op="fwd", lengths="65536", D=4096, dtype="bf16", state=False,
             fused=False),
        # prefill of a batch of requests of very different lengths that continue cached states,
        # the inputs still views of the fused projection's output
        dict(name="fwd_packed_prompts", op="fwd", lengths=_lengths(5, 24, 16, 8192), D=2560,
             dtype="bf16", state=True, fused=True),
        # a few short chat turns of a small model: latency
        dict(name="fwd_short_turns", op="fwd", lengths="1,37,150,64", D=1024, dtype="bf16",
             state=True, fused=False),
        # a training step's recurrence on one long document, forward and gradients
        dict(name="train_long_document", op="train", lengths="32768", D=4096, dtype="bf16",
             state=False, fused=False),
        # gradients on packed documents in fp32, the states passed on from an earlier segment
        dict(name="bwd_packed_f32", op="bwd", lengths="700,1,2049,96,1300", D=1000, dtype="f32",
             state=True, fused=False),
        # gradients of a long document whose activations were kept in 8 bits
        dict(name="bwd_checkpoints", op="bwd8", lengths="65536", D=2048, dtype="bf16",
             state=False, fused=False),
        # keeping a long document's activation in 8 bits, and bringing it back
        dict(name="keep_document", op="keep", T=65536, D=4096, dtype="bf16", fused=False),
        # a decode step of a full batch: states in a pool, a few rows of the batch unused
        dict(name="step_full_batch", op="step", N=256, pool=320, unused=3, D=4096, dtype="bf16",
             fused=True),
        # between two blocks of a prompt: post-norm, gate, residual, the next block's norm
        dict(name="norm_prompt", op="norm", T=32768, D=4096, dtype="bf16", residual="bf16",
             post=True, gate=True, scale=True),
        # the same in a decode step, without a gate
        dict(name="norm_step", op="norm", T=64, D=4096, dtype="bf16", residual="bf16", post=True,
             gate=False, scale=True),
        # its gradients in training, the residual stream held in fp32
        dict(name="norm_bwd_document", op="norm_bwd", T=32768, D=4096, dtype="bf16",
             residual="f32", post=True, gate=True, scale=True),
        # a small model's gradients in fp32 at an odd length, only the next block's norm
        dict(name="norm_bwd_f32", op="norm_bwd", T=4097, D=1000, dtype="f32", residual="f32",
             post=False, gate=False, scale=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_lengths(rng, tokens, most):
    n = _log_int(rng, 1, most)
    cuts = sorted(rng.randint(0, tokens) for _ in range(n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [tokens]))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "train", "bwd", "bwd8", "keep", "step", "norm", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    half = 1 if dtype == "bf16" else 2
    D = 8 * _log_int(rng, 8, 512)
    if op in ("fwd", "train", "bwd", "bwd8"):
        most = (1 << (27 if op == "fwd" else 26)) // (D * half)
        return dict(op=op, lengths=_draw_lengths(rng, _log_int(rng, 1, min(65536, most)), 40),
                    D=D, dtype=dtype, state=rng.random() < 0.6,
                    fused=op != "bwd8" and rng.random() < 0.4)
    if op == "keep":
        return dict(op=op, T=_log_int(rng, 1, min(65536, (1 << 27) // (D * half))), D=D,
                    dtype=dtype, fused=rng.random() < 0.4)
    if op == "step":
        N = _log_int(rng, 1, 512)
        return dict(op=op, N=N, pool=N + rng.randint(0, 64), unused=rng.randint(0, N // 4), D=D,
                    dtype=dtype, fused=rng.random() < 0.4)
    D = 8 * _log_int(rng, 8, 1024)
    return dict(op=op, T=_log_int(rng, 1, min(65536, (1 << 26) // (D * half))), D=D, dtype=dtype,
                residual="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]),
                post=rng.random() < 0.7, gate=rng.random() < 0.6, scale=rng.random() < 0.6)


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    D = c["D"]
    if "lengths" in c:
        lens = [int(x) for x in c["lengths"].split(",")]
        n, h = sum(lens) * D, 4 * len(lens) * D * (1 if c["state"] else 0)
        out = 4 * len(lens) * D
        if c["op"] == "fwd":
            return dict(bytes=4 * n * e + h + out, flops=16.0 * n)
        if c["op"] == "train":  # the inputs are read by the forward and by the gradients
            return dict(bytes=11 * n * e + 4 * h + out, flops=48.0 * n)
        if c["op"] == "bwd":
            return dict(bytes=7 * n * e + 3 * h, flops=32.0 * n)
        return dict(bytes=n * (4 * e + 3) + 3 * n // GROUP + 3 * h, flops=32.0 * n)
    if c["op"] == "keep":
        n = c["T"] * D
        return dict(bytes=n * (2 * e + 2) + 2 * n // GROUP, flops=4.0 * n)
    if c["op"] == "step":
        n = (c["N"] - c["unused"]) * D
        return dict(bytes=n * (4 * e + 8), flops=16.0 * n)
    n, r, g = c["T"] * D, 4 if c["residual"] == "f32" else 2, 1 if c["gate"] else 0
    if c["op"] == "norm":
        return dict(bytes=n * (e * (2 + g) + 2 * r), flops=12.0 * n)
    # without a post-norm, gate and scale the block's output is not read
    y = 1 if c["post"] or c["gate"] or c["scale"] else 0
    return dict(bytes=n * (e * (2 + y + 2 * g) + 3 * r), flops=30.0 * n)


# ----------------------------------------------------------------- inputs --

def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    D = c["D"]

    def normal(*shape, dtype=torch.float32, scale=1.0):
        x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
        return x.mul_(scale).to(dtype)

    s = dict(case=dict(c))
    if c["op"] in ("norm", "norm_bwd"):
        T = c["T"]
        rt = torch.bfloat16 if c["residual"] == "bf16" else torch.float32
        s["y"], s["r"] = normal(T, D, dtype=dt), normal(T, D, dtype=rt, scale=4.0)
        s["gate"] = normal(T, D, dtype=dt, scale=2.0) if c["gate"] else None
        s["scale"] = normal(D, scale=0.1).add_(0.5) if c["scale"] else None
        s["w_post"] = normal(D, scale=0.2).add_(1.0) if c["post"] else None
        s["w_pre"] = normal(D, scale=0.2).add_(1.0)
        if c["op"] == "norm_bwd":
            s["dx"], s["dr"] = normal(T, D, dtype=dt), normal(T, D, dtype=rt)
        return s

    if c["op"] in ("keep", "step"):
        T = c["T"] if c["op"] == "keep" else c["N"]
    else:
        s["lengths"] = [int(x) for x in c["lengths"].split(",")]
        T = sum(s["lengths"])
        cu = [0]
        for n in s["lengths"]:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    if c["op"] == "keep":
        # an activation whose channels differ in size, as they do in earnest
        size = normal(D).exp_()
        x = normal(T, 3 * D if c["fused"] else D).mul_(size.repeat(3) if c["fused"] else size)
        s["x"] = x.to(dt)[:, D:2 * D] if c["fused"] else x.to(dt)
        return s
    # decays with time constants from a token to some thousands, channel by channel
    level = torch.rand(D, generator=gen, device="cuda") * 7.0 - 8.0
    s["A"] = normal(D, scale=0.2)
    if c["fused"]:  # the three side by side, as one projection writes them
        x = normal(T, 3 * D, scale=1.0)
        x[:, D:2 * D].add_(level)
        x = x.to(dt)
        s["x"], s["z"], s["i"] = x[:, :D], x[:, D:2 * D], x[:, 2 * D:]
    else:
        s["x"], s["i"] = normal(T, D, dtype=dt), normal(T, D, dtype=dt)
        s["z"] = normal(T, D).add_(level).to(dt)
    if c["op"] == "step":
        s["h"] = normal(c["pool"], D)
        slots = torch.randperm(c["pool"], generator=gen, device="cuda")[:T].to(torch.int32)
        slots[torch.randperm(T, generator=gen, device="cuda")[:c["unused"]]] = -1
        s["slots"] = slots
        return s
    N = len(s["lengths"])
    s["h0"] = normal(N, D) if c["state"] else None
    if c["op"] != "fwd":
        s["dy"] = normal(T, D, dtype=dt)
        s["dh"] = normal(N, D) if c["state"] else None
    if c["op"] == "bwd8":  # what the forward pass kept
        for n in ("x", "z", "i"):
            s[n] = _plain_pack(s[n])
    return s


# ------------------------------------------------------------ plain forms --

def _plain_pack(x):
    """Codes [T, D] and exponents [groups, T] of an activation."""
    T, D = x.shape
    groups = -(-D // GROUP)
    v = torch.nn.functional.pad(x.float(), (0, groups * GROUP - D)).view(T, groups, GROUP)
    top = v.abs().amax(-1)
    m, k = torch.frexp(top)                  # top = m 2^k with m in [1/2, 1)
    e = torch.where(m * 128.0 < 127.5, k - 7, k - 6)
    e = torch.where(top > 0, e, -127).clamp(-127, 121)
    # (in 64 bits: 2^127 times a small number is exact there)
    q = torch.round(v.double() * torch.exp2(-e.double())[..., None]).clamp(-127, 127)
    codes = q.view(T, groups * GROUP)[:, :D].to(torch.int8)
    return codes, e.to(torch.int8).t().contiguous()


def _plain_unpack(packed):
    codes, e = packed
    per = torch.repeat_interleave(torch.exp2(e.double()), GROUP, dim=0)[:codes.shape[1]].t()
    return (codes.double() * per).float()


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t over the first axis, from h = 0: inside pieces of about sqrt(T)
    tokens, then over the pieces."""
    T, D = b.shape
    C = max(1, int(math.isqrt(T)))
    n = -(-T // C)
    pad = (0, 0, 0, n * C - T)
    A = torch.nn.functional.pad(a, pad, value=1.0).view(n, C, D)
    H = torch.nn.functional.pad(b, pad).view(n, C, D).clone()
    P = A.clone()
    for t in range(1, C):
        H[:, t].addcmul_(A[:, t], H[:, t - 1])
        P[:, t].mul_(P[:, t - 1])
    start = torch.zeros(n, D, dtype=b.dtype, device=b.device)
    for j in range(1, n):
        torch.addcmul(H[j - 1, -1], P[j - 1, -1], start[j - 1], out=start[j])
    return H.addcmul_(P, start[:, None]).view(n * C, D)[:T]


def _logistic(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _places(s):
    """First and last rows of the sequences that have tokens, and which those are."""
    dev = s["A"].device
    ln = torch.tensor(s["lengths"], device=dev)
    some = (ln > 0).nonzero()[:, 0]
    end = ln.cumsum(0)
    return (end - ln)[some], end[some] - 1, some


def _gates(x, z, i, A):
    """In 64 bits: a decay next to one is rounded by as much as it differs from one over a long
    memory, and the sums run over as many tokens."""
    x, z, i = x.double(), z.double(), i.double()
    rate = torch.exp(A.double())
    sz, si = _logistic(rate * z), _logistic(i)
    g = G_MIN * sz
    return rate, sz, si * x, si, g, torch.exp(g), torch.sqrt(-torch.expm1(2.0 * g))


def _states(s, a, b):
    """h_t of every token and h_{t-1}."""
    first, last, some = _places(s)
    h0 = (a.new_zeros(len(s["lengths"]), a.shape[1]) if s["h0"] is None else s["h0"].double())
    a0, b0 = a.clone(), b.clone()
    a0[first] = 0.0
    b0[first] = b[first] + a[first] * h0[some]
    h = _scan(a0, b0)
    before = torch.cat([h[:1], h[:-1]])
    before[first] = h0[some]
    end = h0.clone()
    end[some] = h[last]
    return h, before, end


def _plain_fwd(s):
    _, _, u, _, _, a, m = _gates(s["x"], s["z"], s["i"], s["A"])
    h, _, end = _states(s, a, m * u)
    return dict(y=h.to(s["x"].dtype), h=end.float())


def _plain_bwd(s, x, z, i):
    rate, sz, u, si, g, a, m = _gates(x, z, i, s["A"])
    _, before, _ = _states(s, a, m * u)
    first, last, some = _places(s)
    dy = s["dy"].double()
    if s["dh"] is not None:
        dy[last] += s["dh"][some]
    after = torch.cat([a[1:], torch.zeros_like(a[:1])])   # the next token's decay
    after[last] = 0.0
    lam = _scan(after.flip(0), dy.flip(0)).flip(0)
    dg = lam * (a * before - a * a / m * u)
    dz = dg * g * (1.0 - sz) * rate
    dt = s["dy"].dtype
    out = dict(dx=(lam * m * si).to(dt), dz=dz.to(dt), di=(lam * m * u * (1.0 - si)).to(dt),
               dA=(dz * z).sum(0).float())
    if s["h0"] is not None:
        dh0 = torch.zeros_like(s["h0"]) if s["dh"] is None else s["dh"].clone()
        dh0[some] = (a[first] * lam[first]).float()
        out["dh0"] = dh0
    return out


def _plain_step(s):
    used = s["slots"] >= 0
    at = s["slots"].clamp(min=0).long()
    _, _, u, _, _, a, m = _gates(s["x"], s["z"], s["i"], s["A"])
    h = a * s["h"][at] + m * u
    s["h"][at[used]] = h[used].float()
    return dict(y=torch.where(used[:, None], h, 0.0).to(s["x"].dtype), h=s["h"])


def _rms(x):
    return torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)


def _branch(s, y):
    """What the block adds to the residual: (its value, the factor of n, n, y / rms(y))."""
    hat = y / _rms(y) if s["case"]["post"] else y
    n = hat if s["w_post"] is None else hat * s["w_post"]
    f = torch.ones_like(y)
    if s["gate"] is not None:
        f = f * _logistic(s["gate"].float())
    if s["scale"] is not None:
        f = f * s["scale"]
    return f * n, f, n, hat


def _plain_norm(s):
    r = s["r"].float() + _branch(s, s["y"].float())[0]
    return dict(r=r.to(s["r"].dtype), x=(r / _rms(r) * s["w_pre"]).to(s["y"].dtype))


def _plain_norm_bwd(s):
    """s["r"] is the residual after the block, as the forward left it."""
    y, r, dx = s["y"].float(), s["r"].float(), s["dx"].float()
    hat = r / _rms(r)
    u = dx * s["w_pre"]
    G = s["dr"].float() + (u - hat * (u * hat).mean(-1, keepdim=True)) / _rms(r)
    _, f, n, yhat = _branch(s, y)
    dt = s["y"].dtype
    out = dict(dr=G.to(s["r"].dtype), dw_pre=(dx * hat).sum(0))
    if s["scale"] is not None:
        gate = 1.0 if s["gate"] is None else _logistic(s["gate"].float())
        out["dscale"] = (G * gate * n).sum(0)
    if s["gate"] is not None:
        out["dgate"] = (G * f * n * (1.0 - _logistic(s["gate"].float()))).to(dt)
    dn = G * f
    if s["w_post"] is not None:
        out["dw_post"] = (dn * yhat).sum(0)
        dn = dn * s["w_post"]
    if s["case"]["post"]:
        dn = (dn - yhat * (dn * yhat).mean(-1, keepdim=True)) / _rms(y)
    return dict(out, dy=dn.to(dt))


def _plain(s):
    op = s["case"]["op"]
    if op == "fwd":
        return _plain_fwd(s)
    if op == "train":
        return dict(_plain_fwd(s), **_plain_bwd(s, s["x"], s["z"], s["i"]))
    if op == "bwd":
        return _plain_bwd(s, s["x"], s["z"], s["i"])
    if op == "bwd8":
        return _plain_bwd(s, *(_plain_unpack(s[n]) for n in ("x", "z", "i")))
    if op == "keep":
        return dict(x=_plain_unpack(_plain_pack(s["x"])).to(s["x"].dtype))
    return {"step": _plain_step, "norm": _plain_norm, "norm_bwd": _plain_norm_bwd}[op](s)


def run(state):
    s = state
    if not own:
        return _plain(s)
    from serving_kda_chunkwise_gb300 import kda
    op = s["case"]["op"]
    if op in ("fwd", "train", "bwd", "bwd8"):
        gates = (s["x"], s["z"], s["i"], s["A"], G_MIN)
        out, edges = {}, None
        if op == "fwd":
            y, h = kda.recurrence_fwd(*gates, h0=s["h0"], cu_seqlens=s["cu"])
            return dict(y=y, h=h)
        if op == "train":
            edges = kda.recurrence_edges(s["x"])
            out["y"], out["h"] = kda.recurrence_fwd(*gates, h0=s["h0"], cu_seqlens=s["cu"],
                                                    edges=edges)
        back = kda.recurrence_bwd(*gates, s["dy"], h0=s["h0"], dh_out=s["dh"],
                                  cu_seqlens=s["cu"], edges=edges, want_dh0=s["h0"] is not None)
        out.update(dx=back["dx"], dz=back["dz"], di=back["di"], dA=back["dA_log"])
        if s["h0"] is not None:
            out["dh0"] = back["dh0"]
        return out
    if op == "keep":
        codes, exps = kda.checkpoint_pack(s["x"])
        return dict(x=kda.checkpoint_unpack(codes, exps, s["x"].dtype))
    if op == "step":
        y = kda.recurrence_step(s["x"], s["z"], s["i"], s["A"], G_MIN, s["h"], slots=s["slots"])
        return dict(y=y, h=s["h"])
    kw = dict(gate=s["gate"], scale=s["scale"], w_post=s["w_post"], w_pre=s["w_pre"],
              post_norm=s["case"]["post"], eps=EPS)
    if op == "norm":
        r, x = kda.block_norm(s["y"], s["r"], **kw)
        return dict(r=r, x=x)
    out = kda.block_norm_bwd(s["y"], s["r"], s["dx"], dr=s["dr"], **kw)
    return {n: t for n, t in out.items() if t is not None}


def exact(case, seed):
    """What run() returns, from the definitions in 64 bits."""
    c = case
    s = prepare(case, seed)

    def sigmoid(t):
        return torch.special.expit(t)

    def activation(t):
        """An input in 64 bits, as it is or as its codes stand for it."""
        if not isinstance(t, tuple):
            return t.double()
        codes, e = t
        at = torch.arange(codes.shape[1], device=codes.device) // GROUP
        return torch.ldexp(codes.double(), e.t()[:, at].int())

    def recurrence():
        x, z, i = (activation(s[n]) for n in ("x", "z", "i"))
        rate = s["A"].double().exp()
        gz, gi = sigmoid(z * rate), sigmoid(i)
        g = G_MIN * gz
        a, m = g.exp(), (-torch.expm1(2 * g)).sqrt()
        T, D = x.shape
        N = len(s["lengths"])
        zero = torch.zeros(N, D, dtype=torch.float64, device="cuda")
        h0 = zero if s["h0"] is None else s["h0"].double()
        b = m * gi * x
        h, end, t = torch.empty_like(x), h0.clone(), 0
        starts = []
        for n, ln in enumerate(s["lengths"]):
            starts.append(t)
            state = h0[n]
            for t in range(t, t + ln):
                state = torch.addcmul(b[t], a[t], state, out=h[t])
            t = starts[-1] + ln
            if ln:
                end[n] = state
        out = dict(y=h, h=end) if c["op"] in ("fwd", "train") else {}
        if c["op"] == "fwd":
            return out
        del b
        prev = torch.empty_like(x)
        prev[1:] = h[:-1]
        dh = zero if s["dh"] is None else s["dh"].double()
        dh0 = torch.empty_like(dh)
        lam = s["dy"].double().clone()
        for n, ln in enumerate(s["lengths"]):
            f = starts[n]
            if ln == 0:
                dh0[n] = dh[n]
                continue
            prev[f] = h0[n]
            lam[f + ln - 1] += dh[n]
            for t in range(f + ln - 2, f - 1, -1):
                lam[t].addcmul_(a[t + 1], lam[t + 1])
            dh0[n] = a[f] * lam[f]
        out["dx"] = lam * m * gi
        out["di"] = out["dx"] * x * (1 - gi)
        dm = -(a * a) / m                       # dm / dg
        dz = lam * (a * prev + dm * gi * x) * g * (1 - gz) * rate
        out["dz"], out["dA"] = dz, (dz * z).sum(0)
        if s["h0"] is not None:
            out["dh0"] = dh0
        return out

    def keep():
        """Each group's exponent by trial: the smallest whose codes fit."""
        x = s["x"].double()
        out = torch.empty_like(x)
        for b in range(0, c["D"], GROUP):
            v = x[:, b:b + GROUP]
            top = v.abs().amax(1, keepdim=True)
            e = (top / 128).log2().floor().clamp(min=-140, max=125)
            e = torch.where(top == 0, -127.0, e)
            for _ in range(3):
                e = torch.where(torch.round(top * torch.exp2(-e)) > 127, e + 1, e)
            e = e.clamp(-127, 121)
            out[:, b:b + GROUP] = torch.exp2(e) * (v * torch.exp2(-e)).round().clamp(-127, 127)
        return dict(x=out)

    def step():
        h, y = s["h"].double(), torch.zeros(c["N"], c["D"], dtype=torch.float64, device="cuda")
        rate = s["A"].double().exp()
        for n, slot in enumerate(s["slots"].tolist()):
            if slot < 0:
                continue
            g = G_MIN * sigmoid(rate * s["z"][n].double())
            u = sigmoid(s["i"][n].double()) * s["x"][n].double()
            h[slot] = y[n] = g.exp() * h[slot] + (1 - (2 * g).exp()).sqrt() * u
        return dict(y=y, h=h)

    def norm():
        """The forward as written; its gradients by differentiating it."""
        y = s["y"].double()
        leaf = {n: s[n].double().requires_grad_(c["op"] == "norm_bwd")
                for n in ("gate", "scale", "w_post", "w_pre") if s[n] is not None}

        def rms(t):
            return (t.square().sum(-1, keepdim=True) / c["D"] + EPS).sqrt()

        def added(y):
            n = y / rms(y) if c["post"] else y
            for name in ("w_post", "scale"):
                n = n * leaf[name] if name in leaf else n
            return n * sigmoid(leaf["gate"]) if "gate" in leaf else n

        if c["op"] == "norm":
            r = s["r"].double() + added(y)
            return dict(r=r, x=leaf["w_pre"] * r / rms(r))
        r = s["r"].double().requires_grad_(True)
        dr = s["dr"].double() + torch.autograd.grad(
            leaf["w_pre"] * r / rms(r), [r], s["dx"].double())[0]
        out = dict(dr=dr, dw_pre=(s["dx"].double() * (r / rms(r)).detach()).sum(0))
        y.requires_grad_(True)
        names = [n for n in ("gate", "scale", "w_post") if n in leaf]
        grads = torch.autograd.grad(added(y), [y] + [leaf[n] for n in names], dr)
        return dict(out, **{"d" + n: t for n, t in zip(["y"] + names, grads)})

    if c["op"] == "keep":
        return keep()
    if c["op"] == "step":
        return step()
    return norm() if "T" in c else recurrence()
