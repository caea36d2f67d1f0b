"""GPU parity of the per-head-decay linear attention (forward, gradients, single-token step)
against the recurrence in 64 bits.

Tolerances.  bf16 outputs carry one rounding of the result (at most 2^-9 relative, taken as 2^-8)
plus the intermediate error: operands of a product are held to 2^-17 or better, so a sum of
products is off by at most 2 * 2^-17 of the sum of its absolute terms; against the rms of a head's
outputs, whose absolute sums are up to about 16 times larger here, that is 2.5e-4, taken as 5e-4.
fp32 outputs: 2-norm of the error over 2-norm of the result at most 1e-5 (the operands' 2^-17
spread over independent roundings is 3e-6, fp32 sums of up to some thousand terms about 2e-6).
"""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    from serving_kda_chunkwise_gb300 import kda as _k
    return _k


def _inputs(seed, lengths, H, dk, dv, dtype, per_token=True, state=True, strided=False, decay=0.2):
    import torch
    gen = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    T, N = sum(lengths), len(lengths)

    def rand(*s):
        return torch.randn(s, generator=gen)

    def place(x):
        x = x.to(dt).cuda()
        if not strided:
            return x
        wide = torch.full((x.shape[0], x.shape[1] * x.shape[2] + 16), float("nan"), dtype=dt,
                          device="cuda")
        view = wide[:, 8:8 + x.shape[1] * x.shape[2]].unflatten(1, x.shape[1:])
        view.copy_(x)
        return view

    q, k = (place(x / x.norm(dim=-1, keepdim=True)) for x in (rand(T, H, dk), rand(T, H, dk)))
    v, do = place(rand(T, H, dv)), place(rand(T, H, dv))
    g = -decay * (rand(T, H).abs() if per_token else torch.linspace(0.05, 1.0, H))
    S0 = 0.3 * rand(N, H, dk, dv) if state else None
    dS = 0.3 * rand(N, H, dk, dv) if state else None
    cu = torch.tensor([0] + list(torch.tensor(lengths).cumsum(0)), dtype=torch.int32).cuda()
    return dict(q=q, k=k, v=v, do=do, g=g.float().cuda(), S0=None if S0 is None else S0.cuda(),
                dS=None if dS is None else dS.cuda(), cu=cu, lengths=lengths)


def _near(got, ref, name):
    import torch
    assert got.shape == ref.shape, name
    if ref.numel() == 0:
        return
    d = (got.double() - ref).abs()
    if got.dtype == torch.bfloat16:
        rms = ref.square().mean((0, 2), keepdim=True).sqrt()
        bad = d - 2.0 ** -8 * ref.abs() - 5e-4 * rms
        assert bool((bad <= 0).all()), (name, float(bad.max()))
    else:
        n = float(ref.norm())
        assert float(d.norm()) <= 1e-5 * n, (name, float(d.norm()) / max(n, 1e-300))


def _check_fwd(kda, x):
    import linear_ref
    o, S = kda.linear_fwd_chunked(x["q"], x["k"], x["v"], x["g"], S0=x["S0"], cu_seqlens=x["cu"])
    kda.device_status()
    ro, rS = linear_ref.forward(x["q"], x["k"], x["v"], x["g"], x["S0"], x["lengths"])
    _near(o, ro, "o")
    _near(S, rS, "S")


def _check_bwd(kda, x):
    import linear_ref
    got = kda.linear_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS_out=x["dS"],
                         cu_seqlens=x["cu"])
    kda.device_status()
    ref = linear_ref.gradients(x["q"], x["k"], x["v"], x["g"], x["do"], x["S0"], x["dS"],
                               x["lengths"])
    for n in ("dq", "dk", "dv", "dg", "dS0"):
        _near(got[n], ref[n], n)


LENGTHS = [[1], [63], [129], [300, 0, 1, 17], [0, 700], [64, 128, 65, 2, 0]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
def test_forward(kda, dtype, dk, dv, lengths):
    _check_fwd(kda, _inputs(1, lengths, 3, dk, dv, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
def test_gradients(kda, dtype, dk, dv, lengths):
    _check_bwd(kda, _inputs(2, lengths, 3, dk, dv, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("per_token,state", [(False, True), (True, False), (False, False)])
def test_fixed_decay_and_no_state(kda, dtype, per_token, state):
    x = _inputs(3, [200, 333], 2, 128, 64, dtype, per_token=per_token, state=state)
    _check_fwd(kda, x)
    _check_bwd(kda, x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_inputs(kda, dtype):
    x = _inputs(4, [150, 70], 2, 64, 128, dtype, strided=True)
    _check_fwd(kda, x)
    _check_bwd(kda, x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["none", "strong", "reset", "mixed"])
def test_decays(kda, dtype, kind):
    """No decay; decays whose product underflows inside a chunk; exact resets (g = -inf); strong
    and weak tokens side by side."""
    import torch
    x = _inputs(5, [400, 131], 2, 128, 128, dtype)
    g = x["g"]
    if kind == "none":
        g.zero_()
    elif kind == "strong":
        g.mul_(100.0)
    elif kind == "reset":
        g[[0, 5, 127, 128, 250, 399, 400, 530]] = -float("inf")
        g[300:310] = -float("inf")
    else:
        g[::3] = -40.0
        g[200:260] = -90.0
    _check_fwd(kda, x)
    if kind != "reset":
        _check_bwd(kda, x)
    else:
        out = kda.linear_bwd(x["q"], x["k"], x["v"], g, x["do"], S0=x["S0"], dS_out=x["dS"],
                             cu_seqlens=x["cu"])
        import linear_ref
        ref = linear_ref.gradients(x["q"], x["k"], x["v"], g, x["do"], x["S0"], x["dS"],
                                   x["lengths"])
        for n in ("dq", "dk", "dv", "dS0"):
            _near(out[n], ref[n], n)
        assert bool(torch.isfinite(out["dg"]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_against_differences(kda, dtype):
    """<gradient, direction> against the central difference of the loss computed in 64 bits."""
    import linear_ref
    import torch
    x = _inputs(6, [90, 41], 2, 64, 64, dtype)
    got = kda.linear_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS_out=x["dS"],
                         cu_seqlens=x["cu"])

    def loss(**over):
        y = {**x, **over}
        o, S = linear_ref.forward(y["q"], y["k"], y["v"], y["g"], y["S0"], y["lengths"])
        return float((o * x["do"].double()).sum() + (S * x["dS"].double()).sum())

    gen = torch.Generator(device="cuda").manual_seed(7)
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("S0", "dS0")):
        u = torch.randn(x[name].shape, generator=gen, device="cuda", dtype=torch.float64)
        e = 1e-4
        diff = (loss(**{name: x[name].double() + e * u})
                - loss(**{name: x[name].double() - e * u})) / (2 * e)
        exact = float((got[grad].double() * u).sum())
        # the roundings of the gradient's entries, 2^-9 each for bf16, add up at random
        tol = (2.0 ** -8 if got[grad].dtype == torch.bfloat16 else 1e-4)
        scale = float((got[grad].double() * u).norm()) * 4
        assert abs(diff - exact) <= tol * scale + 1e-6 * abs(diff), name


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_segments(kda, dtype):
    """Long sequences are cut into segments: forward and gradients across their edges."""
    x = _inputs(8, [2500, 3, 1029], 16, 64, 64, dtype, decay=0.02)
    _check_fwd(kda, x)
    _check_bwd(kda, x)


def test_state_in_place_and_equal_lengths(kda):
    """S_out in S0's place, and N equal sequences without offsets."""
    import torch
    x = _inputs(9, [1500, 1500], 8, 128, 128, "bf16")
    o, S = kda.linear_fwd_chunked(x["q"], x["k"], x["v"], x["g"], S0=x["S0"], cu_seqlens=x["cu"])
    S0 = x["S0"].clone()
    o2, S2 = kda.linear_fwd_chunked(x["q"], x["k"], x["v"], x["g"], S0=S0, N=2, S_out=S0)
    assert S2 is S0 and torch.equal(o, o2) and torch.equal(S, S2)
    o3, none = kda.linear_fwd_chunked(x["q"], x["k"], x["v"], x["g"], S0=x["S0"],
                                      cu_seqlens=x["cu"], want_state=False)
    assert none is None and torch.equal(o, o3)


def test_deterministic_and_other_stream(kda):
    import torch
    x = _inputs(10, [900, 77], 4, 128, 128, "bf16")

    def run():
        f = kda.linear_fwd_chunked(x["q"], x["k"], x["v"], x["g"], S0=x["S0"], cu_seqlens=x["cu"])
        b = kda.linear_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS_out=x["dS"],
                           cu_seqlens=x["cu"])
        return list(f) + [b[n] for n in sorted(b)]

    first = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = run()
    s.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_resume_and_step_follow_the_prompt(kda):
    """A prompt in two calls, then tokens one by one, equals the whole in one call."""
    import torch
    H, d, T = 3, 128, 330
    x = _inputs(11, [T], H, d, d, "f32", state=False)
    q, k, v, g = x["q"], x["k"], x["v"], x["g"]
    o, S = kda.linear_fwd_chunked(q, k, v, g)
    o1, S1 = kda.linear_fwd_chunked(q[:201], k[:201], v[:201], g[:201])
    o2, S2 = kda.linear_fwd_chunked(q[201:320], k[201:320], v[201:320], g[201:320], S0=S1)
    pool = torch.zeros(5, H, d, d, device="cuda")
    pool[3] = S2[0]
    outs = [o1, o2]
    slot = torch.tensor([3], dtype=torch.int32, device="cuda")
    for t in range(320, T):
        outs.append(kda.linear_decode_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], g[t:t + 1], pool,
                                           slots=slot))
    _near(torch.cat(outs), o.double(), "o")
    _near(pool[3:4], S.double(), "S")
    assert float(pool[[0, 1, 2, 4]].abs().max()) == 0.0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("N,H,per_token", [(1, 1, True), (7, 3, False), (40, 8, True)])
def test_step(kda, dtype, dk, dv, N, H, per_token):
    import linear_ref
    import torch
    x = _inputs(12, [N], H, dk, dv, dtype, per_token=per_token, state=False, strided=N == 7)
    pool = torch.randn(N + 3, H, dk, dv, device="cuda")
    slots = torch.randperm(N + 3, device="cuda")[:N].to(torch.int32)
    if N > 1:
        slots[1] = -1
    before = pool.clone()
    o = kda.linear_decode_step(x["q"], x["k"], x["v"], x["g"], pool, slots=slots)
    kda.device_status()
    ref = before.double()
    for i, s in enumerate(slots.tolist()):
        if s < 0:
            assert float(o[i].float().abs().max()) == 0.0
            continue
        gi = x["g"][i:i + 1] if per_token else x["g"]
        ro, rS = linear_ref.forward(x["q"][i:i + 1], x["k"][i:i + 1], x["v"][i:i + 1], gi,
                                    before[s:s + 1], [1])
        ref[s] = rS[0]
        _near(o[i:i + 1], ro, f"o {i}")
    _near(pool, ref, "S")


def test_step_without_slots_and_bad_slot(kda):
    import torch
    x = _inputs(13, [3], 2, 64, 64, "f32", state=False)
    pool = torch.randn(3, 2, 64, 64, device="cuda")
    a, b = pool.clone(), pool.clone()
    o = kda.linear_decode_step(x["q"], x["k"], x["v"], x["g"], a)
    ids = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    assert torch.equal(o, kda.linear_decode_step(x["q"], x["k"], x["v"], x["g"], b, slots=ids))
    assert torch.equal(a, b)
    ids[1] = 3  # outside the pool: reported, and the row counts as unused
    o = kda.linear_decode_step(x["q"], x["k"], x["v"], x["g"], b, slots=ids)
    with pytest.raises(kda.KdaError) as e:
        kda.device_status()
    assert e.value.status == kda.KDA_ERR_DEVICE and "slot" in str(e.value)
    assert float(o[1].abs().max()) == 0.0 and torch.equal(a[1], b[1])


def test_malformed_offsets_are_reported(kda):
    import torch
    x = _inputs(14, [40, 60], 2, 64, 64, "bf16", state=False)
    for bad in ([0, 70, 40], [0, 40, 99], [5, 40, 100]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        kda.linear_fwd_chunked(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu)
        with pytest.raises(kda.KdaError) as e:
            kda.device_status()
        assert e.value.status == kda.KDA_ERR_DEVICE


def test_nothing_to_do(kda):
    import torch
    z = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    g = torch.empty(0, 2, device="cuda")
    S0 = torch.randn(2, 2, 64, 64, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    o, S = kda.linear_fwd_chunked(z, z, z, g, S0=S0, cu_seqlens=cu)
    assert o.shape == (0, 2, 64) and torch.equal(S, S0)
    out = kda.linear_bwd(z, z, z, torch.zeros(2, device="cuda"), z, dS_out=S0, cu_seqlens=cu)
    assert torch.equal(out["dS0"], S0) and float(out["dg"].abs().max()) == 0.0
    assert kda.linear_decode_step(z, z, z, g, S0).shape == (0, 2, 64)


def test_binding_refusals(kda):
    import torch
    x = _inputs(15, [20], 2, 64, 64, "bf16")
    q, k, v, g = x["q"], x["k"], x["v"], x["g"]
    with pytest.raises(TypeError):
        kda.linear_fwd_chunked(q, k.float(), v, g)
    with pytest.raises(TypeError):
        kda.linear_fwd_chunked(q, k, v, g.double())
    with pytest.raises(ValueError):
        kda.linear_fwd_chunked(q, k[:19], v, g)
    with pytest.raises(ValueError):
        kda.linear_fwd_chunked(q, k, v, g[:, :1].contiguous())
    with pytest.raises(ValueError):
        kda.linear_fwd_chunked(q.transpose(0, 1), k, v, g)
    with pytest.raises(ValueError):
        kda.linear_fwd_chunked(q, k, v, g, S0=x["S0"][:, :1].contiguous())
    with pytest.raises(kda.KdaError) as e:
        kda.linear_fwd_chunked(q, k, v, g, N=3)
    assert e.value.status == kda.KDA_ERR_INVALID_ARG
    odd = torch.zeros(20, 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")[:, :128]
    with pytest.raises(kda.KdaError):
        kda.linear_fwd_chunked(odd.unflatten(1, (2, 64)), k, v, g)
    with pytest.raises(kda.KdaError) as e:
        kda.linear_decode_step(q, k, v, g, torch.zeros(19, 2, 64, 64, device="cuda"))
    assert "n_slots" in str(e.value)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", [[70, 45, 60], [300, 45, 1000]], ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=str)
def test_not_finite_stays_in_its_sequence(kda, dtype, lengths, bad):
    """A sequence of NaN or infinities, tokens, decays and state, leaves the others' results as
    they were, bit for bit; fp32 outputs before the token too."""
    import torch
    x = _inputs(21, lengths, 2, 128, 64, dtype)

    def run():
        o, S = kda.linear_fwd_chunked(x["q"], x["k"], x["v"], x["g"], S0=x["S0"],
                                      cu_seqlens=x["cu"])
        b = kda.linear_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS_out=x["dS"],
                           cu_seqlens=x["cu"])
        return dict(b, o=o, S=S)

    first = run()
    a, b = lengths[0], lengths[0] + lengths[1]
    for n in ("q", "k", "v", "do", "g"):
        x[n][a:b] = bad
    x["S0"][1] = x["dS"][1] = bad
    second = run()
    kda.device_status()
    for n, t in second.items():
        if n in ("S", "dS0"):
            assert torch.equal(t[[0, 2]], first[n][[0, 2]]), n
        else:
            assert torch.equal(t[:a], first[n][:a]) and torch.equal(t[b:], first[n][b:]), n
    assert not bool(torch.isfinite(second["o"][a:b]).any())
    if dtype == "f32":
        x = _inputs(22, lengths, 2, 128, 64, dtype)
        first, _ = kda.linear_fwd_chunked(x["q"], x["k"], x["v"], x["g"], cu_seqlens=x["cu"])
        x["k"][40] = bad
        second, _ = kda.linear_fwd_chunked(x["q"], x["k"], x["v"], x["g"], cu_seqlens=x["cu"])
        assert torch.equal(second[:40], first[:40])


def test_bf16_token_by_token(kda, monkeypatch):
    """bf16 on CUDA cores (the path of fp32), which the environment can ask for."""
    monkeypatch.setenv("KDA_FWD_PATH", "generic")
    for lengths in ([40, 0, 300], [700, 129]):
        x = _inputs(23, lengths, 3, 64, 128, "bf16")
        _check_fwd(kda, x)
        _check_bwd(kda, x)


@pytest.mark.parametrize("decay", [0.003, 0.49, 0.51, 9.0])
def test_f32_fixed_decay_over_many_tokens(kda, decay):
    """One decay for all of 4000 tokens: its own rounding must not add up."""
    import linear_ref
    import torch
    x = _inputs(24, [4000], 2, 64, 64, "f32", per_token=False)
    x["g"] = torch.full((2,), -decay, device="cuda")
    o, S = kda.linear_fwd_chunked(x["q"], x["k"], x["v"], x["g"], S0=x["S0"], cu_seqlens=x["cu"])
    ro, rS = linear_ref.forward(x["q"], x["k"], x["v"], x["g"], x["S0"], x["lengths"])
    # fp32 sums of some hundred terms, 2^-24 each in quadrature: below 2e-6
    assert float((o.double() - ro).norm()) <= 2e-6 * float(ro.norm())
    assert float((S.double() - rS).norm()) <= 2e-6 * float(rS.norm())


@pytest.mark.parametrize("dtype,lengths", [("bf16", [200, 52]), ("bf16", [2500, 17, 900]),
                                           ("f32", [900, 300])])
def test_graph_and_two_streams(kda, dtype, lengths):
    """Replayed from a graph, and on two streams at once, the results are the same bits."""
    import torch
    x = _inputs(25, lengths, 4, 128, 128, dtype)

    def run():
        f = kda.linear_fwd_chunked(x["q"], x["k"], x["v"], x["g"], S0=x["S0"], cu_seqlens=x["cu"])
        b = kda.linear_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS_out=x["dS"],
                           cu_seqlens=x["cu"])
        return list(f) + [b[n] for n in sorted(b)]

    first = run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, out):
        assert torch.equal(a, b)
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(run())
    torch.cuda.synchronize()
    kda.device_status()
    for o in outs:
        for a, b in zip(first, o):
            assert torch.equal(a, b)
