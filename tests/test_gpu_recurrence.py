"""GPU parity of the gated channel recurrence, its gradients and its single-token step against the
definition in 64 bits, within the running error bounds of recurrence_ref.py (formed from the
arithmetic, element by element) and half a step of a rounded result."""
import pytest

pytestmark = pytest.mark.gpu
G_MIN = -5.0


@pytest.fixture(scope="module")
def kda():
    from serving_kda_chunkwise_gb300 import kda as _k
    return _k


def _inputs(seed, lengths, D, dtype="bf16", state=True, strided=False, level=(-7.0, 1.0)):
    import torch
    gen = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    T, N = sum(lengths), len(lengths)

    def rand(*s):
        return torch.randn(s, generator=gen)

    lv = level[0] + (level[1] - level[0]) * torch.rand(D, generator=gen)
    x, z, i = rand(T, D), rand(T, D) + lv, 2 * rand(T, D)
    if strided:
        pad = torch.full((T, 8), 1e4)
        both = torch.cat([pad, x, z, pad, i], 1).to(dt).cuda()
        x, z, i = both[:, 8:8 + D], both[:, 8 + D:8 + 2 * D], both[:, 16 + 2 * D:]
    else:
        x, z, i = (t.to(dt).cuda() for t in (x, z, i))
    cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32).cuda()
    return dict(x=x, z=z, i=i, A=(0.3 * rand(D)).cuda(), lengths=lengths, cu=cu,
                h0=rand(N, D).cuda() if state else None, dy=rand(T, D).to(dt).cuda(),
                dh=rand(N, D).cuda() if state else None)


def _fwd(kda, s, **kw):
    return kda.recurrence_fwd(s["x"], s["z"], s["i"], s["A"], G_MIN, h0=s["h0"],
                              cu_seqlens=s["cu"], **kw)


def _bwd(kda, s, **kw):
    return kda.recurrence_bwd(s["x"], s["z"], s["i"], s["A"], G_MIN, s["dy"], h0=s["h0"],
                              dh_out=s["dh"], cu_seqlens=s["cu"], **kw)


def _check(kda, s):
    import recurrence_ref as R
    import torch
    edges = kda.recurrence_edges(s["x"])
    y, h = _fwd(kda, s, edges=edges)
    got, kept = _bwd(kda, s), _bwd(kda, s, edges=edges)
    kda.device_status()
    ref = R.recurrence(s["x"], s["z"], s["i"], s["A"], G_MIN, s["h0"], s["lengths"], s["dy"],
                       s["dh"])
    R.near(y, ref["y"], "y")
    R.near(h, ref["h"], "h")
    R.near(edges, ref["edges"], "edges")
    for n, k in (("dx", "dx"), ("dz", "dz"), ("di", "di"), ("dA", "dA_log"), ("dh0", "dh0")):
        R.near(got[k], ref[n], n)
        assert torch.equal(got[k], kept[k]), k


LENGTHS = [[1], [63], [64], [65], [0, 5, 0], [128, 1], [129], [300, 0, 1, 64, 64, 130, 0],
           [1] * 70, [3, 61, 64, 2, 200], [1500]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda x: "-".join(map(str, x[:6])))
def test_lengths(kda, dtype, lengths):
    _check(kda, _inputs(1, lengths, 72, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,state,strided", [(8, True, False), (64, False, True), (128, True, True),
                                             (200, False, False), (1000, True, True),
                                             (2056, True, False)])
def test_widths(kda, dtype, D, state, strided):
    _check(kda, _inputs(2, [70, 0, 131, 1], D, dtype, state, strided))


@pytest.mark.parametrize("level", [(-14.0, -9.0), (3.0, 9.0), (-60.0, -30.0)])
def test_decays(kda, level):
    """Channels that hardly forget, that forget at once, and that hardly take anything in."""
    _check(kda, _inputs(3, [700, 33], 64, "f32", level=level))


def test_many_tiles(kda):
    """More pieces of the sequences than an SM count's worth, ragged."""
    _check(kda, _inputs(4, [2000, 17, 900, 1, 64, 3000], 264, "bf16"))


def test_equal_sequences_without_offsets(kda):
    import torch
    s = _inputs(5, [90] * 7, 80, "f32")
    y, h = _fwd(kda, s)
    got = _bwd(kda, s)
    y2, h2 = kda.recurrence_fwd(s["x"], s["z"], s["i"], s["A"], G_MIN, h0=s["h0"], N=7)
    got2 = kda.recurrence_bwd(s["x"], s["z"], s["i"], s["A"], G_MIN, s["dy"], h0=s["h0"],
                              dh_out=s["dh"], N=7)
    assert torch.equal(y, y2) and torch.equal(h, h2)
    for n in got:
        assert torch.equal(got[n], got2[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 136])
def test_packed_inputs(kda, dtype, D):
    """The gradients from 8-bit inputs are those from the values that these stand for."""
    import recurrence_ref as R
    import torch
    s = _inputs(6, [150, 0, 1, 333], D, dtype)
    kept = [kda.checkpoint_pack(s[n]) for n in ("x", "z", "i")]
    got = kda.recurrence_bwd(*kept, s["A"], G_MIN, s["dy"], h0=s["h0"], dh_out=s["dh"],
                             cu_seqlens=s["cu"])
    x, z, i = (kda.checkpoint_unpack(*k, s["x"].dtype) for k in kept)
    ref = R.recurrence(x, z, i, s["A"], G_MIN, s["h0"], s["lengths"], s["dy"], s["dh"])
    for n, k in (("dx", "dx"), ("dz", "dz"), ("di", "di"), ("dA", "dA_log"), ("dh0", "dh0")):
        R.near(got[k], ref[n], n)
    whole = _bwd(kda, dict(s, x=x, z=z, i=i))
    for n in got:
        assert torch.equal(got[n], whole[n]), n


def test_optional_tensors(kda):
    import torch
    s = _inputs(7, [100, 50], 64, "bf16")
    y, h = _fwd(kda, s)
    y2, none = _fwd(kda, s, want_state=False)
    assert none is None and torch.equal(y, y2)
    got = _bwd(kda, s)
    part = _bwd(kda, s, want_dA=False, want_dh0=False)
    assert part["dA_log"] is None and part["dh0"] is None
    for n in ("dx", "dz", "di"):
        assert torch.equal(part[n], got[n])
    inplace = s["h0"].clone()
    y3, h3 = kda.recurrence_fwd(s["x"], s["z"], s["i"], s["A"], G_MIN, h0=inplace,
                                cu_seqlens=s["cu"], h_out=inplace)
    assert h3 is inplace and torch.equal(h3, h) and torch.equal(y3, y)


@pytest.mark.parametrize("N,T", [(0, 0), (3, 0)])
def test_no_tokens(kda, N, T):
    import torch
    s = _inputs(8, [0] * N, 64, "bf16")
    y, h = _fwd(kda, s)
    assert y.shape == (0, 64) and torch.equal(h, s["h0"])
    got = _bwd(kda, s)
    assert torch.equal(got["dh0"], s["dh"]) and float(got["dA_log"].abs().sum()) == 0.0


@pytest.mark.parametrize("lengths", [
    [0, 3] * 15 + [7], [0, 3] * 16, [0, 3] * 16 + [7], [5] * 31 + [0], [5] * 32 + [0],
    [1500, 0, 1200, 900, 0, 2000], [0] * 30 + [4000, 1], [1200] * 33])
def test_few_and_more_sequences(kda, lengths):
    """On both sides of the numbers that the forward finds its way through by itself, in several runs
    and in one, with empty sequences anywhere."""
    _check(kda, _inputs(24, lengths, 72, "bf16"))


def test_very_many_empty_sequences(kda):
    """300,000 empty sequences at a token, in front of the first and behind the last one."""
    import torch
    s, n = _inputs(29, [40, 9, 25], 72, "f32"), 300000
    want = [*_fwd(kda, s), *_bwd(kda, s).values()]
    some = torch.tensor([n, 2 * n + 1, 3 * n + 2], device="cuda")
    lengths = torch.zeros(4 * n + 3, dtype=torch.int64, device="cuda")
    lengths[some] = torch.tensor(s["lengths"], device="cuda")
    cu = torch.cat([lengths[:1] * 0, lengths.cumsum(0)]).to(torch.int32)
    states = [torch.randn(4 * n + 3, 72, device="cuda") for _ in range(2)]
    for t, part in zip(states, (s["h0"], s["dh"])):
        t[some] = part
    s.update(cu=cu, h0=states[0], dh=states[1])
    got = [*_fwd(kda, s), *_bwd(kda, s).values()]
    kda.device_status()
    for k, (a, b) in enumerate(zip(got, want)):
        empty = dict(((1, 0), (6, 1))).get(k)  # final states, and the first ones' gradients
        if empty is None:
            assert torch.equal(a, b), k
        else:
            assert torch.equal(a[some], b), k
            states[empty][some] = a[some]
            assert torch.equal(a, states[empty]), k


@pytest.mark.parametrize("N", [2, 32, 33])
def test_equal_sequences(kda, N):
    import torch
    s = _inputs(25, [40] * N, 64, "f32")
    want = [*_fwd(kda, s), *_bwd(kda, s).values()]
    s["cu"] = None
    got = [*_fwd(kda, s, N=N), *_bwd(kda, s, N=N).values()]
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_long_memory_of_alike_gates(kda):
    """Gates that are alike make the same rounding again and again: a state that remembers 600 to 1,600
    tokens is as exact as its gates.  c = e^g - 1 is off by 3.3e-7 (polynomial) + 2.4e-7 (exponential
    and reciprocal) + 6.6e-7 (the exponential's argument, up to 13 with a step of 2^-20, and the factor
    log2(e)) at most, the state by one and a half times that, and its own roundings, which are not
    alike, by 6e-8 sqrt(1600 / 16): 2.5e-6 (one rounding of the decay every 8 tokens: 5e-6)."""
    import torch
    T, D = 8192, 128
    z = torch.linspace(-9, -8, D, device="cuda").expand(T, D).contiguous()
    x = torch.randn(T, D, generator=torch.Generator("cuda").manual_seed(26), device="cuda")
    i, A = torch.zeros_like(x), torch.zeros(D, device="cuda")
    y, _ = kda.recurrence_fwd(x, z, i, A, G_MIN)
    g = G_MIN * torch.sigmoid(z[0].double())
    a, b = g.exp(), (-torch.expm1(2 * g)).sqrt() * 0.5
    want, h = torch.empty(T, D, dtype=torch.float64, device="cuda"), 0.0
    for t in range(T):
        want[t] = h = a * h + b * x[t].double()
    off = (y.double() - want).norm(dim=0) / want.norm(dim=0)
    assert float(off.max()) <= 2.5e-6
    # and the rate's gradient, a sum with a hundredth of its terms' size left
    dy = torch.randn(T, D, generator=torch.Generator("cuda").manual_seed(27), device="cuda")
    got = kda.recurrence_bwd(x, z, i, A, G_MIN, dy)
    before = torch.cat([torch.zeros(1, D, dtype=torch.float64, device="cuda"), want[:-1]])
    lam, total = torch.zeros(D, dtype=torch.float64, device="cuda"), 0.0
    s = torch.sigmoid(z[0].double())
    size = 0.0
    for t in range(T - 1, -1, -1):
        lam = dy[t].double() + lam
        dz = lam * (a * before[t] - a * a / (2 * b) * 0.5 * x[t].double()) * g * (1 - s)
        total, size = total + dz * z[t].double(), size + (dz * z[t].double()).abs()
        lam = a * lam
    assert float(((got["dA_log"].double() - total).abs() / size).max()) <= 2.5e-6


def test_outlier_decays(kda):
    """After a token of 1e6 that a fast channel forgets at once, the state is as exact as without it."""
    import torch
    T, D = 200, 64
    x = torch.randn(T, D, generator=torch.Generator("cuda").manual_seed(28), device="cuda")
    z, i, A = torch.full_like(x, 3.0), torch.zeros_like(x), torch.zeros(D, device="cuda")
    big = x.clone()
    big[[5, 70, 127, 130]] = 1e6
    want, h = kda.recurrence_fwd(x, z, i, A, G_MIN)
    got, h2 = kda.recurrence_fwd(big, z, i, A, G_MIN)
    # e^-4.76 a token: 1e6 is below 2^-24 after seven
    for t in (*range(14, 70), *range(79, 127), *range(139, T)):
        assert float((got[t] - want[t]).abs().max()) <= 1e-6
    assert float((h - h2).abs().max()) <= 1e-6


def test_one_sequence_without_tokens(kda):
    import torch
    s = _inputs(8, [0], 64, "bf16")
    for cu in (s["cu"], None):
        s["cu"] = cu
        y, h = _fwd(kda, s)
        assert y.shape == (0, 64) and torch.equal(h, s["h0"])
        got = _bwd(kda, s)
        assert torch.equal(got["dh0"], s["dh"]) and float(got["dA_log"].abs().sum()) == 0.0


def test_infinite_gates(kda):
    """z = -inf keeps the state, z = +inf decays it by e^g_min, i = -inf takes nothing in."""
    import recurrence_ref as R
    import torch
    s = _inputs(9, [130, 20], 64, "f32")
    inf = float("inf")
    for t, name, v in ((5, "z", -inf), (6, "z", -inf), (70, "z", inf), (100, "i", -inf),
                       (101, "i", inf), (131, "z", -inf), (149, "z", -inf)):
        s[name][t, ::2] = v
    _check(kda, s)
    y, _ = _fwd(kda, s)
    assert torch.equal(y[5, ::2], y[4, ::2]) and torch.equal(y[6, ::2], y[4, ::2])
    del R


@pytest.mark.parametrize("name,value", [("x", float("nan")), ("x", float("inf")),
                                        ("z", float("nan")), ("i", float("nan"))])
def test_not_finite_stays_in_its_channel(kda, name, value):
    import torch
    s = _inputs(10, [100, 150, 90], 72, "bf16")
    y, h = _fwd(kda, s)
    g = _bwd(kda, s)
    s[name][140, 9] = value
    y2, h2 = _fwd(kda, s)
    g2 = _bwd(kda, s)
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[140:250, 9] = False
    assert torch.equal(y[keep], y2[keep])
    assert not bool(torch.isfinite(y2[140:250, 9]).any())
    keep[100:140, 9] = False
    for n in ("dx", "dz", "di"):
        assert torch.equal(g[n][keep], g2[n][keep]), n
    some = torch.ones(3, 72, dtype=torch.bool)
    some[1, 9] = False
    some = some.cuda()
    assert torch.equal(h[some], h2[some]) and torch.equal(g["dh0"][some], g2["dh0"][some])
    other = torch.arange(72, device="cuda") != 9
    assert torch.equal(g["dA_log"][other], g2["dA_log"][other])


def test_gradient_against_differences(kda):
    import recurrence_ref as R
    import torch
    s = _inputs(11, [40, 25], 64, "f32", level=(-3.0, 1.0))
    got = _bwd(kda, s)
    e = 1e-5

    def loss(x, z, i, A, h0):
        r = R.recurrence(x, z, i, A, G_MIN, h0, s["lengths"])
        return float((r["y"][0] * s["dy"]).sum() + (r["h"][0] * s["dh"]).sum())

    base = [s[n].double() for n in ("x", "z", "i", "A", "h0")]
    for k, n in enumerate(("dx", "dz", "di", "dA_log", "dh0")):
        by = torch.randn_like(base[k])
        up, dn = list(base), list(base)
        up[k], dn[k] = base[k] + e * by, base[k] - e * by
        diff = (loss(*up) - loss(*dn)) / (2 * e)
        t = got[n].double() * by
        assert abs(diff - float(t.sum())) <= 1e-4 * float(t.norm()) + 1e-6 * abs(diff), n


def test_step_continues_prompts(kda):
    """Tokens one by one give what one call over the whole sequences gives."""
    import recurrence_ref as R
    import torch
    s = _inputs(12, [9] * 5, 200, "f32")
    pool = torch.zeros(8, 200, device="cuda")
    slots = torch.tensor([6, 1, 0, 7, 3], dtype=torch.int32, device="cuda")
    pool[slots.long()] = s["h0"]
    ref = R.recurrence(s["x"], s["z"], s["i"], s["A"], G_MIN, s["h0"], s["lengths"])
    for t in range(9):
        rows = [s[n].view(5, 9, 200)[:, t] for n in ("x", "z", "i")]
        y = kda.recurrence_step(*rows, s["A"], G_MIN, pool, slots=slots)
        R.near(y, [v.view(5, 9, 200)[:, t] for v in ref["y"]], t)
    R.near(pool[slots.long()], ref["h"], "pool")
    assert float(pool[[2, 4, 5]].abs().max()) == 0.0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,D,strided", [(1, 8, False), (1, 4096, False), (37, 72, True),
                                         (300, 2568, True)])
def test_step(kda, dtype, N, D, strided):
    import recurrence_ref as R
    import torch
    s = _inputs(13, [1] * N, D, dtype, strided=strided)
    pool = torch.randn(N + 3, D, device="cuda")
    keep = pool.clone()
    slots = torch.randperm(N + 3, device="cuda")[:N].to(torch.int32)
    unused = torch.arange(N, device="cuda") % 5 == 2
    slots[unused] = -1
    at = slots.clamp(min=0).long()
    ref = R.recurrence(s["x"], s["z"], s["i"], s["A"], G_MIN, keep[at], s["lengths"])
    y = kda.recurrence_step(s["x"], s["z"], s["i"], s["A"], G_MIN, pool, slots=slots)
    kda.device_status()
    used = ~unused
    R.near(y[used], [v[used] for v in ref["y"]], "y")
    assert float(y[unused].abs().sum()) == 0.0
    R.near(pool[at[used]], [v[used] for v in ref["h"]], "pool")
    others = torch.ones(N + 3, dtype=torch.bool, device="cuda")
    others[at[used]] = False
    assert torch.equal(pool[others], keep[others])


def test_step_without_slots_and_bad_slot(kda):
    import torch
    s = _inputs(14, [1] * 4, 64, "bf16")
    a, b = torch.randn(6, 64, device="cuda"), None
    b = a.clone()
    rows = (s["x"], s["z"], s["i"], s["A"], G_MIN)
    y = kda.recurrence_step(*rows, a)
    y2 = kda.recurrence_step(*rows, b, slots=torch.arange(4, dtype=torch.int32, device="cuda"))
    assert torch.equal(y, y2) and torch.equal(a, b)
    kda.device_status()
    c = b.clone()
    slots = torch.tensor([0, 6, 2, 3], dtype=torch.int32, device="cuda")
    y = kda.recurrence_step(*rows, c, slots=slots)
    with pytest.raises(kda.KdaError) as e:
        kda.device_status()
    assert e.value.status == kda.KDA_ERR_DEVICE
    assert float(y[1].abs().max()) == 0.0 and torch.equal(c[[1, 4, 5]], b[[1, 4, 5]])


def test_step_far_slot(kda):
    """Pool offsets past 32 bits."""
    import torch
    s = _inputs(15, [1, 1], 4096, "bf16")
    n = (1 << 32) // 4096 + 3
    pool = torch.empty(n, 4096, device="cuda")
    small = torch.randn(2, 4096, device="cuda")
    pool[n - 1], pool[5] = small[0], small[1]
    rows = (s["x"], s["z"], s["i"], s["A"], G_MIN)
    y = kda.recurrence_step(*rows, pool, slots=torch.tensor([n - 1, 5], dtype=torch.int32,
                                                            device="cuda"))
    y2 = kda.recurrence_step(*rows, small)
    assert torch.equal(y, y2)
    assert torch.equal(pool[n - 1], small[0]) and torch.equal(pool[5], small[1])


def test_far_rows(kda):
    """Row offsets past 32 bits: the last sequence of a long batch equals itself alone."""
    import torch
    D, last = 4096, 100
    T = (1 << 32) // D + 200
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, z, i = (torch.randn(T, D, generator=gen, device="cuda", dtype=torch.bfloat16)
               for _ in range(3))
    A = torch.zeros(D, device="cuda")
    cu = torch.tensor([0, T - last, T], dtype=torch.int32, device="cuda")
    y, h = kda.recurrence_fwd(x, z, i, A, G_MIN, cu_seqlens=cu)
    y2, h2 = kda.recurrence_fwd(x[-last:], z[-last:], i[-last:], A, G_MIN)
    kda.device_status()

    def same(a, b):  # (pieces of the sequence begin elsewhere: the sums' order differs)
        d = (a.float() - b.float()).abs()
        return bool((d <= 2.0 ** -7 * b.float().abs() + 1e-4).all())

    assert same(y[-last:], y2) and same(h[1], h2[0])
    g = kda.recurrence_bwd(x, z, i, A, G_MIN, y, cu_seqlens=cu)
    g2 = kda.recurrence_bwd(x[-last:], z[-last:], i[-last:], A, G_MIN, y[-last:])
    for n in ("dx", "dz", "di"):
        assert same(g[n][-last:], g2[n]), n


def test_malformed_offsets_are_reported(kda):
    import torch
    for bad in ([0, 60, 40, 100], [0, 40, 60, 101], [1, 40, 60, 100], [0, -5, 60, 100],
                [0, 40, 1 << 30, 100], [0, 40, 60, 99]):
        s = _inputs(16, [40, 20, 40], 72, "bf16")
        s["cu"] = torch.tensor(bad, dtype=torch.int32, device="cuda")
        for call in (_fwd, _bwd):
            call(kda, s)
            with pytest.raises(kda.KdaError) as e:
                kda.device_status()
            assert e.value.status == kda.KDA_ERR_DEVICE


def test_deterministic(kda):
    import torch
    s = _inputs(17, [3000, 500, 1, 2500], 520, "bf16")
    edges = kda.recurrence_edges(s["x"])
    first = [*_fwd(kda, s, edges=edges), edges, *_bwd(kda, s).values()]
    for _ in range(5):
        edges = kda.recurrence_edges(s["x"])
        again = [*_fwd(kda, s, edges=edges), edges, *_bwd(kda, s).values()]
        for a, b in zip(first, again):
            assert torch.equal(a, b)


def test_two_streams_and_graphs(kda):
    """Calls at once on two streams, and two graphs that share a workspace, replayed in turn with
    new inputs."""
    import torch
    s, r = _inputs(18, [2000, 30], 256, "bf16"), _inputs(19, [400, 900], 320, "f32")
    want = [[*_fwd(kda, q), *_bwd(kda, q).values()] for q in (s, r)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for q, st in zip((s, r), streams):
            got.append([*_fwd(kda, q, stream=st), *_bwd(kda, q, stream=st).values()])
    torch.cuda.synchronize()
    for k, outs in enumerate(got):
        for a, b in zip(outs, want[k % 2]):
            assert torch.equal(a, b)
    need = max(kda.library().kda_recurrence_bwd_workspace_size(q["x"].shape[0], 2, q["x"].shape[1])
               for q in (s, r))
    need = max(need, *(kda.library().kda_recurrence_fwd_workspace_size(q["x"].shape[0], 2,
                                                                       q["x"].shape[1])
                       for q in (s, r)))
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for q in (s, r):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([*_fwd(kda, q, workspace=ws), *_bwd(kda, q, workspace=ws).values()])
        graphs.append(g)
    for _ in range(2):
        for k in (0, 1, 0):
            for t in outs[k]:
                t.zero_()
            graphs[k].replay()
            for a, b in zip(outs[k], want[k]):
                assert torch.equal(a, b)
        for q, k in ((s, 0), (r, 1)):  # new inputs in the graphs' tensors
            q["x"].mul_(0.5)
            q["dy"].neg_()
            want[k] = [*_fwd(kda, q), *_bwd(kda, q).values()]
    kda.device_status()


def test_binding_refusals(kda):
    import torch
    s = _inputs(20, [10, 6], 64, "bf16")
    args = dict(x=s["x"], z=s["z"], i=s["i"], A_log=s["A"], g_min=G_MIN)
    fwd = kda.recurrence_fwd
    with pytest.raises(TypeError):
        fwd(**{**args, "z": s["z"].float()})
    with pytest.raises(TypeError):
        fwd(**{**args, "x": s["x"].half(), "z": s["z"].half(), "i": s["i"].half()})
    with pytest.raises(ValueError):
        fwd(**{**args, "i": s["i"][:, :56]})
    with pytest.raises(ValueError):
        fwd(**{**args, "x": s["x"].t().contiguous().t()})
    with pytest.raises(ValueError):
        fwd(**{**args, "x": s["x"].cpu()})
    with pytest.raises(ValueError):
        fwd(**args, h0=s["h0"])  # of two sequences, without offsets
    with pytest.raises(ValueError):
        fwd(**args, edges=torch.empty(1, 64, device="cuda"))
    with pytest.raises(ValueError):
        fwd(**args, cu_seqlens=s["cu"], N=3)
    with pytest.raises(kda.KdaError) as e:
        fwd(**{**args, "g_min": 0.0})
    assert e.value.status == kda.KDA_ERR_INVALID_ARG
    odd = {n: args[n][:, :60].contiguous() for n in ("x", "z", "i")}
    with pytest.raises(kda.KdaError) as e:
        fwd(**{**args, **odd, "A_log": s["A"][:60].contiguous()})
    assert e.value.status == kda.KDA_ERR_UNSUPPORTED
    off = torch.zeros(16, 66, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(kda.KdaError):  # rows that do not begin on 16 bytes
        fwd(**{**args, "x": off[:, :64]})
    kept = kda.checkpoint_pack(s["x"])
    with pytest.raises(TypeError):
        kda.recurrence_bwd(kept, s["z"], s["i"], s["A"], G_MIN, s["dy"])
    with pytest.raises(ValueError):
        kda.recurrence_bwd(kept, kept, kept, s["A"], G_MIN, s["dy"],
                           edges=kda.recurrence_edges(s["x"]))
    with pytest.raises(ValueError):
        kda.recurrence_bwd(kept, kept, (kept[0], kept[1][:, :8]), s["A"], G_MIN, s["dy"])
    with pytest.raises(TypeError):
        kda.recurrence_step(s["x"], s["z"], s["i"], s["A"], G_MIN, s["h0"].bfloat16())
    with pytest.raises(kda.KdaError):
        kda.recurrence_step(s["x"], s["z"], s["i"], s["A"], G_MIN, s["h0"])  # 2 states, 16 rows
    kda.device_status()
