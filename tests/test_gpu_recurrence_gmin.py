"""The channel recurrence under gates of other bounds than -5: the number of times a gate's exponential
is doubled comes from g_min (none down to -1.25, then one for every factor of two), and the decay of
several tokens from their summed gates.  Against the definition in 64 bits.

Bounds, beside those of recurrence_ref.py.  What include/kda.h states:
  - 1 - e^g is off by at most REL(u) = 1e-6 + 2.6e-7 |u| of itself, u = e^A z: 2^-22 (exponential) + 2^-24
    (the sum with one) + 2^-23 (reciprocal) + 2^-24 (times g_min) of the gate, 2^-23 |u| + 2^-24 |u| + 2^-24 |u|
    + 1.3e-8 |u| (e^A, its product with log2(e), that constant, the exponent's product; 2.5e-7 |u|) of the
    gate, 3.3e-7 of the polynomial and 2^-23 of its roundings and the doublings'.
  - e^g by at most ABS(u) = 6e-7 + 1e-7 |u|: of the gate's relative error |g| e^g <= 0.37 arrives, of the
    polynomial's (up to 2.4e-7 there) and the roundings' with the doublings 3e-7 at most.
recurrence_ref.py's bounds of states hold for any g_min (their term eps |1 - e^g| |h| is larger than
ABS |h| wherever e^g is small: eps = 2^-22 (6 + |u| + |i|)).  Its bound of dz takes e^g as exact to eps of
itself, which holds down to e^-5; so here dz's has the term of ABS beside it:
    |l| e^A (1 - s(u)) |g| ABS (|h_{t-1}| + 2 (e^g / m) s(i) |x|).
"""
import pytest

pytestmark = pytest.mark.gpu
G_MINS = [-0.01, -0.5, -1.25, -1.3, -2.0, -2.5, -2.6, -7.0, -20.0, -1000.0]


@pytest.fixture(scope="module")
def kda():
    from serving_kda_chunkwise_gb300 import kda as _k
    return _k


def _inputs(seed, lengths, D, dtype, level):
    import torch
    gen = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    T, N = sum(lengths), len(lengths)

    def rand(*s):
        return torch.randn(s, generator=gen)

    lv = level[0] + (level[1] - level[0]) * torch.rand(D, generator=gen)
    s = dict(x=rand(T, D), z=rand(T, D) + lv, i=2 * rand(T, D), dy=rand(T, D))
    s = {n: t.to(dt).cuda() for n, t in s.items()}
    s.update(A=(0.3 * rand(D)).cuda(), h0=rand(N, D).cuda(), dh=rand(N, D).cuda(), lengths=lengths,
             cu=torch.tensor([0] + lengths).cumsum(0).to(torch.int32).cuda())
    return s


def _reference(s, g_min):
    """recurrence_ref.recurrence's pairs, the bounds of dz and dA with the absolute term of e^g."""
    import recurrence_ref as R
    import torch
    ref = R.recurrence(s["x"], s["z"], s["i"], s["A"], g_min, s["h0"], s["lengths"], s["dy"], s["dh"])
    x, z, i, A = (s[n].double() for n in ("x", "z", "i", "A"))
    u = A.exp() * z
    g = g_min * u.sigmoid()
    m = (-torch.expm1(2 * g)).sqrt()
    h = ref["y"][0]
    before, lam = torch.empty_like(h), torch.empty_like(h)
    first = 0
    for n, length in enumerate(s["lengths"]):
        l = s["dh"][n].double()
        for t in range(first + length - 1, first - 1, -1):
            before[t] = s["h0"][n].double() if t == first else h[t - 1]
            l = l + s["dy"][t].double()
            lam[t] = l
            l = g[t].exp() * l
        first += length
    v = torch.where(m > 0, g.exp() / m * i.sigmoid() * x.abs(), 0.0)
    more = lam.abs() * A.exp() * (-u).sigmoid() * g.abs() * (6e-7 + 1e-7 * u.abs()) * (
        before.abs() + 2 * v)
    ref["dz"] = (ref["dz"][0], ref["dz"][1] + more)
    ref["dA"] = (ref["dA"][0], ref["dA"][1] + (more * z.abs()).sum(0))
    return ref


def _check(kda, s, g_min):
    import recurrence_ref as R
    import torch
    edges = kda.recurrence_edges(s["x"])
    args = (s["x"], s["z"], s["i"], s["A"], g_min)
    kw = dict(h0=s["h0"], cu_seqlens=s["cu"])
    y, h = kda.recurrence_fwd(*args, edges=edges, **kw)
    got = kda.recurrence_bwd(*args, s["dy"], dh_out=s["dh"], **kw)
    kept = kda.recurrence_bwd(*args, s["dy"], dh_out=s["dh"], edges=edges, **kw)
    kda.device_status()
    ref = _reference(s, g_min)
    R.near(y, ref["y"], "y")
    R.near(h, ref["h"], "h")
    R.near(edges, ref["edges"], "edges")
    for n, k in (("dx", "dx"), ("dz", "dz"), ("di", "di"), ("dA", "dA_log"), ("dh0", "dh0")):
        R.near(got[k], ref[n], n)
        assert torch.equal(got[k], kept[k]), k


LEVELS = [(-7.0, 1.0), (-14.0, -9.0), (3.0, 9.0), (-60.0, -30.0)]


@pytest.mark.parametrize("level", LEVELS)
@pytest.mark.parametrize("g_min", G_MINS)
def test_decays(kda, g_min, level):
    """Over warps, tiles and the tiles of a cluster: 700 tokens; a short sequence and one behind it."""
    _check(kda, _inputs(31, [700, 33, 1], 72, "f32", level), g_min)


@pytest.mark.parametrize("g_min", G_MINS)
def test_decays_bf16(kda, g_min):
    _check(kda, _inputs(32, [0, 300, 150], 72, "bf16", (-12.0, 2.0)), g_min)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("g_min", G_MINS)
def test_packed_inputs(kda, g_min, dtype):
    import recurrence_ref as R
    import torch
    s = _inputs(33, [150, 0, 1, 200], 136, dtype, (-7.0, 1.0))
    kept = [kda.checkpoint_pack(s[n]) for n in ("x", "z", "i")]
    kw = dict(h0=s["h0"], dh_out=s["dh"], cu_seqlens=s["cu"])
    got = kda.recurrence_bwd(*kept, s["A"], g_min, s["dy"], **kw)
    s.update(zip("xzi", (kda.checkpoint_unpack(*k, s["x"].dtype) for k in kept)))
    ref = _reference(s, g_min)
    for n, k in (("dx", "dx"), ("dz", "dz"), ("di", "di"), ("dA", "dA_log"), ("dh0", "dh0")):
        R.near(got[k], ref[n], n)
    whole = kda.recurrence_bwd(s["x"], s["z"], s["i"], s["A"], g_min, s["dy"], **kw)
    for n in got:
        assert torch.equal(got[n], whole[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("g_min", G_MINS)
def test_step(kda, g_min, dtype):
    import recurrence_ref as R
    import torch
    s = _inputs(34, [1] * 64, 200, dtype, (-12.0, 4.0))
    pool = s["h0"].clone()
    y = kda.recurrence_step(s["x"], s["z"], s["i"], s["A"], g_min, pool)
    ref = R.recurrence(s["x"], s["z"], s["i"], s["A"], g_min, s["h0"], s["lengths"])
    R.near(y, ref["y"], "y")
    R.near(pool, ref["h"], "pool")


@pytest.mark.parametrize("g_min", [*G_MINS, -1.0, -3.0, -5.0, -6.0, -1e4])
def test_exactness_of_a_gate(kda, g_min):
    """The two statements, for 2^19 gates with |e^A z| up to 80.  A step from a state of one that takes
    nothing in (x = 0) leaves e^g, rounded; one from a state of zero that takes in all of x = 1 leaves
    the root m of (1 - e^g) (1 + e^g), off by half of REL and 2^-22 (its own) + 2^-24 (the square's) +
    2^-23 (two products) more: 4.2e-7; less where e^g is small, whose error is ABS then and not m's."""
    import torch
    N, D = 8192, 64
    gen = torch.Generator(device="cuda").manual_seed(35)
    A = torch.linspace(-1.2, 1.2, D, device="cuda")
    u = torch.rand(N, D, generator=gen, device="cuda") * 100 - 80
    u[: N // 2] = torch.rand(N // 2, D, generator=gen, device="cuda") * 16 - 12
    z = u / A.exp()
    one, zero, inf = torch.ones_like(z), torch.zeros_like(z), torch.full_like(z, float("inf"))
    a = kda.recurrence_step(zero, z, zero, A, g_min, one.clone()).double()
    m = kda.recurrence_step(one, z, inf, A, g_min, zero.clone()).double()
    u = A.double().exp() * z.double()
    g = torch.tensor(g_min, dtype=torch.float32).double().cuda() * u.sigmoid()
    want = g.exp()
    rel, ab = 1e-6 + 2.6e-7 * u.abs(), 6e-7 + 1e-7 * u.abs()
    over = ((a - want).abs() - 2.0 ** -24 * want) / ab
    assert float(over.max()) <= 1.0, float(over.max())
    want_m = (-torch.expm1(2 * g)).sqrt()
    seen = want_m > 1e-16  # (below, its square is next to the smallest normal number)
    over = ((m - want_m).abs() / want_m / (0.5 * rel + 4.2e-7))[seen]
    assert float(over.max()) <= 1.0, float(over.max())
