"""GPU parity of the norms around a block and of their gradients against the definition in 64 bits.

Tolerances.  Every value is fp32 arithmetic rounded once.  The sums over a row's D channels are of
positive terms (the norms) or enter as a correction, and are off by at most 2^-20 relative of the sum
of their magnitudes (lanes add at most 64 terms one after the other, then a tree); sigmoid and rsqrt
by 2^-21.  So a result is within 2^-18 of the sum S of its terms' magnitudes (r' = r + added: |r| +
|added|; x' inherits r'; a gradient behind a norm: the row's rms as well), plus half a step of its
type.  Sums over T tokens: 2^-18 of the sum of magnitudes.
"""
import pytest

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def kda():
    from serving_kda_chunkwise_gb300 import kda as _k
    return _k


def _inputs(seed, T, D, dtype="bf16", residual=None, post=True, gate=True, scale=True, w_post=None,
            w_pre=True):
    import torch
    gen = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    rt = torch.bfloat16 if (residual or dtype) == "bf16" else torch.float32

    def rand(*s):
        return torch.randn(s, generator=gen)

    s = dict(y=rand(T, D).to(dt), r=(3 * rand(T, D)).to(rt), gate=(2 * rand(T, D)).to(dt) if gate
             else None, scale=0.5 + 0.2 * rand(D) if scale else None,
             w_post=1 + 0.2 * rand(D) if (post if w_post is None else w_post) else None,
             w_pre=1 + 0.2 * rand(D) if w_pre else None, dx=rand(T, D).to(dt), dr=rand(T, D).to(rt))
    s = {n: None if t is None else t.cuda() for n, t in s.items()}
    s["post"] = post
    return s


def _kw(s):
    return dict(gate=s["gate"], scale=s["scale"], w_post=s["w_post"], w_pre=s["w_pre"],
                post_norm=s["post"], eps=EPS)


def _near(got, ref, size, name):
    import torch
    if ref.numel() == 0:
        return
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    d = (got.double() - ref).abs()
    tol = half * ref.abs() + 2.0 ** -18 * size + 1e-30
    assert bool((d <= tol).all()), (name, float((d - tol).max()))


def _check(kda, s):
    import recurrence_ref as R
    args = (s["gate"], s["scale"], s["w_post"], s["w_pre"], s["post"], EPS)
    r, x = kda.block_norm(s["y"], s["r"], **_kw(s))
    ref_r, ref_x = R.block_norm(s["y"], s["r"], *args)
    size = s["r"].double().abs() + (ref_r - s["r"].double()).abs()
    _near(r, ref_r, size, "r")
    rms = (ref_r.square().mean(-1, keepdim=True) + EPS).sqrt()
    w = 1.0 if s["w_pre"] is None else s["w_pre"].double().abs()
    _near(x, ref_x, size / rms * w, "x")

    got = kda.block_norm_bwd(s["y"], r, s["dx"], s["dr"], **_kw(s))
    kda.device_status()
    ref = R.block_norm_gradients(s["y"], r, s["dx"], s["dr"], *args)
    if r.numel() == 0:
        for n in ("dscale", "dw_post", "dw_pre"):
            assert ref[n] is None or float(got[n].abs().max()) == 0.0
        return
    rr = (r.double().square().mean(-1, keepdim=True) + EPS).sqrt()
    u = s["dx"].double().abs() * w / rr
    size = (0.0 if s["dr"] is None else s["dr"].double().abs()) + u + u.square().mean(
        -1, keepdim=True).sqrt() * (1 + (r.double() / rr).abs())
    _near(got["dr"], ref["dr"], size, "dr")
    f = 1.0 if s["gate"] is None else s["gate"].double().sigmoid()
    f = f if s["scale"] is None else f * s["scale"].double().abs()
    yd = s["y"].double()
    ry = (yd.square().mean(-1, keepdim=True) + EPS).sqrt() if s["post"] else 1.0
    wp = 1.0 if s["w_post"] is None else s["w_post"].double().abs()
    dn = size * f
    n = (yd / ry).abs()
    v = dn * wp / ry
    if s["post"]:
        v = v + v.square().mean(-1, keepdim=True).sqrt() * (1 + n)
    _near(got["dy"], ref["dy"], v, "dy")
    if s["gate"] is None:
        assert got["dgate"] is None
    else:
        _near(got["dgate"], ref["dgate"], dn * n * wp, "dgate")
    f = 1.0 if s["gate"] is None else s["gate"].double().sigmoid()
    sums = dict(dscale=size * f * n * wp, dw_post=dn * n,
                dw_pre=(s["dx"].double() * r.double() / rr).abs())
    for nm, terms in sums.items():
        if ref[nm] is None:
            assert got[nm] is None
        else:
            _near(got[nm], ref[nm], terms.sum(0), nm)


TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


@pytest.mark.parametrize("dtype,residual", TYPES)
@pytest.mark.parametrize("D", [8, 64, 72, 256, 1000, 1032, 2048, 4096, 4104, 8192])
def test_widths(kda, dtype, residual, D):
    _check(kda, _inputs(1, 37, D, dtype, residual))


@pytest.mark.parametrize("dtype,residual", TYPES)
@pytest.mark.parametrize("T", [0, 1, 2, 153, 1000])
def test_rows(kda, dtype, residual, T):
    _check(kda, _inputs(2, T, 320, dtype, residual))


@pytest.mark.parametrize("post,w_post", [(True, True), (True, False), (False, False)])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("scale", [True, False])
@pytest.mark.parametrize("w_pre", [True, False])
def test_parts(kda, post, w_post, gate, scale, w_pre):
    for dtype, residual in TYPES:
        _check(kda, _inputs(3, 50, 520, dtype, residual, post, gate, scale, w_post, w_pre))


def test_no_gradient_of_the_residual(kda):
    s = _inputs(4, 40, 256)
    s["dr"] = None
    _check(kda, s)


def test_in_place(kda):
    import torch
    for dtype, residual in TYPES:
        s = _inputs(5, 300, 1032, dtype, residual)
        r, x = kda.block_norm(s["y"], s["r"], **_kw(s))
        y, rr = s["y"].clone(), s["r"].clone()
        r2, x2 = kda.block_norm(y, rr, **_kw(s), r_out=rr, x_out=y)
        assert r2 is rr and x2 is y and torch.equal(r, r2) and torch.equal(x, x2)


def test_special_rows(kda):
    """Rows of zeros are finite throughout; a residual that cancels what is added; gates at their
    ends; a row that is not finite spoils itself only."""
    import torch
    s = _inputs(6, 8, 128, "f32")
    s["y"][1] = 0.0
    s["r"][2] = 0.0
    s["y"][3], s["r"][3] = 0.0, 0.0
    s["gate"][4, ::2], s["gate"][4, 1::2] = float("inf"), -float("inf")
    added = kda.block_norm(s["y"], torch.zeros_like(s["r"]), **_kw(s))[0]
    s["r"][5] = -added[5] * (1 + 2.0 ** -12)
    _check(kda, s)
    clean = kda.block_norm(s["y"], s["r"], **_kw(s))
    for t in clean:
        assert bool(torch.isfinite(t).all())
    grads = kda.block_norm_bwd(s["y"], clean[0], s["dx"], s["dr"], **_kw(s))
    s["y"][6, 3], s["r"][7, 4] = float("nan"), float("inf")
    spoiled = kda.block_norm(s["y"], s["r"], **_kw(s))
    for a, b in zip(clean, spoiled):
        assert torch.equal(a[:6], b[:6])
    again = kda.block_norm_bwd(s["y"], spoiled[0], s["dx"], s["dr"], **_kw(s))
    for n in ("dr", "dy", "dgate"):
        assert torch.equal(grads[n][:6], again[n][:6]), n


def test_gradient_against_differences(kda):
    import recurrence_ref as R
    import torch
    s = _inputs(7, 20, 64, "f32")
    names = ("y", "r", "gate", "scale", "w_post", "w_pre")
    base = [s[n].double() for n in names]
    r, _ = R.block_norm(*base, True, EPS)
    got = kda.block_norm_bwd(s["y"], r.float(), s["dx"], s["dr"], **_kw(s))

    def loss(*args):
        r, x = R.block_norm(*args, True, EPS)
        return float((r * s["dr"]).sum() + (x * s["dx"]).sum())

    e = 1e-5
    for k, n in enumerate(names):
        by = torch.randn_like(base[k])
        up, dn = list(base), list(base)
        up[k], dn[k] = base[k] + e * by, base[k] - e * by
        diff = (loss(*up) - loss(*dn)) / (2 * e)
        t = got["d" + n].double() * by
        assert abs(diff - float(t.sum())) <= 1e-4 * float(t.norm()) + 1e-6 * abs(diff), n


def test_deterministic_and_graph(kda):
    import torch
    s = _inputs(8, 3000, 1000)
    r, x = kda.block_norm(s["y"], s["r"], **_kw(s))
    want = kda.block_norm_bwd(s["y"], r, s["dx"], s["dr"], **_kw(s))
    ws = torch.full((kda.library().kda_block_norm_bwd_workspace_size(1000),), 255,
                    dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r2, x2 = kda.block_norm(s["y"], s["r"], **_kw(s))
        got = kda.block_norm_bwd(s["y"], r2, s["dx"], s["dr"], workspace=ws, **_kw(s))
    for _ in range(3):
        ws.fill_(255)
        graph.replay()
        assert torch.equal(r, r2) and torch.equal(x, x2)
        for n in want:
            assert torch.equal(want[n], got[n]), n


def test_far_rows(kda):
    """Element offsets past 32 bits."""
    import torch
    T, D = (1 << 32) // 4096 + 40, 4096
    gen = torch.Generator(device="cuda").manual_seed(1)
    y, r, dx = (torch.randn(T, D, generator=gen, device="cuda", dtype=torch.bfloat16)
                for _ in range(3))
    a = kda.block_norm(y, r)
    b = kda.block_norm(y[-50:], r[-50:])
    for u, v in zip(a, b):
        assert torch.equal(u[-50:], v)
    g, h = kda.block_norm_bwd(y, a[0], dx), kda.block_norm_bwd(y[-50:], b[0], dx[-50:])
    for n in ("dr", "dy"):
        assert torch.equal(g[n][-50:], h[n])


def test_refusals(kda):
    import torch
    s = _inputs(9, 10, 64)
    with pytest.raises(TypeError):
        kda.block_norm(s["y"], s["r"], gate=s["gate"].float())
    with pytest.raises(ValueError):
        kda.block_norm(s["y"], s["r"][:9])
    with pytest.raises(ValueError):
        kda.block_norm(s["y"], s["r"], scale=s["scale"][:32].contiguous())
    with pytest.raises(ValueError):
        kda.block_norm(s["y"][:, ::2], s["r"][:, ::2])
    with pytest.raises(kda.KdaError):
        kda.block_norm(s["y"], s["r"], eps=-1.0)
    with pytest.raises(kda.KdaError):  # a weight for a norm that is not taken
        kda.block_norm(s["y"], s["r"], w_post=s["w_post"], post_norm=False)
    with pytest.raises(kda.KdaError):  # an fp32 block with a bf16 residual
        kda.block_norm(s["y"].float(), s["r"])
    with pytest.raises(TypeError):
        kda.block_norm_bwd(s["y"], s["r"], s["dx"], s["dr"].float())
    for D in (60, 8200):
        with pytest.raises(kda.KdaError) as e:
            kda.block_norm(*(torch.zeros(2, D, device="cuda") for _ in range(2)))
        assert e.value.status == kda.KDA_ERR_UNSUPPORTED
