"""GPU parity of the query/key norm with position rotation and of its gradients against their
definitions in 64 bits.

Tolerances.  Rows are fp32 throughout with one rounding at the end: bf16 outputs are within
2^-8 relative of the reference plus 1e-5 of the row's rms (the rotation's subtraction can leave an
entry far below the row's size), fp32 outputs within 2e-6 of the row's rms times 4.  The weight
gradients are fp32 sums over rows in a fixed order: 1e-5 in the 2-norm.
"""
import pytest

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def kda():
    from serving_kda_chunkwise_gb300 import kda as _k
    return _k


def _inputs(seed, T, Hq, Hk, d, rot, dtype, weight=True, strided=False):
    import torch
    gen = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32

    def rand(*s):
        return torch.randn(s, generator=gen)

    if strided:
        x = (2 * rand(T, (Hq + 2 * Hk) * d + 16)).to(dt).cuda()
        q = x[:, 8:8 + Hq * d].unflatten(1, (Hq, d))
        k = x[:, 8 + Hq * d:8 + (Hq + Hk) * d].unflatten(1, (Hk, d))
    else:
        q, k = ((2 * rand(T, h, d)).to(dt).cuda() for h in (Hq, Hk))
    wq, wk = ((1 + 0.2 * rand(d)).cuda() for _ in range(2)) if weight else (None, None)
    P = 512
    a = torch.arange(P)[:, None] * torch.exp(-torch.arange(max(rot // 2, 1)) * 0.3)
    cs = torch.cat([a.cos(), a.sin()], 1).float().cuda() if rot else None
    pos = torch.randint(0, P, (T,), generator=gen).to(torch.int32).cuda()
    dyq, dyk = (rand(T, h, d).to(dt).cuda() for h in (Hq, Hk))
    return dict(q=q, k=k, wq=wq, wk=wk, cs=cs, pos=pos, dyq=dyq, dyk=dyk)


def _near(got, ref, name):
    import torch
    if ref.numel() == 0:
        return
    d = (got.double() - ref).abs()
    rms = ref.square().mean(-1, keepdim=True).sqrt()
    tol = 2.0 ** -8 * ref.abs() + 1e-5 * rms if got.dtype == torch.bfloat16 else 8e-6 * (
        rms + ref.abs())
    assert bool((d <= tol).all()), (name, float((d - tol).max()))


def _check(kda, x, d, interleaved):
    import linear_ref
    R = linear_ref.rotation(x["cs"], x["pos"], d, interleaved)
    kw = dict(eps=EPS, cos_sin=x["cs"], positions=x["pos"], interleaved=interleaved)
    yq, yk = kda.qk_norm_rope(x["q"], x["k"], x["wq"], x["wk"], **kw)
    got = kda.qk_norm_rope_bwd(x["q"], x["k"], x["dyq"], x["dyk"], x["wq"], x["wk"], **kw)
    kda.device_status()
    for n, y in (("q", yq), ("k", yk)):
        w = x["w" + n]
        _near(y, linear_ref.norm(x[n], w, EPS, R), n)
        dx, dw = linear_ref.norm_gradients(x[n], x["dy" + n], w, EPS, R)
        _near(got["d" + n], dx, "d" + n)
        if w is None:
            assert got["dw" + n] is None
        elif x[n].numel():
            assert float((got["dw" + n].double() - dw).norm()) <= 1e-5 * float(dw.norm())
        else:
            assert float(got["dw" + n].abs().max()) == 0.0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot", [(64, 0), (64, 16), (64, 48), (64, 64), (128, 32), (128, 96),
                                   (128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_matches_definition(kda, dtype, d, rot, interleaved):
    _check(kda, _inputs(1, 37, 5, 2, d, rot, dtype), d, interleaved)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hq,Hk,weight,strided", [
    (1, 1, 1, True, False), (1, 32, 8, False, True), (3, 9, 0, True, False),
    (1000, 16, 16, True, False), (513, 7, 3, True, True), (0, 4, 2, True, False)])
def test_shapes(kda, dtype, T, Hq, Hk, weight, strided):
    _check(kda, _inputs(2, T, Hq, Hk, 128, 64, dtype, weight, strided), 128, False)


def test_in_place_and_default_positions(kda):
    import torch
    x = _inputs(3, 300, 4, 2, 128, 128, "bf16")
    pos = torch.arange(300, dtype=torch.int32, device="cuda")
    yq, yk = kda.qk_norm_rope(x["q"], x["k"], x["wq"], x["wk"], EPS, x["cs"], pos)
    q, k = x["q"].clone(), x["k"].clone()
    kda.qk_norm_rope(q, k, x["wq"], x["wk"], EPS, x["cs"], q_out=q, k_out=k)
    assert torch.equal(q, yq) and torch.equal(k, yk)


def test_zero_rows_and_special_values(kda):
    """A row of zeros gives zeros (its gradient is finite); a row with an infinity or a NaN
    spoils itself only."""
    import torch
    x = _inputs(4, 6, 2, 2, 64, 64, "f32")
    x["q"][1] = 0.0
    clean, _ = kda.qk_norm_rope(x["q"], x["k"], x["wq"], x["wk"], EPS, x["cs"], x["pos"])
    assert float(clean[1].abs().max()) == 0.0
    out = kda.qk_norm_rope_bwd(x["q"], x["k"], x["dyq"], x["dyk"], x["wq"], x["wk"], EPS, x["cs"],
                               x["pos"])
    assert bool(torch.isfinite(out["dq"]).all()) and bool(torch.isfinite(out["dwq"]).all())
    x["q"][3, 1, 7] = float("inf")
    x["q"][4, 0, 2] = float("nan")
    y, _ = kda.qk_norm_rope(x["q"], x["k"], x["wq"], x["wk"], EPS, x["cs"], x["pos"])
    assert bool(y[4, 0].isnan().all())
    keep = torch.ones(6, 2, dtype=torch.bool)
    keep[3, 1] = keep[4, 0] = False
    assert torch.equal(y[keep.cuda()], clean[keep.cuda()])


def test_bad_position_is_reported(kda):
    import torch
    x = _inputs(5, 8, 2, 1, 64, 32, "f32")
    pos = x["pos"].clone()
    pos[3] = 512
    y, _ = kda.qk_norm_rope(x["q"], x["k"], None, None, EPS, x["cs"], pos)
    with pytest.raises(kda.KdaError) as e:
        kda.device_status()
    assert e.value.status == kda.KDA_ERR_DEVICE and "position" in str(e.value)
    plain, _ = kda.qk_norm_rope(x["q"], x["k"], None, None, EPS)
    assert torch.equal(y[3], plain[3])
    good, _ = kda.qk_norm_rope(x["q"], x["k"], None, None, EPS, x["cs"], x["pos"])
    keep = [i for i in range(8) if i != 3]
    assert torch.equal(y[keep], good[keep])


def test_gradient_against_differences(kda):
    import linear_ref
    import torch
    x = _inputs(6, 20, 3, 2, 64, 32, "f32")
    R = linear_ref.rotation(x["cs"], x["pos"], 64, True)
    got = kda.qk_norm_rope_bwd(x["q"], x["k"], x["dyq"], x["dyk"], x["wq"], x["wk"], EPS, x["cs"],
                               x["pos"], interleaved=True)
    e = 1e-5
    for n in ("q", "k"):
        def loss(a, w):
            return float((linear_ref.norm(a, w, EPS, R) * x["dy" + n].double()).sum())

        a, w = x[n].double(), x["w" + n].double()
        u, z = torch.randn_like(a), torch.randn_like(w)
        dx = (loss(a + e * u, w) - loss(a - e * u, w)) / (2 * e)
        dw = (loss(a, w + e * z) - loss(a, w - e * z)) / (2 * e)
        for diff, grad, by in ((dx, got["d" + n], u), (dw, got["dw" + n], z)):
            t = grad.double() * by
            assert abs(diff - float(t.sum())) <= 1e-4 * float(t.norm()) + 1e-6 * abs(diff)


def test_deterministic(kda):
    import torch
    x = _inputs(7, 5000, 8, 2, 128, 64, "bf16")
    a, b = (kda.qk_norm_rope_bwd(x["q"], x["k"], x["dyq"], x["dyk"], x["wq"], x["wk"], EPS,
                                 x["cs"], x["pos"]) for _ in range(2))
    for n in a:
        assert torch.equal(a[n], b[n])


def test_binding_refusals(kda):
    import torch
    x = _inputs(8, 10, 2, 1, 64, 32, "bf16")
    with pytest.raises(TypeError):
        kda.qk_norm_rope(x["q"], x["k"].float())
    with pytest.raises(ValueError):
        kda.qk_norm_rope(x["q"], x["k"], x["wq"][:32].contiguous())
    with pytest.raises(ValueError):
        kda.qk_norm_rope(x["q"], x["k"], cos_sin=x["cs"], positions=x["pos"][:9])
    with pytest.raises(kda.KdaError) as e:
        kda.qk_norm_rope(x["q"], x["k"], cos_sin=torch.zeros(20, 24, device="cuda"))
    assert e.value.status == kda.KDA_ERR_UNSUPPORTED
    with pytest.raises(kda.KdaError) as e:
        kda.qk_norm_rope(x["q"], x["k"], cos_sin=torch.zeros(9, 32, device="cuda"))
    assert "n_pos" in str(e.value)
    with pytest.raises(kda.KdaError):
        kda.qk_norm_rope(x["q"], x["k"], eps=-1.0)
