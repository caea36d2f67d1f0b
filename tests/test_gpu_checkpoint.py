"""GPU parity of the 8-bit checkpoints: every step of the formula is exact in binary, so codes,
exponents and the values that come back are compared bit by bit with the definition in 64 bits."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    from serving_kda_chunkwise_gb300 import kda as _k
    return _k


def _check(kda, x):
    import recurrence_ref as R
    import torch
    codes, exps = kda.checkpoint_pack(x)
    c, e = R.pack(x)
    assert torch.equal(codes, c) and torch.equal(exps, e)
    ref = R.unpack(c, e)
    for dt in (torch.bfloat16, torch.float32):
        got = kda.checkpoint_unpack(codes, exps, dt)
        assert got.dtype == dt
        assert torch.equal(got.double().nan_to_num(123.0), ref.nan_to_num(123.0))
    return codes, exps


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,D,strided", [(1, 8, False), (3, 64, False), (70, 72, True),
                                         (5, 1000, True), (513, 320, False), (0, 64, False)])
def test_matches_definition(kda, dtype, T, D, strided):
    import torch
    gen = torch.Generator().manual_seed(T + D)
    x = torch.randn(T, D + 16, generator=gen) * torch.exp(3 * torch.randn(T, 1, generator=gen))
    x = x.to(getattr(torch, dtype)).cuda()
    _check(kda, x[:, 8:8 + D] if strided else x[:, :D].contiguous())


def test_borders(kda):
    """Largest magnitudes at and beside the borders of the exponents, halves between codes, the
    ends of the types' ranges, zeros, denormal numbers."""
    import torch
    top = []
    for k in (-149, -140, -133, -130, -127, -126, -121, -120, -10, 0, 1, 60, 119, 120, 121):
        for f in (1.0, 1.5, 127.0 / 64, 127.4999 / 64, 127.5 / 64, 127.5001 / 64, 1.99999):
            top.append(f * 2.0 ** (k + 6) if k > -140 else f * 2.0 ** k)
    top += [0.0, 3.4028234e38, 1e-45]
    x = torch.zeros(len(top), 64, dtype=torch.float64)
    x[:, 17] = torch.tensor(top, dtype=torch.float64)
    ramp = torch.arange(-126, 126, 4.0, dtype=torch.float64) / 128 + 1.0 / 256
    x[:, :17] = ramp[:17] * x[:, 17:18]
    x[:, 18:] = ramp[17:63] * x[:, 17:18]
    x[1::2] *= -1
    x = x.float().cuda()
    assert bool(torch.isfinite(x).all())
    _check(kda, x)
    _check(kda, x.bfloat16().clamp(-3.3e38, 3.3e38))
    halves = torch.zeros(2, 64, device="cuda")
    halves[:, 0] = torch.tensor([64.0, 127.0])
    halves[:, 1:] = torch.arange(63, device="cuda") - 31.5
    codes, _ = _check(kda, halves)
    assert codes[0, 1:5].tolist() == [-32, -30, -30, -28]  # halves to even


def test_not_finite(kda):
    """A group with an infinity or a NaN comes back as NaN, and no other."""
    import torch
    x = torch.randn(4, 200, device="cuda")
    clean = kda.checkpoint_pack(x)
    x[1, 70], x[2, 199], x[3, 0] = float("inf"), float("nan"), -float("inf")
    codes, exps = _check(kda, x)
    assert exps[1, 1] == exps[3, 2] == exps[0, 3] == -128
    back = kda.checkpoint_unpack(codes, exps, torch.float32)
    good = torch.ones(4, 200, dtype=torch.bool, device="cuda")
    good[1, 64:128] = good[2, 192:] = good[3, :64] = False
    assert torch.equal(torch.isfinite(back), good)
    assert torch.equal(codes[good], clean[0][good])


def test_far_rows(kda):
    """Element offsets past 32 bits."""
    import torch
    T, D = (1 << 32) // 4096 + 9, 4096
    x = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, D, device="cuda").bfloat16()
    codes, exps = kda.checkpoint_pack(x)
    c, e = kda.checkpoint_pack(x[-3:])
    assert torch.equal(codes[-3:], c) and torch.equal(exps[:, -3:], e)
    y = kda.checkpoint_unpack(codes, exps)
    assert torch.equal(y[-3:], kda.checkpoint_unpack(c, e))
    assert float(y[:-3].abs().max()) == 0.0


def test_refusals(kda):
    import torch
    x = torch.randn(6, 64, device="cuda")
    codes, exps = kda.checkpoint_pack(x)
    with pytest.raises(TypeError):
        kda.checkpoint_pack(x.half())
    with pytest.raises(ValueError):
        kda.checkpoint_pack(x.t())
    with pytest.raises(ValueError):
        kda.checkpoint_pack(x[None])
    with pytest.raises(ValueError):
        kda.checkpoint_unpack(codes, exps[:, :5])
    with pytest.raises(TypeError):
        kda.checkpoint_unpack(codes.float(), exps)
    with pytest.raises(TypeError):
        kda.checkpoint_unpack(codes, exps, torch.float16)
    for D in (60, 4):
        with pytest.raises(kda.KdaError) as e:
            kda.checkpoint_pack(x[:, :D].contiguous())
        assert e.value.status == kda.KDA_ERR_UNSUPPORTED
