"""The decay's gradient of the linear attention, head by head: a head whose decay is strong has a
gradient of the size of e^g, far below the others', so one norm over all heads would not see it.

Tolerances, relative to the head's 2-norm. dg is a running sum over up to 1,024 tokens of the
difference of two dot products, each a sum of terms of dg's own size, pinned to the right value at
both ends; of independent errors of such a sum, sqrt(1024 / 6) = 13 times one term's remains on
average. bf16: a term carries up to three operands held to 2^-17 (2.4e-6 in the mean each, 4e-6
together), two dot products: 13 * 1.4 * 4e-6 = 7.5e-5, taken as 1e-4. fp32: 1e-7 a dot product of
128 terms, 2e-6, and as much again for the running sum in fp32: taken as 1e-5. A fixed decay's
gradient is the sum over T tokens of these: the errors of neighbours are alike, and 1024^1.5 /
sqrt(12) / sqrt(1024) = 300 times a term's remains beside the norm: bf16 300 * 1.4 * 4e-6 = 1.7e-3,
taken as 2e-3; fp32 4e-5, taken as 1e-4."""
import pytest

pytestmark = pytest.mark.gpu

HEADS = [-0.01, -1.0, -3.0, -5.0, -8.0, -10.0, -14.0, -20.0]


def _inputs(seed, lengths, dk, dv, dtype, states):
    import torch
    gen = torch.Generator().manual_seed(seed)
    T, H, N = sum(lengths), len(HEADS), len(lengths)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32

    def rand(*s):
        return torch.randn(s, generator=gen)

    x = dict(q=rand(T, H, dk), k=rand(T, H, dk), v=rand(T, H, dv), do=rand(T, H, dv))
    for n in ("q", "k"):
        x[n] = x[n] / x[n].norm(dim=-1, keepdim=True)
    x = {n: t.to(dt).cuda() for n, t in x.items()}
    x["g"] = torch.tensor(HEADS).cuda()
    x["S0"], x["dS"] = ((0.3 * rand(N, H, dk, dv)).cuda() if states else None for _ in range(2))
    x["cu"] = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()],
                           dtype=torch.int32).cuda()
    return x


def _check(kda, x, lengths, dtype):
    import linear_ref
    T, H = x["q"].shape[:2]
    args = dict(S0=x["S0"], dS_out=x["dS"], cu_seqlens=x["cu"])
    per = kda.linear_bwd(x["q"], x["k"], x["v"], x["g"].expand(T, H).contiguous(), x["do"], **args)
    one = kda.linear_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], **args)
    kda.device_status()
    ref = linear_ref.gradients(x["q"], x["k"], x["v"], x["g"].expand(T, H), x["do"], x["S0"],
                               x["dS"], lengths)
    want = ref["dg"]
    norm = want.norm(dim=0)
    tol, tol_sum = (1e-4, 2e-3) if dtype == "bf16" else (1e-5, 1e-4)
    off = (per["dg"].double() - want).norm(dim=0) / norm
    assert bool((off <= tol).all()), off.tolist()
    off = (one["dg"].double() - want.sum(0)).abs() / norm
    assert bool((off <= tol_sum).all()), off.tolist()
    for n in ("dq", "dk", "dv"):  # the same outputs whichever way dg is asked for
        assert bool((per[n] == one[n]).all())
    return ref, per


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("lengths,dk,dv", [([1024], 128, 128), ([300, 1, 0, 129], 64, 128),
                                           ([128, 700], 128, 64)], ids=str)
def test_head_by_head(kda, dtype, states, lengths, dk, dv):
    _check(kda, _inputs(1, lengths, dk, dv, dtype, states), lengths, dtype)


def test_bf16_token_by_token(kda, monkeypatch):
    monkeypatch.setenv("KDA_FWD_PATH", "generic")
    _check(kda, _inputs(2, [500, 77], 128, 64, "bf16", True), [500, 77], "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_without_it(kda, dtype):
    """dq, dk, dv against the recurrence with and without dg asked for: a token's own term
    reaches them by another way when it is."""
    lengths = [333, 64]
    x = _inputs(3, lengths, 128, 128, dtype, True)
    ref, per = _check(kda, x, lengths, dtype)
    no = kda.linear_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS_out=x["dS"],
                        cu_seqlens=x["cu"], want_dg=False)
    kda.device_status()
    # one rounding of the result (2^-9), and 1e-5 as of all fp32 results here
    tol = 2.0 ** -9 if dtype == "bf16" else 1e-5
    for got in (per, no):
        for n in ("dq", "dk", "dv"):
            off = (got[n].double() - ref[n]).norm(dim=(0, 2)) / ref[n].norm(dim=(0, 2))
            assert bool((off <= tol).all()), (n, off.tolist())
    assert no["dg"] is None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_token_a_reset(kda, dtype):
    """g = -inf everywhere: nothing is kept, and the gradient of every g is exactly zero."""
    import torch
    x = _inputs(4, [200], 64, 64, dtype, True)
    g = torch.full((200, len(HEADS)), -float("inf"), device="cuda")
    out = kda.linear_bwd(x["q"], x["k"], x["v"], g, x["do"], S0=x["S0"], dS_out=x["dS"])
    kda.device_status()
    assert float(out["dg"].abs().max()) == 0.0 and float(out["dS0"].abs().max()) == 0.0


@pytest.fixture(scope="module")
def kda():
    from serving_kda_chunkwise_gb300 import kda as _k
    return _k
