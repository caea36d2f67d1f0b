"""The linear attention over many sequences of all sizes, empty, shorter and longer than a
segment: more work items than CTAs (each takes several, some at a time), edge states of few
sequences among many, and blocks of the edges' kernel that look at several.  Tolerances as in
test_gpu_linear."""
import pytest

from test_gpu_linear import _inputs, _near

pytestmark = pytest.mark.gpu


def _lengths(seed, n, longest, tokens):
    """n lengths: a third empty, most up to 9 tokens, the rest of `tokens` in a few long ones."""
    import random
    r = random.Random(seed)
    x = [0 if r.random() < 0.33 else r.randint(1, 9) for _ in range(n)]
    rest = tokens - sum(x)
    while rest > 0:
        i, k = r.randrange(n), min(rest, r.randint(longest // 2, longest))
        x[i] += k
        rest -= k
    return x


CASES = [  # sequences, longest, tokens, heads, dk, dv
    (300, 500, 2600, 16, 128, 64), (300, 2500, 9000, 32, 64, 128), (40, 300, 1200, 5, 128, 128)]


@pytest.fixture(scope="module")
def kda():
    from serving_kda_chunkwise_gb300 import kda as _k
    return _k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("n,longest,tokens,H,dk,dv", CASES)
def test_forward_and_gradients(kda, dtype, state, n, longest, tokens, H, dk, dv):
    import linear_ref
    lengths = _lengths(n + tokens, n, longest, tokens)
    x = _inputs(31, lengths, H, dk, dv, dtype, state=state, decay=0.05)
    args = dict(S0=x["S0"], cu_seqlens=x["cu"])
    o, S = kda.linear_fwd_chunked(x["q"], x["k"], x["v"], x["g"], **args)
    o2, none = kda.linear_fwd_chunked(x["q"], x["k"], x["v"], x["g"], want_state=False, **args)
    got = kda.linear_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], dS_out=x["dS"], **args)
    no = kda.linear_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], dS_out=x["dS"], want_dg=False,
                        want_dS0=False, **args)
    dS0 = kda.linear_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], dS_out=x["dS"], want_dS0=False,
                         **args)
    kda.device_status()
    ro, rS = linear_ref.forward(x["q"], x["k"], x["v"], x["g"], x["S0"], lengths)
    _near(o, ro, "o")
    _near(S, rS, "S")
    assert none is None and bool((o == o2).all())
    ref = linear_ref.gradients(x["q"], x["k"], x["v"], x["g"], x["do"], x["S0"], x["dS"], lengths)
    for name in ("dq", "dk", "dv", "dg", "dS0"):
        _near(got[name], ref[name], name)
    for name in ("dq", "dk", "dv"):
        _near(no[name], ref[name], name)
        assert bool((got[name] == dS0[name]).all())
    assert bool((got["dg"] == dS0["dg"]).all()) and no["dg"] is None and dS0["dS0"] is None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_reset_gradients(kda, dtype):
    """The decays' gradients around exact resets (g = -inf): those tokens' own are zero."""
    import linear_ref
    import torch
    x = _inputs(32, [400, 131], 2, 128, 128, dtype)
    at = [0, 5, 127, 128, 250, 399, 400, 530] + list(range(300, 310))
    x["g"][at] = -float("inf")
    got = kda.linear_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], S0=x["S0"], dS_out=x["dS"],
                         cu_seqlens=x["cu"])["dg"]
    ref = linear_ref.gradients(x["q"], x["k"], x["v"], x["g"], x["do"], x["S0"], x["dS"],
                               x["lengths"])["dg"]
    _near(got, ref, "dg")
    assert float(ref[at].abs().max()) == 0.0
    # sums that should end at zero: 13 roundings of terms of dg's size, as in the other tests
    rms = ref.square().mean(0).sqrt()
    assert bool((got[at].double().abs() <= 1e-3 * rms).all())
