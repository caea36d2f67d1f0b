"""States of bf16 inputs are fp32 results: S_out and dS0 within 1e-6 of 64 bits (2-norm), however long
the sequence and however weak the decay.

A product of two bf16 numbers is exact in fp32; each decay carries about 2e-7 (2^x to 2^-22),
different for every token. A tensor core's addition truncates, 4.3e-8 of the sum in the mean,
towards zero; a segment of 2,048 tokens is 128 such additions in turns to three accumulators, 43
each, at which a sum of random terms has half its final size in the mean square: 43 / 2 * 4.3e-8 =
9e-7 where nothing decays, less where it does. Segments are joined by rounding fp32 operations
(6e-8 each, either way)."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,g", [(65536, 4, 0.0), (65536, 4, -0.001), (8192, 16, -0.003),
                                   (2000, 8, -0.01), (300, 2, -0.05), (130, 2, -1.0)])
@pytest.mark.parametrize("per_token", [True, False])
def test_states(T, H, g, per_token):
    import torch
    from serving_kda_chunkwise_gb300 import kda
    d = 128
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k, v, do = (torch.randn(T, H, d, generator=gen, device="cuda") for _ in range(4))
    q, k = (x / x.norm(dim=-1, keepdim=True) for x in (q, k))
    q, k, v, do = (x.bfloat16() for x in (q, k, v, do))
    S0, dS = (torch.randn(1, H, d, d, generator=gen, device="cuda") for _ in range(2))
    if per_token:
        g = g * 2 * torch.rand(T, H, generator=gen, device="cuda")
    else:
        g = torch.full((H,), g, device="cuda")
    G = g.double().expand(T, H).cumsum(0)
    after, upto = (G[-1] - G).exp()[..., None], G.exp()[..., None]
    ref = torch.einsum("thk,thv->hkv", k.double() * after, v.double())
    ref += G[-1].exp()[:, None, None] * S0[0].double()
    refD = torch.einsum("thk,thv->hkv", q.double() * upto, do.double())
    refD += G[-1].exp()[:, None, None] * dS[0].double()
    _, S = kda.linear_fwd_chunked(q, k, v, g, S0=S0)
    in_place = S0.clone()
    kda.linear_fwd_chunked(q, k, v, g, S0=in_place, S_out=in_place)
    dS0 = kda.linear_bwd(q, k, v, g, do, S0=S0, dS_out=dS)["dS0"]
    kda.device_status()
    assert float((S[0] - ref).norm()) <= 1e-6 * float(ref.norm())
    assert float((dS0[0] - refD).norm()) <= 1e-6 * float(refD.norm())
    assert bool((in_place == S).all())


def test_in_place_among_others():
    """S_out in S0's place where some sequences are longer than a segment, some empty, some short."""
    import torch
    from serving_kda_chunkwise_gb300 import kda
    lengths, H, d = [900, 0, 17, 2500, 128, 0, 300], 16, 64
    gen = torch.Generator(device="cuda").manual_seed(6)
    T, N = sum(lengths), len(lengths)
    q, k, v = (torch.randn(T, H, d, generator=gen, device="cuda").bfloat16() for _ in range(3))
    g = -0.1 * torch.rand(T, H, generator=gen, device="cuda")
    S0 = torch.randn(N, H, d, d, generator=gen, device="cuda")
    cu = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32).cuda()
    o, S = kda.linear_fwd_chunked(q, k, v, g, S0=S0, cu_seqlens=cu)
    same = S0.clone()
    o2, S2 = kda.linear_fwd_chunked(q, k, v, g, S0=same, S_out=same, cu_seqlens=cu)
    o3, none = kda.linear_fwd_chunked(q, k, v, g, S0=S0, cu_seqlens=cu, want_state=False)
    kda.device_status()
    assert S2 is same and torch.equal(S, S2) and torch.equal(o, o2)
    assert none is None and torch.equal(o, o3) and torch.equal(S[[1, 5]], S0[[1, 5]])
