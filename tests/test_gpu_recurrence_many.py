"""The channel recurrence over more states than 2^29 numbers: 131,200 sequences of one token or none x
4096 channels, against the same calls for the last 1,000 of them and against the single-token step.  (What
a sequence of one token gets does not depend on the others, so all are equal bit by bit.)"""
import pytest

pytestmark = pytest.mark.gpu


def test_many_sequences():
    import torch
    from serving_kda_chunkwise_gb300 import kda
    N, D, last = 131200, 4096, 1000
    gen = torch.Generator(device="cuda").manual_seed(41)
    lengths = (torch.rand(N, generator=gen, device="cuda") < 0.9).int()
    cu = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
    cu[1:] = lengths.cumsum(0)
    T = int(cu[-1])
    x, z, i, dy = (torch.randn(T, D, generator=gen, device="cuda", dtype=torch.bfloat16)
                   for _ in range(4))
    h0 = torch.randn(N, D, generator=gen, device="cuda")
    A = 0.3 * torch.randn(D, generator=gen, device="cuda")
    y, h = kda.recurrence_fwd(x, z, i, A, -5.0, h0=h0, cu_seqlens=cu)
    kda.device_status()
    first = int(cu[-1 - last])
    tail = [t[first:] for t in (x, z, i)]
    cu2 = (cu[-1 - last:] - first).contiguous()
    y2, h2 = kda.recurrence_fwd(*tail, A, -5.0, h0=h0[-last:], cu_seqlens=cu2)
    assert torch.equal(y[first:], y2) and torch.equal(h[-last:], h2)
    empty = lengths == 0
    assert torch.equal(h[empty], h0[empty])
    slots = (~empty).nonzero()[:, 0].to(torch.int32)
    pool = h0.clone()
    assert torch.equal(kda.recurrence_step(x, z, i, A, -5.0, pool, slots=slots), y)
    assert torch.equal(pool, h)
    del pool, y
    g = kda.recurrence_bwd(x, z, i, A, -5.0, dy, h0=h0, dh_out=h, cu_seqlens=cu)
    kda.device_status()
    g2 = kda.recurrence_bwd(*tail, A, -5.0, dy[first:], h0=h0[-last:], dh_out=h[-last:],
                            cu_seqlens=cu2)
    for n in ("dx", "dz", "di"):
        assert torch.equal(g[n][first:], g2[n]), n
    assert torch.equal(g["dh0"][-last:], g2["dh0"]) and torch.equal(g["dh0"][empty], h[empty])
