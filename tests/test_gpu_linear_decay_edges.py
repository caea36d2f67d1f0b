"""The decay's gradient across the edges of segments.  It is a running sum inside a segment, pinned at
both ends; if the sums that find out by how much they miss the end are not those that are used, the
difference comes down on a segment's last token.

The step from one token's gradient to the next is one term, a difference of two dot products, whose
error is the same at every place but for its sampling: over 9 edges x 8 heads 8 % in its root mean
square.  So the step across an edge may be off by at most twice the mean step's error."""
import pytest

pytestmark = pytest.mark.gpu


def test_steps_across_edges():
    import linear_ref
    import torch
    from serving_kda_chunkwise_gb300 import kda
    T, H, d, L = 10240, 8, 128, 1024  # long enough for the longest segments
    gen = torch.Generator().manual_seed(3)
    q, k, v, do = (torch.randn(T, H, d, generator=gen) for _ in range(4))
    q, k = (x / x.norm(dim=-1, keepdim=True) for x in (q, k))
    q, k, v, do = (x.bfloat16().cuda() for x in (q, k, v, do))
    g = -(0.3 + 0.3 * torch.rand(T, H, generator=gen)).cuda()
    got = kda.linear_bwd(q, k, v, g, do)["dg"].double()
    kda.device_status()
    ref = linear_ref.gradients(q, k, v, g, do, None, None, [T])["dg"]
    off = (got - ref).diff(dim=0) / ref.square().mean(0).sqrt()
    mean = float(off.square().mean().sqrt())
    at = float(off[L - 1::L].square().mean().sqrt())
    assert at <= 2 * mean, (at, mean)
