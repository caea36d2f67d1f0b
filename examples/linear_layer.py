"""A linear-attention layer with one decay per head, between its projections, from a packed batch
of prompts to single tokens and back through a training step:

    queries, keys (views of the fused projection)
        -> qk_norm_rope          norm of every head, rotation by position
        -> linear_fwd_chunked    prompts; the final states go to the requests' slots of a pool
           linear_decode_step    one token of every request, states updated in the pool
        -> output_norm_gate      the gated, normalised output
    training: output gradient -> linear_bwd -> qk_norm_rope_bwd

    python examples/linear_layer.py          # needs a CUDA GPU and the built library
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from serving_kda_chunkwise_gb300 import kda  # noqa: E402


class LinearLayer:
    """What such a layer keeps: norm weights, the rotation table and the decay's parameters."""

    def __init__(self, heads, d, rot_dim, max_pos, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.H, self.d = heads, d
        # heads of length about 1: an RMS norm with weights near 1 / sqrt(d)
        self.wq, self.wk = ((1 + 0.1 * torch.randn(d, generator=gen, device=device))
                            / math.sqrt(d) for _ in range(2))
        self.w_out = 1 + 0.1 * torch.randn(d, generator=gen, device=device)
        self.slope = torch.exp2(-8.0 * torch.arange(1, heads + 1, device=device) / heads)
        f = 1e4 ** (-torch.arange(rot_dim // 2, device=device) * 2.0 / rot_dim)
        a = torch.arange(max_pos, device=device)[:, None] * f
        self.cos_sin = torch.cat([a.cos(), a.sin()], 1)

    def split(self, x):
        """Queries, keys, values and output gates out of one projection [T, 4 H d], as views."""
        return [t.unflatten(1, (self.H, self.d)) for t in x.chunk(4, dim=1)]

    def decay(self, z):
        """Log decays [T, H] from the layer's logits."""
        return -self.slope * torch.nn.functional.softplus(z.float())

    def attend(self, x, z, positions, cu_seqlens, S0=None):
        q, k, v, gate = self.split(x)
        qn, kn = kda.qk_norm_rope(q, k, self.wq, self.wk, cos_sin=self.cos_sin,
                                  positions=positions)
        g = self.decay(z)
        o, S = kda.linear_fwd_chunked(qn, kn, v, g, S0=S0, cu_seqlens=cu_seqlens)
        return (qn, kn, v, g, gate.contiguous()), o, S

    def prompts(self, x, z, positions, cu_seqlens, pool, slots):
        """y [T, H, d] of packed prompts; each request's final state into its slot."""
        (*_, gate), o, S = self.attend(x, z, positions, cu_seqlens)
        pool[slots.long()] = S
        return kda.output_norm_gate(o, gate, self.w_out)

    def step(self, x, z, positions, pool, slots):
        """y [N, H, d] of one token a request, the pool's states updated in place."""
        q, k, v, gate = self.split(x)
        qn, kn = kda.qk_norm_rope(q, k, self.wq, self.wk, cos_sin=self.cos_sin,
                                  positions=positions)
        o = kda.linear_decode_step(qn, kn, v, self.decay(z), pool, slots=slots)
        return kda.output_norm_gate(o, gate.contiguous(), self.w_out)

    def gradients(self, x, z, positions, cu_seqlens, do):
        """For a gradient do on the attention's output: those of q, k, v, the log decays and the
        norm weights."""
        q, k, *_ = self.split(x)
        (qn, kn, v, g, _), _, _ = self.attend(x, z, positions, cu_seqlens)
        out = kda.linear_bwd(qn, kn, v, g, do, cu_seqlens=cu_seqlens, want_dS0=False)
        back = kda.qk_norm_rope_bwd(q, k, out["dq"], out["dk"], self.wq, self.wk,
                                    cos_sin=self.cos_sin, positions=positions)
        return dict(dq=back["dq"], dk=back["dk"], dv=out["dv"], dg=out["dg"], dwq=back["dwq"],
                    dwk=back["dwk"])


def demo(lengths=(300, 45, 1024), new_tokens=3, heads=8, d=128, dtype=torch.bfloat16, seed=0):
    """Prompts then single tokens, against the whole sequences in one call; returns the largest
    difference of the outputs, relative to their rms, and a training step's gradients."""
    layer = LinearLayer(heads, d, rot_dim=64, max_pos=max(lengths) + new_tokens, seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    N, ends = len(lengths), [n + new_tokens for n in lengths]

    def packed(sizes):
        cu = torch.tensor([0, *torch.tensor(sizes).cumsum(0).tolist()], dtype=torch.int32)
        pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in sizes])
        return cu.cuda(), pos.cuda()

    cu_all, pos_all = packed(ends)
    x = torch.randn(sum(ends), 4 * heads * d, generator=gen, device="cuda").to(dtype)
    z = torch.randn(sum(ends), heads, generator=gen, device="cuda")
    pool = torch.zeros(N + 2, heads, d, d, device="cuda")
    slots = torch.randperm(N + 2, generator=gen, device="cuda")[:N].to(torch.int32)
    whole = layer.prompts(x, z, pos_all, cu_all, pool, slots)
    states = pool[slots.long()].clone()

    first = cu_all[:-1].tolist()
    rows = torch.cat([torch.arange(b, b + n) for b, n in zip(first, lengths)]).cuda()
    cu, pos = packed(lengths)
    pool.zero_()
    parts = [(rows, layer.prompts(x[rows], z[rows], pos, cu, pool, slots))]
    for i in range(new_tokens):
        at = torch.tensor([b + n + i for b, n in zip(first, lengths)], device="cuda")
        parts.append((at, layer.step(x[at], z[at], pos_all[at], pool, slots)))
    kda.device_status()
    got = torch.empty_like(whole)
    for at, y in parts:
        got[at] = y
    rms = whole.float().square().mean().sqrt()
    off = float((got.float() - whole.float()).abs().max() / rms)
    off_state = float((pool[slots.long()] - states).norm() / states.norm())
    grads = layer.gradients(x, z, pos_all, cu_all, torch.randn_like(whole))
    kda.device_status()
    return off, off_state, grads


if __name__ == "__main__":
    off, off_state, grads = demo()
    print(f"prompts then single tokens against one call: outputs within {off:.1e} of their rms, "
          f"states within {off_state:.1e}")
    for name, t in grads.items():
        print(f"{name:4s} {tuple(t.shape)} {t.dtype} norm {float(t.float().norm()):.3f}")
