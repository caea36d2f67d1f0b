"""Blocks with the gated channel recurrence on a residual stream, from a packed batch of prompts to
single tokens and back through a training step:

    x (normed) --W_in--> x, z, i, gate
        -> recurrence_fwd        prompts; the final states go to the requests' slots of a pool
           recurrence_step       one token of every request, states updated in the pool
        --W_out--> y
        -> block_norm            post-norm, gate and scale, residual, the next block's norm
    training: the inputs x, z, i are kept in 8 bits (checkpoint_pack); the gradients come back through
        block_norm_bwd and recurrence_bwd, which reads them as they were kept

    python examples/recurrent_block.py       # needs a CUDA GPU and the built library
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from serving_kda_chunkwise_gb300 import kda  # noqa: E402

G_MIN, EPS = -5.0, 1e-6


class Block:
    """What a block keeps: projections, decay rates, norm weights and the residual's scale."""

    def __init__(self, D, dtype, gen):
        def rand(*shape, scale=1.0):
            return torch.randn(shape, generator=gen, device="cuda") * scale

        self.D = D
        self.w_in = rand(D, 4 * D, scale=D ** -0.5).to(dtype)
        self.w_out = rand(D, D, scale=D ** -0.5).to(dtype)
        self.A_log = rand(D, scale=0.3)
        self.bias = torch.rand(D, generator=gen, device="cuda").mul(-4.0).to(dtype)  # of z: memory
        self.norm = dict(scale=0.5 + rand(D, scale=0.1), w_post=1 + rand(D, scale=0.1),
                         w_pre=1 + rand(D, scale=0.1), eps=EPS)

    def project(self, x):
        """x, z, i as views of the fused projection's output, and the gate."""
        p = x @ self.w_in
        D = self.D
        p[:, D:2 * D] += self.bias
        return p[:, :D], p[:, D:2 * D], p[:, 2 * D:3 * D], p[:, 3 * D:].contiguous()

    def prompts(self, x, r, cu_seqlens, kept=None, in_8_bits=True):
        """(the next block's input, the residual, final states); kept: what the gradients need."""
        *inputs, gate = self.project(x)
        edges = None if kept is None or in_8_bits else kda.recurrence_edges(inputs[0])
        h, states = kda.recurrence_fwd(*inputs, self.A_log, G_MIN, cu_seqlens=cu_seqlens,
                                       edges=edges)
        y = h @ self.w_out
        r, out = kda.block_norm(y, r, gate=gate, **self.norm)
        if kept is not None:
            if in_8_bits:
                inputs = [kda.checkpoint_pack(t) for t in inputs]
            kept.append((x, inputs, edges, h, y, gate, r))
        return out, r, states

    def step(self, x, r, pool, slots):
        """The same for one token a request, the pool's states updated in place."""
        *inputs, gate = self.project(x)
        h = kda.recurrence_step(*inputs, self.A_log, G_MIN, pool, slots=slots)
        r, out = kda.block_norm(h @ self.w_out, r, gate=gate, **self.norm)
        return out, r

    def gradients(self, kept, dx, dr, cu_seqlens):
        """For gradients on the two outputs of prompts(): those of its inputs and of the weights."""
        x, inputs, edges, h, y, gate, r = kept
        n = kda.block_norm_bwd(y, r, dx, dr, gate=gate, **self.norm)
        g = kda.recurrence_bwd(*inputs, self.A_log, G_MIN, n["dy"] @ self.w_out.t(),
                               cu_seqlens=cu_seqlens, edges=edges, want_dh0=False)
        dp = torch.cat([g["dx"], g["dz"], g["di"], n["dgate"]], 1)
        weights = dict(w_in=x.t() @ dp, w_out=h.t() @ n["dy"], A_log=g["dA_log"],
                       bias=g["dz"].sum(0), scale=n["dscale"], w_post=n["dw_post"],
                       w_pre=n["dw_pre"])
        return dp @ self.w_in.t(), n["dr"], weights


def model(D=256, blocks=2, dtype=torch.bfloat16, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [Block(D, dtype, gen) for _ in range(blocks)]


def train_step(net, x, r, cu_seqlens, dx, dr, in_8_bits=True):
    """Outputs of a whole batch and, for gradients on them, those of the inputs and the weights."""
    kept = []
    for b in net:
        x, r, _ = b.prompts(x, r, cu_seqlens, kept, in_8_bits)
    out, grads = (x, r), []
    for b, k in zip(reversed(net), reversed(kept)):
        dx, dr, w = b.gradients(k, dx, dr, cu_seqlens)
        grads.append(w)
    return out, dx, dr, grads[::-1]


def demo(lengths=(300, 45, 1024), new_tokens=3, D=256, dtype=torch.bfloat16, seed=0):
    """Prompts then single tokens, against the whole sequences in one call: the largest difference of
    the outputs and of the states, relative to their rms."""
    net = model(D, 2, dtype, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    N, ends = len(lengths), [n + new_tokens for n in lengths]

    def offsets(sizes):
        return torch.tensor([0, *torch.tensor(sizes).cumsum(0).tolist()], dtype=torch.int32).cuda()

    def run(x, r, cu, pools, slots):
        for b, pool in zip(net, pools):
            x, r, states = b.prompts(x, r, cu)
            pool[slots.long()] = states
        return x

    cu_all, cu = offsets(ends), offsets(lengths)
    x, r = (torch.randn(sum(ends), D, generator=gen, device="cuda").to(dtype) for _ in range(2))
    slots = torch.randperm(N + 2, generator=gen, device="cuda")[:N].to(torch.int32)
    pools, want = ([torch.zeros(N + 2, D, device="cuda") for _ in net] for _ in range(2))
    whole = run(x, r, cu_all, want, slots)
    first = cu_all[:-1].tolist()
    rows = torch.cat([torch.arange(b, b + n) for b, n in zip(first, lengths)]).cuda()
    got = torch.empty_like(whole)
    got[rows] = run(x[rows], r[rows], cu, pools, slots)
    for i in range(new_tokens):
        at = torch.tensor([b + n + i for b, n in zip(first, lengths)], device="cuda")
        xs, rs = x[at], r[at]
        for b, pool in zip(net, pools):
            xs, rs = b.step(xs, rs, pool, slots)
        got[at] = xs
    kda.device_status()
    rms = whole.float().square().mean().sqrt()
    off = float((got.float() - whole.float()).abs().max() / rms)
    state = max(float((a - b).abs().max() / b.square().mean().sqrt()) for a, b in zip(pools, want))
    return off, state


if __name__ == "__main__":
    off, state = demo()
    print(f"prompts then single tokens against one call: outputs within {off:.1e} of their rms, "
          f"states within {state:.1e}")
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, r, dx, dr = (torch.randn(1500, 256, generator=gen, device="cuda").bfloat16()
                    for _ in range(4))
    cu = torch.tensor([0, 700, 701, 1500], dtype=torch.int32, device="cuda")
    exact, kept = (train_step(model(), x, r, cu, dx, dr, in_8_bits=b)[3] for b in (False, True))
    for i, (a, b) in enumerate(zip(exact, kept)):
        for n in a:
            d = (a[n].float() - b[n].float()).norm() / a[n].float().norm()
            print(f"block {i} d{n:7s} {str(tuple(a[n].shape)):12s} from 8-bit inputs within {d:.1e}")
