"""The recurrent block of examples/recurrent_block.py: prompts followed by single tokens equal the whole
sequences in one call, and a training step's gradients are those of the formulas.

Tolerances.  bf16: both ways make the same roundings but where a state or a product differs in its last
bits; a value then rounds to the neighbour (2^-8), twice (two blocks, each with five roundings in a row,
of values up to 6 times the rms): within 2^-3 of the rms.  fp32: 1e-4 (projections by a library's
products of 2^-13 inputs on tensor cores are off on both sides alike, rows apart by their order).
Gradients in fp32 against 64 bits: 1e-3 in the 2-norm for two blocks.  From 8-bit inputs: an input is
off by half a step, at most 1/127 of its group's largest, which is 4 times the rms at most: 2 % of the
rms on average over three inputs and two blocks; 10 % are allowed.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "recurrent_block.py")
    spec = importlib.util.spec_from_file_location("recurrent_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("dtype,lengths,D", [("bfloat16", (300, 45, 1024), 256),
                                             ("float32", (70, 1), 72)])
def test_prompts_then_tokens(ex, dtype, lengths, D):
    import torch
    off, state = ex.demo(lengths, 3, D, getattr(torch, dtype))
    bound = 2.0 ** -3 if dtype == "bfloat16" else 1e-4
    assert off <= bound and state <= bound


def _formulas(net, x, r, lengths, dx, dr):
    """The two blocks in 64 bits, differentiated."""
    import torch
    leaves, x0, r0 = [], x.double().requires_grad_(True), r.double().requires_grad_(True)
    x, r = x0, r0
    for b in net:
        p = {n: t.double().detach().clone().requires_grad_(True)
             for n, t in dict(w_in=b.w_in, w_out=b.w_out, A_log=b.A_log, bias=b.bias,
                              **{n: b.norm[n] for n in ("scale", "w_post", "w_pre")}).items()}
        leaves.append(p)
        D = b.D
        q = x @ p["w_in"]
        xi, z, i, gate = q[:, :D], q[:, D:2 * D] + p["bias"], q[:, 2 * D:3 * D], q[:, 3 * D:]
        g = -5.0 * torch.sigmoid(p["A_log"].exp() * z)
        u = (-torch.expm1(2 * g)).sqrt() * torch.sigmoid(i) * xi
        hs, t = [], 0
        for n in lengths:
            h = torch.zeros(D, dtype=torch.float64, device=x.device)
            for t in range(t, t + n):
                h = g[t].exp() * h + u[t]
                hs.append(h)
            t += 1
        y = torch.stack(hs) @ p["w_out"]
        y = y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt() * p["w_post"]
        r = r + p["scale"] * torch.sigmoid(gate) * y
        x = r / (r.square().mean(-1, keepdim=True) + 1e-6).sqrt() * p["w_pre"]
    torch.autograd.backward([x, r], [dx.double(), dr.double()])
    return x0.grad, r0.grad, [{n: t.grad for n, t in p.items()} for p in leaves]


def _off(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def test_training_step(ex):
    import torch
    net = ex.model(128, 2, torch.float32)
    lengths = [40, 1, 90]
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, r, dx, dr = (torch.randn(131, 128, generator=gen, device="cuda") for _ in range(4))
    cu = torch.tensor([0, 40, 41, 131], dtype=torch.int32, device="cuda")
    want = _formulas(net, x, r, lengths, dx, dr)
    for in_8_bits, bound in ((False, 1e-3), (True, 0.1)):
        _, gx, gr, grads = ex.train_step(net, x, r, cu, dx, dr, in_8_bits)
        assert _off(gx, want[0]) <= bound and _off(gr, want[1]) <= bound
        for got, ref in zip(grads, want[2]):
            for n in ref:
                assert _off(got[n], ref[n]) <= bound, (in_8_bits, n)


def test_training_step_captured(ex):
    """A whole step, forward and gradients, in a graph, replayed with new inputs."""
    import torch
    net = ex.model(128, 2)
    gen = torch.Generator(device="cuda").manual_seed(4)
    ins = [torch.randn(600, 128, generator=gen, device="cuda").bfloat16() for _ in range(4)]
    cu = torch.tensor([0, 300, 310, 600], dtype=torch.int32, device="cuda")

    def flat(out):
        return [*out[0], out[1], out[2], *(t for g in out[3] for t in g.values())]

    def run():
        return flat(ex.train_step(net, ins[0], ins[1], cu, ins[2], ins[3]))

    run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(2):
        graph.replay()
        for a, b in zip(got, run()):
            assert torch.equal(a, b)
        for t in ins:
            t.mul_(0.75)
