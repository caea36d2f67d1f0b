"""What a call of the binding allocates for itself when it is given a stream: the workspace and the
outputs must be of that stream's memory (the workspace is dropped when the call returns, while its
kernels may still be queued), and the outputs kept from reuse while the caller's stream reads them.

On the CPU: tensors that say they are on the device, a library that does nothing, and streams of
which only the current one is known.  On the GPU: results while the default stream takes and
overwrites whatever memory it is given."""
import contextlib

import pytest
import torch

T, H, D = 6, 2, 64


class OnDevice(torch.Tensor):
    is_cuda = True


def tensor(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


class Nothing:
    """Entry points that succeed; sizes of a workspace that is needed."""

    def __getattr__(self, name):
        return lambda *args: 64 if name.endswith("_size") else 0


def calls(kda):
    f32 = torch.float32
    q, k, v, z, gate = (tensor(T, H, D) for _ in range(5))
    beta, A, g = tensor(T, H), tensor(H, dtype=f32), tensor(T, H, dtype=f32)
    S, w = tensor(T, H, D, D, dtype=f32), tensor(D, dtype=f32)
    scores, bias = tensor(8, 4, dtype=f32), tensor(4, dtype=f32)
    return dict(
        gate=lambda s: kda.gate(z, A, -5.0, stream=s),
        fwd=lambda s: kda.fwd_chunked(q, k, v, beta, z, A, -5.0, stream=s),
        softplus=lambda s: kda.fwd_chunked_softplus(q, k, v, beta, z, A, stream=s),
        bwd=lambda s: kda.bwd(q, k, v, beta, z, A, -5.0, v, stream=s),
        step=lambda s: kda.decode_step(q, k, v, beta, z, A, -5.0, S, stream=s),
        norm_gate=lambda s: kda.output_norm_gate(v, gate, stream=s),
        step_gated=lambda s: kda.decode_step_gated(q, k, v, beta, z, A, -5.0, S, gate, stream=s),
        linear=lambda s: kda.linear_fwd_chunked(q, k, v, g, stream=s),
        linear_bwd=lambda s: kda.linear_bwd(q, k, v, g, v, stream=s),
        linear_step=lambda s: kda.linear_decode_step(q, k, v, g, S, stream=s),
        qk_norm=lambda s: kda.qk_norm_rope(q, k, w, w, stream=s),
        qk_norm_bwd=lambda s: kda.qk_norm_rope_bwd(q, k, q, k, w, w, stream=s),
        quantile=lambda s: kda.quantile_balance(scores, bias, 2, True, True, stream=s))


NAMES = ["gate", "fwd", "softplus", "bwd", "step", "norm_gate", "step_gated", "linear",
         "linear_bwd", "linear_step", "qk_norm", "qk_norm_bwd", "quantile"]
WITH_WORKSPACE = {"fwd", "softplus", "bwd", "linear", "linear_bwd", "qk_norm_bwd", "quantile"}


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_the_given_stream(name, monkeypatch):
    from serving_kda_chunkwise_gb300 import build
    build.build()
    from serving_kda_chunkwise_gb300 import kda

    class Stream:
        def __init__(self, handle):
            self.cuda_stream = handle

    given, current = Stream(7), [Stream(1)]
    caller = current[0]
    made, kept = [], []

    @contextlib.contextmanager
    def on(stream):
        before, current[0] = current[0], stream
        yield
        current[0] = before

    def made_by(make):
        def wrapped(*args, **kwargs):
            kwargs.pop("device", None)
            t = make(*args, **kwargs).as_subclass(OnDevice)
            made.append((t.dtype, current[0]))
            return t
        return wrapped

    run = calls(kda)[name]
    monkeypatch.setattr(kda, "_lib", Nothing())
    monkeypatch.setattr(torch, "empty", made_by(torch.empty))
    monkeypatch.setattr(torch, "empty_like", made_by(torch.empty_like))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[0])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: kept.append(s))
    run(given)
    assert made and all(s is given for _, s in made)
    scratch = [s for dtype, s in made if dtype == torch.uint8]
    assert len(scratch) == (name in WITH_WORKSPACE)
    assert len(kept) == len(made) - len(scratch) and all(s is caller for s in kept)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["linear", "linear_bwd", "qk_norm_bwd"])
def test_results_while_the_current_stream_reuses_memory(name):
    from serving_kda_chunkwise_gb300 import kda
    gen = torch.Generator(device="cuda").manual_seed(1)

    def rand(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)

    T, H, d = 3000, 8, 128
    q, k, v, do = (rand(T, H, d) / d ** 0.5 for _ in range(4))
    g = -rand(T, H, dtype=torch.float32).abs()
    w = rand(d, dtype=torch.float32)
    run = dict(
        linear=lambda **s: kda.linear_fwd_chunked(q, k, v, g, **s),
        linear_bwd=lambda **s: list(kda.linear_bwd(q, k, v, g, do, **s).values()),
        qk_norm_bwd=lambda **s: list(kda.qk_norm_rope_bwd(q, k, do, v, w, w, **s).values()))[name]
    want = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # the call's kernels wait behind this
        got = run(stream=side)
        for n in (1 << 12, 1 << 20, 1 << 23, 1 << 25, 1 << 27):
            torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.current_stream().wait_stream(side)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del got
    kda.device_status()
