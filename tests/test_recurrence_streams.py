"""What a call of the channel recurrence, the 8-bit checkpoints and the norms around a block allocates
for itself when it is given a stream, as tests/test_binding_streams.py has it for the other calls: the
workspace and the outputs are of that stream's memory, and the outputs kept from reuse while the
caller's stream reads them.  And what the binding refuses before the library is called.

On the CPU: tensors that say they are on the device, a library that does nothing, and streams of which
only the current one is known.  On the GPU: results while the default stream takes and overwrites
whatever memory it is given."""
import contextlib

import pytest
import torch

T, D = 20, 64


class OnDevice(torch.Tensor):
    is_cuda = True


class Elsewhere(OnDevice):
    def get_device(self):
        return 1


def tensor(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


class Nothing:
    """Entry points that succeed; sizes of a workspace that is needed."""

    def __getattr__(self, name):
        return lambda *args: 64 if name.endswith("_size") else 0


def calls(kda):
    f32, i8 = torch.float32, torch.int8
    x, z, i, dy = (tensor(T, D) for _ in range(4))
    A, h = tensor(D, dtype=f32), tensor(T, D, dtype=f32)
    kept = (tensor(T, D, dtype=i8), tensor(1, T, dtype=i8))
    return dict(
        fwd=lambda s: kda.recurrence_fwd(x, z, i, A, -5.0, stream=s),
        bwd=lambda s: kda.recurrence_bwd(x, z, i, A, -5.0, dy, stream=s),
        bwd_packed=lambda s: kda.recurrence_bwd(kept, kept, kept, A, -5.0, dy, stream=s),
        step=lambda s: kda.recurrence_step(x, z, i, A, -5.0, h, stream=s),
        pack=lambda s: kda.checkpoint_pack(x, stream=s),
        unpack=lambda s: kda.checkpoint_unpack(*kept, stream=s),
        norm=lambda s: kda.block_norm(x, z, gate=i, scale=A, w_post=A, w_pre=A, stream=s),
        norm_bwd=lambda s: kda.block_norm_bwd(x, z, dy, gate=i, scale=A, w_post=A, w_pre=A,
                                              stream=s))


NAMES = ["fwd", "bwd", "bwd_packed", "step", "pack", "unpack", "norm", "norm_bwd"]
WITH_WORKSPACE = {"fwd", "bwd", "bwd_packed", "norm_bwd"}


@pytest.fixture
def kda(monkeypatch):
    from serving_kda_chunkwise_gb300 import build
    build.build()
    from serving_kda_chunkwise_gb300 import kda
    monkeypatch.setattr(kda, "_lib", Nothing())
    return kda


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_the_given_stream(name, kda, monkeypatch):
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


def test_tensors_of_several_devices(kda, monkeypatch):
    """A tensor of another device than the others, or than the current one."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(kda, "_stream", lambda s: 0)
    x, A = tensor(T, D), tensor(D, dtype=torch.float32)
    far, far_A = x.as_subclass(Elsewhere), A.as_subclass(Elsewhere)
    kept = (tensor(T, D, dtype=torch.int8), tensor(1, T, dtype=torch.int8))
    with pytest.raises(ValueError, match="different devices"):
        kda.recurrence_fwd(x, far, x, A, -5.0)
    with pytest.raises(ValueError, match="not the current"):
        kda.recurrence_fwd(far, far, far, far_A, -5.0)
    with pytest.raises(ValueError, match="different devices"):
        kda.recurrence_bwd(kept, kept, (kept[0], kept[1].as_subclass(Elsewhere)), A, -5.0, x)
    with pytest.raises(ValueError, match="different devices"):
        kda.block_norm(x, x, w_pre=far_A)
    with pytest.raises(ValueError, match="not the current"):
        kda.checkpoint_pack(far)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["fwd", "bwd", "norm_bwd"])
def test_results_while_the_current_stream_reuses_memory(name):
    from serving_kda_chunkwise_gb300 import kda
    gen = torch.Generator(device="cuda").manual_seed(1)

    def rand(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)

    x, z, i, dy = (rand(3000, 512) for _ in range(4))
    A, w = rand(512, dtype=torch.float32), rand(512, dtype=torch.float32)
    cu = torch.tensor([0, 1000, 1001, 3000], dtype=torch.int32, device="cuda")
    run = dict(
        fwd=lambda **s: kda.recurrence_fwd(x, z, i, A, -5.0, cu_seqlens=cu, **s),
        bwd=lambda **s: list(kda.recurrence_bwd(x, z, i, A, -5.0, dy, cu_seqlens=cu, **s).values()),
        norm_bwd=lambda **s: [t for t in kda.block_norm_bwd(x, z, dy, i, scale=w, w_pre=w,
                                                            **s).values() if t is not None])[name]
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
