"""Norm gradients called by several host threads at once: their kernels are the same and need different
amounts of shared memory, which must not depend on what another thread asked for."""
import ctypes
import threading

import pytest

pytestmark = pytest.mark.gpu


def test_threads():
    import torch
    from serving_kda_chunkwise_gb300 import kda
    fn, null = kda.library().kda_block_norm_bwd, None
    shapes = [(4, 64), (4, 4096)] * 2
    want, outs, calls, failed, kept = [], [], [], [], []
    for k, (T, D) in enumerate(shapes):
        gen = torch.Generator(device="cuda").manual_seed(k)
        y, r, dx = (torch.randn(T, D, generator=gen, device="cuda") for _ in range(3))
        want.append(kda.block_norm_bwd(y, r, dx))
        out = [torch.empty_like(y) for _ in range(2)]
        stream = torch.cuda.Stream()
        outs.append(out)
        kept.append((y, r, dx, stream))
        p = [ctypes.c_void_p(t.data_ptr()) for t in (y, r, dx, *out)]
        # y, gate, r_out, dx, dr, three weights | dr, dy, dgate and the weights' gradients
        calls.append([p[0], null, p[1], p[2], null, null, null, null, 1, 1e-6, p[3], p[4], null, null,
                      null, null, T, D, kda.KDA_F32, kda.KDA_F32, null, 0,
                      ctypes.c_void_p(stream.cuda_stream)])
    torch.cuda.synchronize()

    def run(k):
        for _ in range(20000):
            if fn(*calls[k]) != kda.KDA_OK:
                failed.append((shapes[k], kda.library().kda_last_error()))
                return

    threads = [threading.Thread(target=run, args=(k,)) for k in range(len(shapes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for (dr, dy), b in zip(outs, want):
        assert torch.equal(dr, b["dr"]) and torch.equal(dy, b["dy"])
    kda.device_status()
