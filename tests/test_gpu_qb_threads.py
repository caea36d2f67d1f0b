"""Bias updates of different token counts from several host threads at once: the sampled path's kernel
needs shared memory by the count, which must not depend on what another thread asked for."""
import ctypes
import threading

import pytest

pytestmark = pytest.mark.gpu


def test_threads():
    import torch
    from serving_kda_chunkwise_gb300 import kda
    lib, n, k = kda.library(), 4, 2
    counts = [8192, 16380] * 2  # samples of 2048 and 4095 tokens
    want, outs, calls, kept, failed = [], [], [], [], []
    for j, m in enumerate(counts):
        gen = torch.Generator(device="cuda").manual_seed(j)
        scores, bias = torch.rand(m, n, generator=gen, device="cuda"), torch.zeros(n, device="cuda")
        want.append(kda.quantile_balance(scores, bias, k))
        out, stream = torch.empty_like(bias), torch.cuda.Stream()
        need = lib.kda_quantile_balance_workspace_size(m, n)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        outs.append(out)
        kept.append((scores, bias, ws, stream))
        p = [ctypes.c_void_p(t.data_ptr()) for t in (scores, bias, out, ws)]
        calls.append([p[0], p[1], m, n, k, p[2], None, None, p[3], ws.numel(),
                      ctypes.c_void_p(stream.cuda_stream)])
    torch.cuda.synchronize()

    def run(j):
        for _ in range(10000):
            if lib.kda_quantile_balance(*calls[j]) != kda.KDA_OK:
                failed.append((counts[j], lib.kda_last_error()))
                return

    threads = [threading.Thread(target=run, args=(j,)) for j in range(len(counts))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for a, b in zip(outs, want):
        assert torch.equal(a, b)
    kda.device_status()
