"""The linear attention of no sequences at all: the gradients take it as the forward does."""
import ctypes

import pytest

vp, i64 = ctypes.c_void_p, ctypes.c_int64


def test_gradients_take_no_sequences():
    from serving_kda_chunkwise_gb300 import build
    lib = ctypes.CDLL(build.build())
    lib.kda_last_error.restype = ctypes.c_char_p
    ld = i64(512)

    def bwd(T, dg, per_token=1):
        return lib.kda_linear_bwd(None, ld, None, ld, None, ld, None, per_token, None, None, 0,
                                  i64(T), 4, 128, 128, 1, None, ld, None, None, None, None, dg,
                                  None, None, ctypes.c_size_t(0), None)

    assert bwd(0, None) == 0, lib.kda_last_error()
    assert bwd(0, None, 0) == 0, lib.kda_last_error()
    assert bwd(0, vp(0x10000)) == 0, lib.kda_last_error()
    assert bwd(5, None) == 1 and b"N=0" in lib.kda_last_error()
    assert bwd(0, vp(0x10002)) == 1 and b"dg" in lib.kda_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("per_token", [True, False])
def test_binding(per_token):
    import torch
    from serving_kda_chunkwise_gb300 import kda
    z = torch.empty(0, 3, 64, device="cuda")
    g = torch.empty(0, 3, device="cuda") if per_token else torch.ones(3, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, S = kda.linear_fwd_chunked(z, z, z, g, cu_seqlens=cu)
    assert o.shape == (0, 3, 64) and S.shape == (0, 3, 64, 64)
    out = kda.linear_bwd(z, z, z, g, z, cu_seqlens=cu)
    assert out["dg"].shape == g.shape and float(out["dg"].abs().sum()) == 0.0
    assert out["dq"].shape == (0, 3, 64) and out["dS0"].shape == (0, 3, 64, 64)
    kda.device_status()
