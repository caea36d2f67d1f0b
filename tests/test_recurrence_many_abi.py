"""The C ABI of the channel recurrence for very many sequences, without a GPU: the product of sequences
and channels is limited as the step's pool is, not as heads of a larger state are."""
import ctypes

import pytest

vp, i64, f, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
A = vp(0x10000)


@pytest.fixture(scope="module")
def lib():
    from serving_kda_chunkwise_gb300 import build
    lib = ctypes.CDLL(build.build())
    lib.kda_last_error.restype = ctypes.c_char_p
    return lib


# (sequences, channels): just above 2^29 in all, and a product that is too large for any memory
@pytest.mark.parametrize("N,D,says", [(131073, 4096, "workspace is NULL"),
                                      ((1 << 26) + 1, 8, "workspace is NULL"),
                                      ((1 << 20), 1 << 16, "N*D=68719476736 is too large"),
                                      ((1 << 31) - 4096, 4096, "N*D=")])
def test_many_sequences(lib, N, D, says):
    rows = [A, i64(D)]
    mid = [A, f(-5.0), None]
    size = [None, N, i64(N), D, 0]
    for name, args in (
            ("kda_recurrence_fwd", rows * 3 + mid + [None] + size + [A, None, None, sz(0), None]),
            ("kda_recurrence_bwd", rows * 3 + mid + size + rows + [None] * 2 + [A] * 3 + [None] * 3
             + [sz(0), None]),
            ("kda_recurrence_bwd_packed", [A] * 6 + mid + size + rows + [None] + [A] * 3
             + [None] * 3 + [sz(0), None])):
        rc = getattr(lib, name)(*args)
        msg = lib.kda_last_error().decode()
        assert rc == 1 and says in msg, (name, rc, msg)
