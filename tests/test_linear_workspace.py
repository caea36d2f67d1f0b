"""Workspace of the linear attention: what its kernels can use, however many sequences share the
tokens.  Only a sequence longer than a segment has states at segments' edges, and decays are kept
for the chunks of 128 tokens that exist."""
import ctypes

import pytest

i64 = ctypes.c_int64


@pytest.fixture(scope="module")
def sizes():
    from serving_kda_chunkwise_gb300 import build
    lib = ctypes.CDLL(build.build())
    out = []
    for n in ("kda_linear_fwd_workspace_size", "kda_linear_bwd_workspace_size"):
        f = getattr(lib, n)
        f.restype = ctypes.c_size_t
        out.append(lambda T, N, H, dk, dv, dt, f=f: f(i64(T), N, H, dk, dv, dt))
    return out


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("T,N,H,dk,dv", [
    (1024, 1024, 32, 128, 128), (4096, 4096, 32, 128, 128), (65536, 4096, 32, 128, 128),
    (76800, 256, 32, 128, 128), (65536, 65536, 8, 64, 64), (512, 512, 4, 64, 128), (7, 100, 2, 64, 64)])
def test_grows_by_what_can_exist(sizes, T, N, H, dk, dv, dt):
    """Two arrays (gradients: four) of at most 2 T / L edge states, where segments are at least 64
    (bf16: 128) tokens and there is about one a SM at most (bf16; gradients up to 1,024 tokens,
    forward 2,048; fp32 four); the chunks' decays (bf16: 4.7 KB each); dot products; 16 parts of
    <S, D> at both ends of a sequence."""
    state = H * dk * dv * 4
    for bwd, size in enumerate(sizes):
        L = 128 if dt else 64
        while L < (1024 if bwd or not dt else 2048) and T // L * H > (152 if dt else 608):
            L *= 2
        edges = 2 * T // L
        chunks = T // 128 + N
        most = (4 if bwd else 2) * edges * state + (chunks * H * 4736 if dt else 0)
        most += 2 * edges * H * 4 + (bwd and 2 * (dk // 32) * T * H * 4 + T * H * 4 + N * H * 2 * 16 * 4)
        assert size(T, N, H, dk, dv, dt) <= most + 4096 + (1 << 20)


def test_one_long_sequence_as_before(sizes):
    """One sequence keeps one slot a segment (and one more)."""
    fwd, bwd = sizes
    state = 32 * 128 * 128 * 4
    assert fwd(65536, 1, 32, 128, 128, 1) <= 2 * 33 * state + 513 * 32 * 4736 + (1 << 20)
    assert bwd(65536, 1, 16, 128, 128, 1) <= (4 * 65 * state // 2 + 513 * 16 * 4736
                                              + 9 * 65536 * 16 * 4 + (1 << 20))
