"""The C ABI of the per-head-decay linear attention and of the query/key norm without a GPU:
malformed arguments are refused on the host before any CUDA work is enqueued."""
import ctypes

import pytest

vp, i64, f, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
A = vp(0x10000)


@pytest.fixture(scope="module")
def lib():
    from serving_kda_chunkwise_gb300 import build
    lib = ctypes.CDLL(build.build())
    lib.kda_last_error.restype = ctypes.c_char_p
    for n in ("kda_linear_fwd_workspace_size", "kda_linear_bwd_workspace_size",
              "kda_qk_norm_rope_bwd_workspace_size"):
        getattr(lib, n).restype = sz
    return lib


def _call(lib, name, args, cases):
    fn = getattr(lib, name)
    fn.restype = ctypes.c_int
    for over, code, frag in cases:
        unknown = set(over) - set(args)
        assert not unknown, unknown
        rc = fn(*{**args, **over}.values())
        msg = lib.kda_last_error().decode()
        assert rc == code, (name, over, rc, msg)
        assert frag in msg, (name, over, msg)


LINEAR = [
    (dict(q=None), 1, "q is NULL"), (dict(k=vp(0x10008)), 1, "k is not 16-byte"),
    (dict(g=None), 1, "g is NULL"), (dict(g=vp(0x10002)), 1, "g is not 4-byte"),
    (dict(q_ld=i64(4 * 128 - 8)), 1, "q_ld"), (dict(k_ld=i64(4 * 128 + 4)), 1, "k_ld"),
    (dict(v_ld=i64(0)), 1, "v_ld"), (dict(dk=96), 2, "only 64 and 128"),
    (dict(dv=-1), 1, "positive"), (dict(H=0), 1, "H=0"), (dict(H=70000), 1, "H=70000"),
    (dict(dt=2), 1, "kda_dtype_t"),
]
PACKED = [
    (dict(T=i64(-1)), 1, "T_total"), (dict(T=i64(1 << 31)), 1, "T_total"),
    (dict(N=-1), 1, "N=-1"), (dict(N=3), 1, "multiple of N"), (dict(N=0), 1, "N=0"),
    (dict(cu=vp(0x10004)), 1, "cu_seqlens is not 16-byte"), (dict(ws=None), 1, "workspace is NULL"),
    (dict(S0=vp(0x10004)), 1, "S0 is not 16-byte"),
]


def test_forward(lib):
    need = lib.kda_linear_fwd_workspace_size(i64(40000), 2, 4, 128, 128, 1)
    assert need > 0
    args = dict(q=A, q_ld=i64(512), k=A, k_ld=i64(512), v=A, v_ld=i64(512), g=A, per=1, S0=None,
                S_out=None, cu=None, N=2, T=i64(40000), H=4, dk=128, dv=128, dt=1, o=A, ws=A,
                ws_bytes=sz(need), stream=None)
    _call(lib, "kda_linear_fwd_chunked", args, LINEAR + PACKED + [
        (dict(o=None), 1, "o is NULL"), (dict(ws_bytes=sz(need - 1)), 1, "smaller than"),
        (dict(S_out=vp(0x10004)), 1, "S_out is not 16-byte"), (dict(N=0, T=i64(0)), 0, "")])
    for bad in ((i64(-1), 1, 4, 128, 128), (i64(5), 0, 4, 128, 128), (i64(5), 1, 4, 96, 128)):
        assert lib.kda_linear_fwd_workspace_size(*bad, 1) == 0
        assert lib.kda_linear_bwd_workspace_size(*bad, 1) == 0


def test_backward(lib):
    need = lib.kda_linear_bwd_workspace_size(i64(4000), 2, 4, 128, 128, 1)
    args = dict(q=A, q_ld=i64(512), k=A, k_ld=i64(512), v=A, v_ld=i64(512), g=A, per=1, S0=None,
                cu=None, N=2, T=i64(4000), H=4, dk=128, dv=128, dt=1, dout=A, do_ld=i64(512),
                dS_out=None, dq=A, dk_out=A, dv_out=A, dg=None, dS0=None, ws=A, ws_bytes=sz(need),
                stream=None)
    _call(lib, "kda_linear_bwd", args, LINEAR + PACKED + [
        (dict(dout=None), 1, "dout is NULL"), (dict(do_ld=i64(8)), 1, "dout_ld"),
        (dict(dq=None), 1, "dq is NULL"), (dict(dv_out=None), 1, "dv is NULL"),
        (dict(dS0=vp(0x10004)), 1, "dS0 is not 16-byte"),
        (dict(ws_bytes=sz(need - 1)), 1, "smaller than")])


def test_step(lib):
    args = dict(q=A, q_ld=i64(512), k=A, k_ld=i64(512), v=A, v_ld=i64(512), g=A, per=1, S=A,
                slots=None, n_slots=8, N=8, H=4, dk=128, dv=128, dt=1, o=A, stream=None)
    _call(lib, "kda_linear_decode_step", args, LINEAR + [
        (dict(S=None), 1, "S is NULL"), (dict(n_slots=7), 1, "n_slots=7"),
        (dict(n_slots=-1), 1, "n_slots=-1"), (dict(slots=vp(0x10002)), 1, "slots"),
        (dict(N=-1), 1, "N=-1"), (dict(N=0), 0, "")])


NORM = [
    (dict(q=None), 1, "q is NULL"), (dict(k=None), 1, "k is NULL"),
    (dict(q_ld=i64(504)), 1, "q_ld"), (dict(k_ld=i64(260)), 1, "k_ld"),
    (dict(wq=vp(0x10004)), 1, "wq is not"), (dict(eps=f(-1.0)), 1, "eps"),
    (dict(eps=f(float("nan"))), 1, "eps"), (dict(cs=None), 1, "cos_sin is NULL"),
    (dict(pos=None), 1, "n_pos"), (dict(pos=vp(0x10001)), 1, "positions"),
    (dict(rot=24), 2, "rot_dim=24"), (dict(rot=144), 1, "rot_dim=144"),
    (dict(rot=-16), 1, "rot_dim=-16"), (dict(T=i64(-1)), 1, "T=-1"), (dict(Hq=0), 1, "Hq=0"),
    (dict(Hk=-1), 1, "Hk=-1"), (dict(d=96), 2, "d=96"), (dict(dt=5), 1, "kda_dtype_t"),
]


def test_norm(lib):
    args = dict(q=A, q_ld=i64(512), k=A, k_ld=i64(256), wq=A, wk=None, eps=f(1e-6), cs=A,
                n_pos=i64(5), pos=A, rot=64, inter=0, q_out=vp(0x20000), k_out=vp(0x30000),
                T=i64(10), Hq=4, Hk=2, d=128, dt=1, stream=None)
    _call(lib, "kda_qk_norm_rope", args, NORM + [
        (dict(q_out=None), 1, "q_out is NULL"), (dict(k_out=None), 1, "k_out is NULL"),
        (dict(q_out=A, q_ld=i64(1024)), 1, "only where q is contiguous"), (dict(T=i64(0)), 0, "")])


def test_norm_backward(lib):
    need = lib.kda_qk_norm_rope_bwd_workspace_size(128)
    assert need > 0 and lib.kda_qk_norm_rope_bwd_workspace_size(96) == 0
    args = dict(q=A, q_ld=i64(512), k=A, k_ld=i64(256), dyq=A, dyk=A, wq=A, wk=None, eps=f(1e-6),
                cs=A, n_pos=i64(5), pos=A, rot=64, inter=0, dq=A, dk=A, dwq=A, dwk=None,
                T=i64(10), Hq=4, Hk=2, d=128, dt=1, ws=A, ws_bytes=sz(need), stream=None)
    _call(lib, "kda_qk_norm_rope_bwd", args, NORM + [
        (dict(dyq=None), 1, "dyq is NULL"), (dict(dyk=None), 1, "dyk is NULL"),
        (dict(dq=None), 1, "dq is NULL"), (dict(dk=None), 1, "dk is NULL"),
        (dict(ws=None), 1, "workspace is NULL"), (dict(ws_bytes=sz(need - 1)), 1, "smaller than")])
