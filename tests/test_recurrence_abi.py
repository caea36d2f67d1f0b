"""The C ABI of the channel recurrence, the 8-bit checkpoints and the norms around a block without a
GPU: malformed arguments are refused on the host before any CUDA work is enqueued."""
import ctypes

import pytest

vp, i64, f, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
A = vp(0x10000)


@pytest.fixture(scope="module")
def lib():
    from serving_kda_chunkwise_gb300 import build
    lib = ctypes.CDLL(build.build())
    lib.kda_last_error.restype = ctypes.c_char_p
    for n in ("kda_recurrence_fwd_workspace_size", "kda_recurrence_bwd_workspace_size",
              "kda_block_norm_bwd_workspace_size"):
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


PACKED = [
    (dict(A_log=None), 1, "A_log is NULL"), (dict(g_min=f(0.0)), 1, "g_min"),
    (dict(g_min=f(float("nan"))), 1, "g_min"), (dict(D=0), 1, "D=0"),
    (dict(D=60), 2, "multiples of 8"), (dict(dt=2), 1, "kda_dtype_t"),
    (dict(T=i64(-1)), 1, "T_total"), (dict(T=i64(1 << 31)), 1, "T_total"),
    (dict(T=i64((1 << 31) - 2048)), 1, "T_total"),
    (dict(N=-1), 1, "N=-1"), (dict(N=3), 1, "multiple of N"), (dict(N=0), 1, "N=0"),
    (dict(cu=vp(0x10004)), 1, "cu_seqlens is not 16-byte"),
    (dict(h0=vp(0x10004)), 1, "h0 is not 16-byte"),
]
WHOLE = [
    (dict(x=None), 1, "x is NULL"), (dict(z=vp(0x10008)), 1, "z is not 16-byte"),
    (dict(i=None), 1, "i is NULL"), (dict(x_ld=i64(56)), 1, "x_ld"),
    (dict(z_ld=i64(68)), 1, "z_ld"), (dict(i_ld=i64(-64)), 1, "i_ld"),
    (dict(edges=vp(0x10004)), 1, "edges is not 16-byte"),
]


def test_forward(lib):
    need = lib.kda_recurrence_fwd_workspace_size(i64(4000), 2, 64)
    args = dict(x=A, x_ld=i64(64), z=A, z_ld=i64(64), i=A, i_ld=i64(64), A_log=A, g_min=f(-5.0),
                h0=None, h_out=None, cu=None, N=2, T=i64(4000), D=64, dt=1, y=A, edges=None, ws=A,
                ws_bytes=sz(need), stream=None)
    _call(lib, "kda_recurrence_fwd", args, PACKED + WHOLE + [
        (dict(y=None), 1, "y is NULL"), (dict(h_out=vp(0x10004)), 1, "h_out is not"),
        (dict(N=0, T=i64(0)), 0, "")])
    for n in ("fwd", "bwd"):
        size = getattr(lib, f"kda_recurrence_{n}_workspace_size")
        for bad in ((i64(-1), 1, 64), (i64(5), 0, 64), (i64(5), 1, 60), (i64(5), 1, -8)):
            assert size(*bad) == 0


def test_backward(lib):
    need = lib.kda_recurrence_bwd_workspace_size(i64(4000), 2, 64)
    assert need > 0
    back = dict(dy=A, dy_ld=i64(64), dh_out=None)
    outs = dict(dx=A, dz=A, di=A, dA=None, dh0=None, ws=A, ws_bytes=sz(need), stream=None)
    mid = dict(A_log=A, g_min=f(-5.0), h0=None, cu=None, N=2, T=i64(4000), D=64, dt=1)
    both = PACKED + [
        (dict(dy=None), 1, "dy is NULL"), (dict(dy_ld=i64(60)), 1, "dy_ld"),
        (dict(dx=None), 1, "dx is NULL"), (dict(dz=None), 1, "dz is NULL"),
        (dict(di=None), 1, "di is NULL"), (dict(dA=vp(0x10004)), 1, "dA_log is not"),
        (dict(dh0=vp(0x10004)), 1, "dh0 is not"), (dict(dh_out=vp(0x10004)), 1, "dh_out is not"),
        (dict(ws=None), 1, "workspace is NULL"), (dict(ws_bytes=sz(need - 1)), 1, "smaller than"),
        (dict(N=0, T=i64(0)), 0, "")]
    whole = dict(x=A, x_ld=i64(64), z=A, z_ld=i64(64), i=A, i_ld=i64(64))
    _call(lib, "kda_recurrence_bwd", {**whole, **mid, **back, "edges": None, **outs}, both + WHOLE)
    codes = dict(x=A, xe=A, z=A, ze=A, i=A, ie=A)
    _call(lib, "kda_recurrence_bwd_packed", {**codes, **mid, **back, **outs}, both + [
        (dict(x=None), 1, "x_codes is NULL"), (dict(ze=None), 1, "z_exps is NULL"),
        (dict(i=vp(0x10008)), 1, "i_codes is not 16-byte")])


def test_step(lib):
    args = dict(x=A, x_ld=i64(64), z=A, z_ld=i64(64), i=A, i_ld=i64(64), A_log=A, g_min=f(-5.0),
                h=A, slots=None, n_slots=8, N=8, D=64, dt=1, y=A, stream=None)
    _call(lib, "kda_recurrence_step", args, WHOLE[:-1] + [
        (dict(h=None), 1, "h is NULL"), (dict(y=None), 1, "y is NULL"),
        (dict(n_slots=7), 1, "n_slots=7"), (dict(n_slots=-1), 1, "n_slots=-1"),
        (dict(slots=vp(0x10002)), 1, "slots"), (dict(N=-1), 1, "N=-1"), (dict(D=20), 2, "D=20"),
        (dict(g_min=f(1.0)), 1, "g_min"), (dict(dt=7), 1, "kda_dtype_t"), (dict(N=0), 0, "")])


def test_checkpoint(lib):
    common = [(dict(T=i64(-1)), 1, "T=-1"), (dict(D=-8), 1, "D=-8"), (dict(D=12), 2, "D=12"),
              (dict(dt=3), 1, "kda_dtype_t"), (dict(codes=None), 1, "codes is NULL"),
              (dict(codes=vp(0x10004)), 1, "codes is not"), (dict(exps=None), 1, "exps is NULL"),
              (dict(x=None), 1, "x is NULL"), (dict(T=i64(0)), 0, "")]
    _call(lib, "kda_checkpoint_pack", dict(x=A, x_ld=i64(64), T=i64(5), D=64, dt=1, codes=A, exps=A,
                                           stream=None), common + [(dict(x_ld=i64(60)), 1, "x_ld")])
    _call(lib, "kda_checkpoint_unpack", dict(codes=A, exps=A, T=i64(5), D=64, dt=0, x=A,
                                             stream=None), common)


NORM = [
    (dict(y=None), 1, "y is NULL"), (dict(D=0), 1, "D=0"), (dict(D=20), 2, "D=20"),
    (dict(D=8200), 2, "at most 8192"), (dict(dt=2), 1, "kda_dtype_t"), (dict(rdt=9), 1, "r_dt"),
    (dict(dt=0, rdt=1), 1, "r_dt"), (dict(eps=f(-1.0)), 1, "eps"), (dict(T=i64(-1)), 1, "T=-1"),
    (dict(eps=f(float("inf"))), 1, "eps"), (dict(post=0), 1, "w_post must be NULL"),
    (dict(gate=vp(0x10004)), 1, "gate is not"), (dict(scale=vp(0x10004)), 1, "scale is not"),
    (dict(w_pre=vp(0x10004)), 1, "w_pre is not"),
]


def test_block_norm(lib):
    args = dict(y=A, gate=None, r=A, scale=None, w_post=A, w_pre=None, post=1, eps=f(1e-6), r_out=A,
                x_out=A, T=i64(9), D=64, dt=1, rdt=1, stream=None)
    _call(lib, "kda_block_norm", args, NORM + [
        (dict(r=None), 1, "r is NULL"), (dict(r_out=None), 1, "r_out is NULL"),
        (dict(x_out=vp(0x10004)), 1, "x_out is not"), (dict(T=i64(0)), 0, "")])


def test_block_norm_backward(lib):
    need = lib.kda_block_norm_bwd_workspace_size(64)
    assert need > 0 and lib.kda_block_norm_bwd_workspace_size(60) == 0
    assert lib.kda_block_norm_bwd_workspace_size(8200) == 0
    args = dict(y=A, gate=None, r=A, dx=A, dr=None, scale=None, w_post=A, w_pre=None, post=1,
                eps=f(1e-6), dr_in=A, dy=A, dgate=None, dscale=None, dw_post=A, dw_pre=None,
                T=i64(9), D=64, dt=1, rdt=0, ws=A, ws_bytes=sz(need), stream=None)
    _call(lib, "kda_block_norm_bwd", args, NORM + [
        (dict(r=None), 1, "r_out is NULL"), (dict(dx=None), 1, "dx is NULL"),
        (dict(dr=vp(0x10004)), 1, "dr is not"), (dict(dr_in=None), 1, "dr_in is NULL"),
        (dict(dy=None), 1, "dy is NULL"), (dict(gate=A), 1, "dgate is NULL"),
        (dict(dgate=A), 1, "dgate must be NULL"),
        (dict(post=0, w_post=None), 1, "dw_post must be NULL"),
        (dict(dscale=vp(0x10004)), 1, "dscale is not"), (dict(ws=None), 1, "workspace is NULL"),
        (dict(ws_bytes=sz(need - 1)), 1, "smaller than")])
