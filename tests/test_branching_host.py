"""Windowed attention, beam selection and cache reorder without a GPU: every refusal
is made on the host before CUDA is touched, and the documented workspace sizes."""
import ctypes as C

import numpy as np
import pytest

import session_decode_step_gb300 as kd
from session_decode_step_gb300 import build as kbuild

D = 1 << 20  # never dereferenced: every check runs on the host first
I32P = C.POINTER(C.c_int32)
INVALID, BAD_SESSION, POSITION, BATCH, UNSUPPORTED = -1, -5, -6, -7, -8


def arr(*v):
    return np.array(v, np.int32)


def p(a):
    return a.ctypes.data_as(I32P) if a is not None else None


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kd.lib()


def window(lib, q=D, kn=D, kc=D, B=2, nh=32, nkv=8, hd=128, n_slots=4, cap=64, win=16, sinks=4, out=D, ws=D,
           ws_bytes=1 << 30, sl=arr(0, 1), ps=arr(0, 3)):
    return lib.kd_attn_window_append_decode(q, kn, D, kc, D, p(sl), p(ps), B, nh, nkv, hd, n_slots, cap, win, sinks,
                                            out, ws, ws_bytes, None)


def window_q8(lib, q=D, ks=D, B=2, nh=32, nkv=8, n_slots=4, cap=64, win=16, sinks=4, ws=D, ws_bytes=1 << 30,
              sl=arr(0, 1), ps=arr(0, 3)):
    return lib.kd_attn_window_append_decode_q8(q, D, D, D, ks, D, D, p(sl), p(ps), B, nh, nkv, n_slots, cap, win, sinks,
                                               D, ws, ws_bytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(kn=None), INVALID), (dict(kc=None), INVALID), (dict(out=None), INVALID),
    (dict(ws=None), INVALID), (dict(sl=None), INVALID), (dict(ps=None), INVALID),
    (dict(B=0), BATCH), (dict(B=17), BATCH),
    (dict(hd=96), UNSUPPORTED), (dict(nh=24), UNSUPPORTED), (dict(nh=30), UNSUPPORTED), (dict(nkv=0), UNSUPPORTED), (dict(nkv=1025, nh=1025), UNSUPPORTED),
    (dict(n_slots=0), INVALID), (dict(cap=0), INVALID), (dict(cap=65537), UNSUPPORTED),
    (dict(cap=2 ** 31 - 1), UNSUPPORTED),
    (dict(win=0), INVALID), (dict(win=-1), INVALID), (dict(sinks=-1), INVALID),
    (dict(n_slots=1 << 20, cap=65536), UNSUPPORTED),  # 2^39 cache rows
    (dict(ws_bytes=256), INVALID), (dict(ws=D + 8), INVALID), (dict(kc=D + 8), INVALID), (dict(q=D + 4), INVALID),
    (dict(kn=D + 2), INVALID), (dict(out=D + 1), INVALID),
    (dict(sl=arr(1, 1)), BAD_SESSION), (dict(sl=arr(0, 4)), BAD_SESSION), (dict(sl=arr(-1, 1)), BAD_SESSION),
    (dict(ps=arr(0, 64)), POSITION), (dict(ps=arr(-1, 0)), POSITION),
])
def test_window_refusals(lib, change, status):
    assert window(lib, **change) == status, kd.kd_last_error()
    assert "kd_attn_window_append_decode" in kd.kd_last_error()


@pytest.mark.parametrize("change,status", [
    (dict(ks=None), INVALID), (dict(cap=63), INVALID), (dict(q=D + 8), INVALID), (dict(ks=D + 8), INVALID),
    (dict(nh=12, nkv=4), UNSUPPORTED), (dict(win=0), INVALID), (dict(B=17), BATCH),
    (dict(sl=arr(2, 2)), BAD_SESSION), (dict(ps=arr(64, 0)), POSITION), (dict(ws_bytes=4096), INVALID),
])
def test_window_q8_refusals(lib, change, status):
    assert window_q8(lib, **change) == status, kd.kd_last_error()


def test_window_workspace_bytes(lib):
    def want(B, nh, hd, cap, win, sinks):
        items = min(-(-cap // 64), -(-min(sinks, cap) // 64) + -(-(min(win, cap) + 7) // 64))
        return 256 + B * nh * items * (hd + 4) * 4
    for a in [(1, 4, 64, 1, 1, 0), (16, 32, 128, 65536, 8192, 64), (8, 32, 128, 4097, 1, 1), (2, 8, 64, 300, 2**31 - 1, 2**31 - 1)]:
        assert kd.kd_attn_window_workspace_bytes(*a) == want(*a), a
    for a in [(0, 4, 64, 8, 1, 0), (1, 4, 64, 8, 0, 0), (1, 4, 64, 8, 1, -1)]:
        assert kd.kd_attn_window_workspace_bytes(*a) == 0


def beam(lib, logits=D, ld=1000, G=2, W=4, V=1000, scores=D, done=None, eos=-1, n_out=8, par=D, tok=D, sc=D, ws=D,
         ws_bytes=1 << 30):
    return lib.kd_beam_select(logits, ld, G, W, V, scores, done, eos, n_out, par, tok, sc, None, ws, ws_bytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(logits=None), INVALID), (dict(par=None), INVALID), (dict(tok=None), INVALID), (dict(sc=None), INVALID),
    (dict(ws=None), INVALID), (dict(logits=D + 2), INVALID), (dict(ws=D + 8), INVALID),
    (dict(scores=D + 2), INVALID), (dict(par=D + 1), INVALID), (dict(tok=D + 2), INVALID), (dict(sc=D + 3), INVALID),
    (dict(G=0), BATCH), (dict(W=0), BATCH), (dict(W=17), BATCH), (dict(G=5000, W=16), BATCH),
    (dict(n_out=0), INVALID), (dict(n_out=33), INVALID),
    (dict(V=0), INVALID), (dict(ld=999), INVALID), (dict(V=524289, ld=524289), UNSUPPORTED),
    (dict(eos=1000), INVALID), (dict(done=D), INVALID),  # finished beams need an end token
    (dict(ws_bytes=256), INVALID),
])
def test_beam_refusals(lib, change, status):
    assert beam(lib, **change) == status, kd.kd_last_error()


def test_beam_workspace_bytes(lib):
    for G, W, V, n in [(1, 1, 1, 1), (3, 16, 32003, 32), (32, 8, 128256, 8), (1, 2, 4096, 4), (1, 2, 4097, 4)]:
        assert kd.kd_beam_workspace_bytes(G, W, V, n) == 256 + G * W * -(-V // 4096) * (8 + 8 * n)
    assert kd.kd_beam_workspace_bytes(0, 1, 1, 1) == 0


def reorder(lib, planes=(D, D), widths=(256, 256), n_planes=2, L=2, S=4, nkv=2, cap=64, dst=arr(0, 1), src=arr(1, 0),
            lens=arr(5, 6), n=2, win=0, sinks=0):
    pl = (C.c_void_p * len(planes))(*planes) if planes else None
    rb = (C.c_int32 * len(widths))(*widths) if widths else None
    return lib.kd_kv_reorder(pl, rb, n_planes, L, S, nkv, cap, p(dst), p(src), p(lens), n, win, sinks, None)


@pytest.mark.parametrize("change,status", [
    (dict(planes=None), INVALID), (dict(widths=None), INVALID), (dict(dst=None), INVALID), (dict(src=None), INVALID),
    (dict(lens=None), INVALID), (dict(planes=(D, None)), INVALID), (dict(planes=(D, D + 8)), INVALID),
    (dict(n=0), BATCH), (dict(n=65), BATCH), (dict(n_planes=0), INVALID), (dict(n_planes=5), INVALID),
    (dict(L=0), INVALID), (dict(S=0), INVALID), (dict(nkv=0), INVALID), (dict(cap=0), INVALID),
    (dict(win=-1), INVALID), (dict(sinks=-1), INVALID),
    (dict(widths=(256, 12)), UNSUPPORTED), (dict(widths=(0, 8)), UNSUPPORTED), (dict(widths=(1032, 8)), UNSUPPORTED),
    (dict(L=40000), UNSUPPORTED), (dict(cap=131073), UNSUPPORTED),
    (dict(dst=arr(1, 1)), BAD_SESSION), (dict(dst=arr(0, 4)), BAD_SESSION), (dict(src=arr(0, -1)), BAD_SESSION),
    (dict(lens=arr(65, 0)), POSITION), (dict(lens=arr(-1, 0)), POSITION),
])
def test_reorder_refusals(lib, change, status):
    assert reorder(lib, **change) == status, kd.kd_last_error()


def test_model_calls_refuse_null(lib):
    out = C.c_int32()
    ids = arr(0)
    assert lib.kd_model_set_window(None, 4, 0) == INVALID
    assert lib.kd_session_reorder(None, p(ids), p(ids), 1, None) == INVALID
    assert lib.kd_session_fork(None, 0, C.byref(out), None) == INVALID


def test_binding_checks_plane_sizes():
    t = np.zeros((2, 4, 2, 64, 3), np.uint8)
    with pytest.raises(ValueError):
        kd.kd_kv_reorder([t], [0], [1], [5], 2, 4, 2, 65)
    with pytest.raises(ValueError):
        kd.kd_kv_reorder([t], [0, 1], [1], [5], 2, 4, 2, 64)


def bound_window(slots, positions, cap=64, sinks=4, q8=False, **kw):
    """The binding's call on host buffers: refused before CUDA is touched, and the message shows what arrived."""
    ws = np.zeros(1 << 20, np.uint8)
    x = np.zeros(4096, np.float32)
    buf = {"q": x, "k_new": x, "v_new": x, **kw}
    a = (buf["q"], buf["k_new"], buf["v_new"])
    if q8:
        return kd.kd_attn_window_append_decode_q8(*a, x, x, x, x, slots, positions, 4, 2, 8, cap, 16, sinks, x, ws)
    return kd.kd_attn_window_append_decode(*a, x, x, slots, positions, 4, 2, 64, 8, cap, 16, sinks, x, ws)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("kind", [list, tuple, lambda v: np.array(v, np.int32), lambda v: np.array(v, np.int64),
                                  lambda v: np.array([v, v], np.int32).T.copy()[:, 0], lambda v: np.array(v, ">i4")])
def test_binding_takes_host_arrays_of_any_kind(lib, kind, q8):
    with pytest.raises(kd.KdError, match="position 77 outside"):
        bound_window(kind([3, 5, 1]), kind([1, 2, 77]), q8=q8)
    with pytest.raises(kd.KdError, match="slot 5 repeated"):
        bound_window(kind([5, 2, 5]), kind([1, 2, 3]), q8=q8)
    with pytest.raises(ValueError, match="expected 3 entries, got 2"):
        bound_window(kind([3, 5, 1]), kind([1, 2]), q8=q8)


def test_binding_refuses_what_it_cannot_pass(lib):
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="contiguous"):
        bound_window([0], [0], q=torch.zeros(4, 4).t())
    with pytest.raises(ValueError, match="contiguous"):
        bound_window([0], [0], q=np.zeros((4, 4), np.float32).T)
    with pytest.raises(TypeError):
        bound_window([0], [0], q="a string")
    with pytest.raises(kd.KdError, match="null argument"):
        bound_window([0], [0], q=None)
    with pytest.raises(OverflowError):
        bound_window([0], [0], sinks=2 ** 31)
    with pytest.raises(TypeError):
        bound_window([0], [0], cap=1.5)
    with pytest.raises(kd.KdError, match="B=0"):
        bound_window([], [])
    with pytest.raises(kd.KdError, match="sinks -1"):
        bound_window([0], [0], sinks=np.int64(-1))
    x = torch.zeros(2, 1000)
    i = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(kd.KdError, match="ld=999"):
        kd.kd_beam_select(x, 1, 2, 1000, None, 4, i, i, x, x, ld=999)
    t = np.zeros((2, 4, 2, 64, 8), np.uint8)
    with pytest.raises(kd.KdError, match="slot 3 <- 9 outside"):
        kd.kd_kv_reorder([t], [3], [9], [5], 2, 4, 2, 64)
    with pytest.raises(kd.KdError, match="n_planes=5"):
        kd.kd_kv_reorder((t,) * 5, [3], [1], [5], 2, 4, 2, 64)
    with pytest.raises(ValueError, match="positive"):
        kd.kd_kv_reorder([t], [3], [1], [5], 2, 4, 0, 64)
