"""Rotary positions, paged append and paged attention without a GPU: the plan's frequencies,
every refusal made on the host before CUDA is touched, the workspace size, the binding's checks."""
import ctypes as C
import decimal
import math

import numpy as np
import pytest

import session_decode_step_gb300 as kd
from session_decode_step_gb300 import build as kbuild

D = 1 << 20  # never dereferenced: every check runs on the host first
I32P = C.POINTER(C.c_int32)
INVALID, POSITION, BATCH, UNSUPPORTED = -1, -6, -7, -8
torch = pytest.importorskip("torch")


def arr(*v):
    return np.array(v, np.int32)


def p(a):
    return a.ctypes.data_as(I32P) if a is not None else None


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kd.lib()


@pytest.fixture(params=["module", "ctypes"])
def calls(request, lib, monkeypatch):
    """Both ways to marshal a call."""
    monkeypatch.setattr(kd, "_call", None if request.param == "module" else kd._CtypesCalls)
    return request.param


# ---------------------------------------------------------------------- the plan ---
def turns(table):
    return np.array([t / 2.0 ** 64 for t in table.turns[:table.rot_dim // 2]])


def scaled(f, i, rot, theta, scaling, factor, low, high, original):
    if scaling == kd.KD_ROPE_LINEAR:
        return f / factor
    if scaling == kd.KD_ROPE_BANDS:
        wave = 2 * math.pi / f
        if wave > original / low:
            return f / factor
        if wave < original / high:
            return f
        u = (original / wave - low) / (high - low)
        return (1 - u) * f / factor + u * f
    if scaling == kd.KD_ROPE_RAMP:
        at = [rot * math.log(original / (2 * math.pi * n)) / (2 * math.log(theta)) for n in (high, low)]
        a, b = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
        u = min(1.0, max(0.0, (i - a) / max(b - a, 0.001)))
        return u * f / factor + (1 - u) * f
    return f


@pytest.mark.parametrize("rot", [2, 20, 64, 128, 256])
@pytest.mark.parametrize("theta", [10000.0, 500000.0, 1.5])
@pytest.mark.parametrize("kw", [dict(), dict(scaling=1, factor=4.0), dict(scaling=1, factor=0.25),
                                dict(scaling=2, factor=8.0, low=1.0, high=4.0, original_ctx=8192),
                                dict(scaling=3, factor=10.0, low=1.0, high=32.0, original_ctx=2048),
                                dict(scaling=3, factor=4.0, low=1.0, high=32.0, original_ctx=1)])
def test_plan_frequencies(lib, rot, theta, kw):
    t = kd.kd_rope_plan(256, theta, rot_dim=rot, magnitude=1.25, **kw)
    assert (t.head_dim, t.rot_dim, t.layout, t.magnitude) == (256, rot, kd.KD_ROPE_HALF, 1.25)
    c = dict(scaling=0, factor=1.0, low=1.0, high=4.0, original_ctx=0)
    c.update(kw)
    want = np.array([scaled(theta ** (-2.0 * i / rot), i, rot, theta, c["scaling"], c["factor"], c["low"], c["high"], c["original_ctx"])
                     for i in range(rot // 2)]) / (2 * math.pi)
    # modulo a turn: both are good to a few 2^-53 of the frequency, and the table to 2^-64 of a turn
    err = np.abs((turns(t) - want + 0.5) % 1.0 - 0.5)
    assert np.all(err <= np.abs(want) * 2.0 ** -50 + 2.0 ** -53)


TWO_PI = decimal.Decimal("6.28318530717958647692528676655900576839433879875021164194989")


@pytest.mark.parametrize("rot", [2, 6, 20, 64, 128, 250, 256])
@pytest.mark.parametrize("theta", [10000.0, 500000.0, 1.5, 1e9 / 3, 1.0 + 2.0 ** -40, 1e300])
@pytest.mark.parametrize("kw", [dict(), dict(scaling=1, factor=4.0), dict(scaling=1, factor=0.3), dict(scaling=1, factor=1e-30), dict(scaling=1, factor=1e25),
                                dict(scaling=2, factor=8.1, low=1.1, high=4.0, original_ctx=8192),
                                dict(scaling=3, factor=10.0, low=1.0, high=32.0, original_ctx=2048)])
def test_plan_turns_to_the_last_bit(lib, rot, theta, kw):
    """turns[] against 60 digits: half a unit for the rounding to 2^-64 of a turn, 2^-96 of the frequency for pairs of doubles
    (2^-104 each in some 20 operations), and the digits of 2 pi here."""
    t = kd.kd_rope_plan(256, theta, rot_dim=rot, **kw)
    with decimal.localcontext(decimal.Context(prec=110)):
        one, factor, low, high = (decimal.Decimal(x) for x in (1, kw.get("factor", 1.0), kw.get("low", 1.0), kw.get("high", 4.0)))
        ln = decimal.Decimal(theta).ln()
        for i in range(rot // 2):
            f = (-2 * ln * i / rot).exp()
            if kw.get("scaling") == 1:
                f /= factor
            elif kw.get("scaling") == 2:
                keep = min(one, max(0 * one, (kw["original_ctx"] * f / TWO_PI - low) / (high - low)))
                f *= keep + (1 - keep) / factor
            elif kw.get("scaling") == 3:
                a, b = (rot * math.log(kw["original_ctx"] / (2 * math.pi * x)) / (2 * math.log(theta)) for x in (kw["high"], kw["low"]))
                a, b = max(0, math.floor(a)), min(rot - 1, math.ceil(b))
                r = min(one, max(0 * one, decimal.Decimal(i - a) / decimal.Decimal(max(b - a, 0.001))))
                f *= 1 - r + r / factor
            want = f / TWO_PI * 2 ** 64
            off = (decimal.Decimal(t.turns[i]) - want) % 2 ** 64
            off = min(off, 2 ** 64 - off)
            assert off <= decimal.Decimal("0.5") + f * 2 ** 64 / 2 ** 96 + f * 2 ** 64 / decimal.Decimal(10) ** 58, (i, off)


@pytest.mark.parametrize("scaling", [2, 3])
@pytest.mark.parametrize("low,high", [(1.0, 1.0 + 2.0 ** -52), (5e-324, 1e-323), (1e-320, 1e308), (1e307, 1.7e308), (2.0 ** -1022, 1.0)])
@pytest.mark.parametrize("factor", [8.0, 1e-300, 1e308])
def test_plan_bands_of_any_width(lib, scaling, low, high, factor):
    """Bands so narrow or so far out that a quotient leaves a double's range: pairs keep their pace, are slowed, or between."""
    t = kd.kd_rope_plan(128, 10000.0, scaling=scaling, factor=factor, low=low, high=high, original_ctx=8192)
    keep, slowed = (kd.kd_rope_plan(128, 10000.0, **kw) for kw in (dict(), dict(scaling=1, factor=factor)))
    ends = sum(a in (b, c) for a, b, c in zip(t.turns[:64], keep.turns, slowed.turns))
    assert ends >= (0 if high == 1e308 or low == 2.0 ** -1022 else 62)
    if scaling == 2 and high < 1e-300:
        assert list(t.turns[:64]) == list(keep.turns[:64])
    if scaling == 2 and low == 1e307:
        assert list(t.turns[:64]) == list(slowed.turns[:64])


def test_plan_defaults(lib):
    t = kd.kd_rope_plan(128, 10000.0)
    assert (t.rot_dim, t.layout, t.magnitude) == (128, kd.KD_ROPE_HALF, 1.0)
    assert abs(turns(t)[0] - 1 / (2 * math.pi)) < 2.0 ** -53
    assert list(t.turns[64:]) == [0] * 64


@pytest.mark.parametrize("change,status", [
    (dict(head_dim=258), UNSUPPORTED), (dict(rot_dim=0), INVALID), (dict(rot_dim=3), INVALID), (dict(rot_dim=130), INVALID),
    (dict(rot_dim=-2), INVALID), (dict(layout=2), INVALID), (dict(scaling=4), INVALID), (dict(scaling=-1), INVALID),
    (dict(theta=1.0), INVALID), (dict(theta=float("inf")), INVALID), (dict(theta=float("nan")), INVALID),
    (dict(magnitude=float("nan")), INVALID), (dict(magnitude=1e300), INVALID),
    (dict(scaling=1, factor=0.0), INVALID), (dict(scaling=1, factor=float("nan")), INVALID), (dict(scaling=1, factor=float("inf")), INVALID),
    (dict(scaling=1, factor=5e-324), INVALID), (dict(scaling=2, original_ctx=0), INVALID), (dict(scaling=2, original_ctx=8, low=4.0, high=4.0), INVALID),
    (dict(scaling=3, original_ctx=8, low=0.0), INVALID), (dict(scaling=3, original_ctx=8, high=float("inf")), INVALID),
])
def test_plan_refusals(lib, change, status):
    a = dict(head_dim=128, theta=10000.0)
    a.update(change)
    with pytest.raises(kd.KdError) as e:
        kd.kd_rope_plan(**a)
    assert e.value.status == status and "kd_rope_plan" in str(e.value)


def test_plan_null_and_reserved(lib):
    cfg, t = kd.KdRopeConfig(128, 128, 0, 0, 0, 1, 1e4, 1, 1, 4, 1), kd.KdRopeTable()
    assert lib.kd_rope_plan(None, C.byref(t)) == INVALID
    assert lib.kd_rope_plan(C.byref(cfg), None) == INVALID
    assert lib.kd_rope_plan(C.byref(cfg), C.byref(t)) == INVALID  # reserved
    assert t.head_dim == 0


# ---------------------------------------------------------------------- kd_rope ---
def table(**kw):
    t = kd.kd_rope_plan(128, 10000.0)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


@pytest.mark.parametrize("change,status", [
    (dict(rope=None), INVALID), (dict(x=None), INVALID), (dict(pos=None), INVALID), (dict(out=None), INVALID),
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID),
    (dict(ld=4 * 128 - 1), INVALID), (dict(ld_out=511), INVALID), (dict(ld=2 ** 62), INVALID),
    (dict(x=D + 2), INVALID), (dict(out=D + 1, dtype=1), INVALID), (dict(pos=D + 2), INVALID),
    (dict(out=D, ld_out=1024), INVALID),  # in place with another row distance
    (dict(T=2 ** 31 - 1), UNSUPPORTED),
    (dict(rope=dict(rot_dim=0)), INVALID), (dict(rope=dict(rot_dim=130)), INVALID), (dict(rope=dict(head_dim=512)), INVALID),
    (dict(rope=dict(layout=2)), INVALID), (dict(rope=dict(reserved=1)), INVALID), (dict(rope=dict(magnitude=float("inf"))), INVALID),
    (dict(T=0), 0), (dict(T=0, x=None, out=None, pos=None, ld_out=1024), 0), (dict(T=0, rope=None), INVALID),
])
def test_rope_refusals(lib, change, status):
    a = dict(rope={}, x=D, dtype=0, ld=512, pos=D, T=8, H=4, out=2 * D, ld_out=512)
    a.update(change)
    t = None if a["rope"] is None else C.byref(table(**a["rope"]))
    assert lib.kd_rope(t, a["x"], a["dtype"], a["ld"], a["pos"], a["T"], a["H"], a["out"], a["ld_out"], None) == status
    if status:
        assert "kd_rope" in kd.kd_last_error()


# --------------------------------------------------------------------- append ---
def append(lib, q8=False, rope=True, k=D, v=D, q=D, kld=1024, vld=1024, qld=4096, dtype=0, kp=D, vp=D, ks=D, tab=D, tld=8,
           starts=arr(0, 3), counts=arr(5, 1), n=2, nh=32, nkv=8, hd=128, n_pages=16, ps=16, q_out=D, fault=D):
    t = C.byref(table(**({} if rope is True else rope))) if rope is not None else None
    a = (t, k, kld, v, vld, q, qld, dtype)
    b = (tab, tld, p(starts), p(counts), n, nh, nkv)
    if q8:
        return lib.kd_paged_append_q8(*a, kp, ks, vp, D, *b, n_pages, ps, q_out, fault, None)
    return lib.kd_paged_append(*a, kp, vp, *b, hd, n_pages, ps, q_out, fault, None)


@pytest.mark.parametrize("change,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(q=None), INVALID), (dict(q_out=None), INVALID), (dict(kp=None), INVALID),
    (dict(vp=None), INVALID), (dict(tab=None), INVALID), (dict(starts=None), INVALID), (dict(counts=None), INVALID),
    (dict(nh=0), INVALID),  # queries without heads
    (dict(n=0), BATCH), (dict(n=257), BATCH), (dict(hd=96), UNSUPPORTED), (dict(hd=64), INVALID),  # the rotation's heads
    (dict(ps=0), UNSUPPORTED), (dict(ps=24), UNSUPPORTED), (dict(ps=65552), UNSUPPORTED), (dict(ps=-16), UNSUPPORTED),
    (dict(dtype=3), INVALID), (dict(nkv=0), INVALID), (dict(nh=-1), INVALID), (dict(n_pages=0), INVALID), (dict(tld=0), INVALID),
    (dict(nkv=2 ** 30), UNSUPPORTED),
    (dict(rope=dict(rot_dim=5)), INVALID),
    (dict(kld=1023), INVALID), (dict(vld=0), INVALID), (dict(qld=4095), INVALID), (dict(kld=2 ** 62), INVALID),
    (dict(k=D + 2), INVALID), (dict(kp=D + 8), INVALID), (dict(q_out=D + 8), INVALID), (dict(tab=D + 2), INVALID), (dict(fault=D + 1), INVALID),
    (dict(starts=arr(-1, 3)), POSITION), (dict(counts=arr(5, -1)), POSITION), (dict(starts=arr(0, 128)), POSITION),
    (dict(starts=arr(124, 3)), POSITION), (dict(starts=arr(2 ** 31 - 1, 0), counts=arr(2 ** 31 - 1, 0)), POSITION),
    (dict(tld=2 ** 27, counts=arr(2 ** 30, 2 ** 30)), UNSUPPORTED), (dict(tld=2 ** 30, starts=arr(2 ** 31 - 1, 0), counts=arr(1, 0)), POSITION),
    (dict(counts=arr(0, 0)), 0), (dict(counts=arr(0, 0), rope=None, fault=None, nh=0, q=None, q_out=None), 0),
])
@pytest.mark.parametrize("q8", [False, True])
def test_append_refusals(lib, q8, change, status):
    if q8 and "hd" in change:
        pytest.skip("the Q8_0 form has one head_dim")
    assert append(lib, q8, **change) == status, kd.kd_last_error()
    if status:
        assert ("kd_paged_append_q8" if q8 else "kd_paged_append") in kd.kd_last_error()


def test_append_q8_scales(lib):
    assert append(lib, True, ks=None) == INVALID
    assert append(lib, True, ks=D + 8) == INVALID


# ------------------------------------------------------------------ attention ---
def attn(lib, q8=False, q=D, kp=D, vp=D, ks=D, tab=D, tld=8, lens=arr(5, 100), B=2, rows=None, prefix=None, G=0, nh=32, nkv=8, hd=128,
         n_pages=16, ps=16, out=D, ws=D, ws_bytes=1 << 30, fault=D):
    b = (tab, tld, p(lens), B, p(rows), p(prefix), G, nh, nkv)
    if q8:
        return lib.kd_attn_paged_decode_q8(q, kp, ks, vp, D, *b, n_pages, ps, out, ws, ws_bytes, fault, None)
    return lib.kd_attn_paged_decode(q, kp, vp, *b, hd, n_pages, ps, out, ws, ws_bytes, fault, None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(kp=None), INVALID), (dict(vp=None), INVALID), (dict(tab=None), INVALID), (dict(lens=None), INVALID),
    (dict(out=None), INVALID), (dict(ws=None), INVALID), (dict(G=1), INVALID), (dict(G=1, rows=arr(2)), INVALID),
    (dict(B=0), BATCH), (dict(B=257), BATCH),
    (dict(hd=96), UNSUPPORTED), (dict(nh=24), UNSUPPORTED), (dict(nh=30), UNSUPPORTED), (dict(nh=128), UNSUPPORTED), (dict(nkv=0), UNSUPPORTED),
    (dict(nkv=1025, nh=1025), UNSUPPORTED), (dict(ps=8), UNSUPPORTED), (dict(ps=40), UNSUPPORTED), (dict(ps=1 << 17), UNSUPPORTED),
    (dict(n_pages=0), INVALID), (dict(tld=0), INVALID), (dict(G=-1), INVALID), (dict(n_pages=1 << 24), UNSUPPORTED),
    (dict(ws_bytes=4096), INVALID), (dict(ws=D + 8), INVALID), (dict(q=D + 8), INVALID), (dict(kp=D + 8), INVALID), (dict(tab=D + 2), INVALID),
    (dict(out=D + 1), INVALID), (dict(fault=D + 2), INVALID),
    (dict(lens=arr(-1, 5)), POSITION), (dict(lens=arr(5, 129)), POSITION), (dict(tld=2 ** 27, lens=arr(5, 2 ** 30 + 1)), POSITION),
    (dict(G=1, rows=arr(2), prefix=arr(6)), POSITION), (dict(G=1, rows=arr(2), prefix=arr(-1)), POSITION),
    (dict(G=1, rows=arr(1), prefix=arr(0)), INVALID), (dict(G=2, rows=arr(1, 2), prefix=arr(0, 0)), INVALID),
    (dict(G=2, rows=arr(0, 2), prefix=arr(0, 0)), INVALID), (dict(G=2, rows=arr(2, 2 ** 31 - 1), prefix=arr(0, 0)), INVALID),
])
@pytest.mark.parametrize("q8", [False, True])
def test_attention_refusals(lib, q8, change, status):
    if q8 and "hd" in change:
        pytest.skip("the Q8_0 form has one head_dim")
    assert attn(lib, q8, **change) == status, kd.kd_last_error()
    assert ("kd_attn_paged_decode_q8" if q8 else "kd_attn_paged_decode") in kd.kd_last_error()


def test_attention_q8_scales(lib):
    assert attn(lib, True, ks=None) == INVALID
    assert attn(lib, True, ks=D + 8) == INVALID


def test_workspace_bytes(lib):
    f = kd.kd_attn_paged_workspace_bytes
    assert f(1, 32, 8, 128) > 256 and f(256, 8192, 1024, 64) > f(255, 8192, 1024, 64) > 0
    for a in [(0, 32, 8, 128), (257, 32, 8, 128), (1, 30, 8, 128), (1, 32, 8, 96), (1, 0, 8, 128), (1, 1025, 1025, 64)]:
        assert f(*a) == 0


# The rule's sides: (rows, 8 KV heads of gq queries, heads of hd, Q8_0) -> the least MB of other sessions' reading.
@pytest.mark.parametrize("q8,hd,gq,rows,least", [(0, 128, 1, 2, 24), (0, 128, 8, 256, 24), (0, 64, 4, 2, None), (0, 64, 4, 3, 24), (0, 64, 1, 60, 24),
                                                 (1, 128, 4, 2, None), (1, 128, 4, 3, None), (1, 128, 4, 4, 24), (1, 128, 1, 90, 24), (1, 128, 8, 2, 40),
                                                 (1, 128, 8, 3, 16), (0, 128, 4, 1, None), (1, 128, 8, 1, None)])
def test_reads_once(lib, q8, hd, gq, rows, least):
    row = 8 * (272 if q8 else 4 * hd)
    once = lambda keys, page=16: kd.kd_attn_paged_reads_once(rows, keys, 8 * gq, 8, hd, page, q8)
    if least is None:
        assert not once(1 << 30) and not once(0)
        return
    keys = -(-(least << 20) // ((rows - 1) * row))  # the fewest that save this much
    pages = -(-keys // 16) * 16
    assert once(pages) and not once(pages - 1) and once(1 << 30)  # whole pages count
    assert once(pages, 65536) == (pages % 65536 == 0)


def test_reads_once_refuses_like_the_call(lib):
    assert kd.kd_attn_paged_reads_once(16, 1 << 16, 32, 8, 128, 16)
    for a in ((0, 1 << 16, 32, 8, 128, 16), (257, 1 << 16, 32, 8, 128, 16), (16, -1, 32, 8, 128, 16), (16, (1 << 30) + 1, 32, 8, 128, 16),
              (16, 1 << 16, 30, 8, 128, 16), (16, 1 << 16, 32, 8, 96, 16), (16, 1 << 16, 32, 8, 128, 24), (16, 1 << 16, 32, 8, 128, 1 << 17),
              (16, 1 << 16, 32, 8, 64, 16, True), (16, 1 << 16, 1025, 1025, 128, 16)):
        assert not kd.kd_attn_paged_reads_once(*a), a


# -------------------------------------------------------------------- binding ---
def test_binding_shapes_and_types(calls):
    plan = kd.kd_rope_plan(64, 10000.0)
    x, pos = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int32)
    for bad in (dict(x=torch.zeros(3, 64, 2).transpose(1, 2)), dict(x=torch.zeros(3, 2, 64, dtype=torch.float64)), dict(x=torch.zeros(6, 64)),
                dict(x=torch.zeros(3, 4, 64)[:, ::2]), dict(out=torch.zeros(3, 2, 64, dtype=torch.float16)), dict(out=torch.zeros(2, 2, 64)),
                dict(pos=torch.zeros(2, dtype=torch.int32)), dict(pos=torch.zeros(3, dtype=torch.int64)), dict(pos=torch.zeros(3)),
                dict(x=torch.zeros(3, 2, 32), out=torch.zeros(3, 2, 32))):
        a = dict(x=x, pos=pos, out=x.clone())
        a.update(bad)
        with pytest.raises(ValueError):
            kd.kd_rope(plan, a["x"], a["pos"], a["out"])
    with pytest.raises(kd.KdError, match="in place"):
        wide = torch.zeros(3, 4, 64)
        kd.kd_rope(plan, wide.as_strided((3, 2, 64), (128, 64, 1)), pos, wide[:, :2])


def test_binding_append(calls):
    pages = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    k = torch.zeros(5, 2, 64)
    tab = torch.zeros(2, 3, dtype=torch.int32)

    def call(k=k, v=k, tab=tab, starts=(0, 0), counts=(2, 3), **kw):
        kd.kd_paged_append(None, k, v, pages, pages, tab, starts, counts, 2, 64, 4, 16, **kw)
    with pytest.raises(ValueError, match="5 new rows for counts of 4"):
        call(counts=[1, 3])
    with pytest.raises(kd.KdError, match="-3 rows"):
        call(counts=[2, -3])
    with pytest.raises(kd.KdError, match="from position 46 on"):
        call(starts=np.array([0, 46], np.int64))
    with pytest.raises(ValueError, match="expected 2 entries"):
        call(counts=[5])
    with pytest.raises(ValueError, match="alike"):
        call(v=torch.zeros(5, 2, 64, dtype=torch.float16))
    with pytest.raises(ValueError, match="alike"):
        call(k=torch.zeros(5, 2, 128), v=torch.zeros(5, 2, 128))
    for bad in (torch.zeros(1, 3, dtype=torch.int32), torch.zeros(2, 3), torch.zeros(6, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int64)):
        with pytest.raises(ValueError, match="page table"):
            call(tab=bad)
    with pytest.raises(ValueError, match="contiguous"):
        call(tab=torch.zeros(3, 2, dtype=torch.int32).t())
    q = torch.zeros(5, 4, 64)
    for bad in (dict(q_out=torch.zeros(5, 4, 64, dtype=torch.float16)), dict(q_out=torch.zeros(5, 8, 64)[:, :4]), dict(q_out=torch.zeros(4, 4, 64)),
                dict(q=torch.zeros(4, 4, 64), q_out=q), dict(q_out=q, n_heads=3)):
        a = dict(q=q, q_out=q, n_heads=4)
        a.update(bad)
        with pytest.raises(ValueError, match="q must be"):
            call(**a)
    with pytest.raises(kd.KdError, match="heads of 64 for head_dim 128"):
        big = torch.zeros(1, 1, 128)
        kd.kd_paged_append(kd.kd_rope_plan(64, 1e4), big, big, pages, pages, tab, [0], [1], 1, 128, 4, 16)


def test_binding_attention(calls):
    pages = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    q, out = torch.zeros(2, 4, 64), torch.zeros(2, 256, dtype=torch.float16)
    tab, ws = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(kd.kd_attn_paged_workspace_bytes(2, 4, 2, 64), dtype=torch.uint8)

    def call(lens=(5, 6), tab=tab, ws=ws, **kw):
        kd.kd_attn_paged_decode(q, pages, pages, tab, lens, 4, 2, 64, 4, 16, out, ws, **kw)
    with pytest.raises(kd.KdError, match="length 49"):
        call(lens=np.array([0, 49]))
    with pytest.raises(kd.KdError, match="workspace too small"):
        call(ws=ws[:1024])
    with pytest.raises(kd.KdError, match="prefix 6 of a session of length 5"):
        call(group_rows=[2], group_prefix=[6])
    with pytest.raises(ValueError):
        call(group_rows=[2])
    with pytest.raises(ValueError):
        call(group_rows=[1, 1], group_prefix=[3])
    with pytest.raises(ValueError, match="page table"):
        call(lens=[1, 2, 3])
    with pytest.raises(ValueError, match="contiguous"):
        kd.kd_attn_paged_decode(torch.zeros(2, 4, 128)[:, :, :64], pages, pages, tab, [1, 1], 4, 2, 64, 4, 16, out, ws)


def test_binding_sizes(calls):
    """q, out and the cache's planes have what the call's sizes say."""
    pages, small = (torch.zeros(n, 2, 16, 64, dtype=torch.float16) for n in (4, 3))
    k, tab = torch.zeros(1, 2, 64), torch.zeros(1, 3, dtype=torch.int32)
    for planes in ((pages, small), (small, pages)):
        with pytest.raises(ValueError, match="a plane of the cache"):
            kd.kd_paged_append(None, k, k, *planes, tab, [0], [1], 2, 64, 4, 16)
    q, out, ws = torch.zeros(1, 4, 64), torch.zeros(1, 256, dtype=torch.float16), torch.zeros(kd.kd_attn_paged_workspace_bytes(1, 4, 2, 64), dtype=torch.uint8)
    for change, what in ((dict(q=q.half()), "q"), (dict(out=out[:, :255].contiguous()), "out"), (dict(k=small), "a plane"), (dict(v=small), "a plane")):
        a = dict(q=q, k=pages, v=pages, out=out)
        a.update(change)
        with pytest.raises(ValueError, match=what + ".* is smaller"):
            kd.kd_attn_paged_decode(a["q"], a["k"], a["v"], tab, [3], 4, 2, 64, 4, 16, a["out"], ws)
    quants, scales = torch.zeros(4, 2, 16, 128, dtype=torch.uint8), torch.zeros(4, 2, 16, 4, dtype=torch.float16)
    for i in range(4):
        planes = [quants, scales, quants, scales]
        planes[i] = planes[i][:3]
        with pytest.raises(ValueError, match="a plane of the cache"):
            kd.kd_attn_paged_decode_q8(torch.zeros(1, 4, 128), *planes, tab, [3], 4, 2, 4, 16, torch.zeros(1, 512, dtype=torch.float16), ws)
        with pytest.raises(ValueError, match="a plane of the cache"):
            kd.kd_paged_append_q8(None, torch.zeros(1, 2, 128), torch.zeros(1, 2, 128), *planes, tab, [0], [1], 2, 4, 16)


def test_nothing_to_do(calls):
    """No tokens, or no new row in any session: torch's empty tensors have no address."""
    plan = kd.kd_rope_plan(64, 1e4)
    x = torch.zeros(0, 2, 64)
    assert x.data_ptr() == 0
    kd.kd_rope(plan, x, torch.zeros(0, dtype=torch.int32), x)
    kd.kd_rope(plan, torch.zeros(4, 4, 64)[:0, :2], torch.zeros(0, dtype=torch.int32), x)
    pages, tab = torch.zeros(4, 2, 16, 64, dtype=torch.float16), torch.zeros(2, 3, dtype=torch.int32)
    for kw in (dict(), dict(q=torch.zeros(0, 4, 64), q_out=torch.zeros(0, 4, 64), n_heads=4)):
        kd.kd_paged_append(plan, x, x, pages, pages, tab, [5, 9], [0, 0], 2, 64, 4, 16, **kw)
    with pytest.raises(kd.KdError, match="position"):
        kd.kd_paged_append(plan, x, x, pages, pages, tab, [5, 49], [0, 0], 2, 64, 4, 16)
