"""Rotary positions, paged append and paged attention on the GPU against plain fp64.

Tolerances, per element (derived; u = x_a, w = x_b the pair, m the magnitude):
- Rotation.  The angle of position p is p f, of which f is good to 2^-50 relative
  (pow, the division by a turn and the reference's own product) and a whole multiple of
  2^-64 turns absolutely: p times the rounding to one is |p| 2 pi 2^-65 (2^-64 where the
  rest is cut off), which is more than the relative part for slow pairs: at p = 2^31 and f = 3e-5 it is
  3.7e-10, |p| f 2^-50 = 5.7e-11.  So a result moves by at most |p| (f 2^-50 + 2 pi 2^-64)
  (|u| + |w|) m.  fp32: cosine, sine and products are carried to about
  2^-44 and rounded once: 2^-40 (|u| + |w|) m + 2^-24 |y|.  16 bits: cosine and sine to
  2^-23, three products and a sum of 2^-24: 2^-21 (|u| + |w|) m, and the rounding of y, 2^-11
  (fp16; 2^-25 below its normal range) or 2^-8 (bf16).
- Q8_0 rows: the codes of the fp64 rotation rounded to fp32; equal bit for bit, since
  neither side's error (2^-44) moves an fp32 rounding that matters.
- Attention, o = sum_t p_t v_t.  Scores: q as an fp16 pair loses 2^-21 |q|, the products'
  fp32 sums at most hd/16 + 1 truncated adds of 2^-23, so a score moves by at most S (2^-21
  + 9 2^-23), S = max_t sum_i |q_i k_ti| / sqrt(hd).  Weights: twice that (numerator and
  denominator) plus 2^-21 (expf, p's pair); a key's weight passes at most len/32 + 20
  further sums or products with a rescaling factor (its chain's pieces, warps, records), 2^-22
  each.  (On the fifth-generation tensor cores, where prefixes are read once, a sum takes up to three
  times as many in the worst case; it is held to the same bound.)  So o moves by at most eps sum_t p_t |v_t|; then it is rounded to fp16 once."""
import math
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

HALF, PAIRS = 0, 1
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
ROUND = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"fp32": 2.0 ** -149, "fp16": 2.0 ** -25, "bf16": 2.0 ** -134}


# ------------------------------------------------------------------ rotation ---
def frequencies(rot, theta, scaling="none", factor=1.0, low=1.0, high=4.0, original=8192):
    i = np.arange(rot // 2)
    f = theta ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor
    if scaling == "bands":
        keep = np.clip((original * f / (2 * math.pi) - low) / (high - low), 0, 1)
        return f * (keep + (1 - keep) / factor)
    if scaling == "ramp":
        a, b = (rot * math.log(original / (2 * math.pi * n)) / (2 * math.log(theta)) for n in (high, low))
        a, b = max(0, math.floor(a)), min(rot - 1, math.ceil(b))
        r = np.clip((i - a) / max(b - a, 0.001), 0, 1)
        return f * (1 - r + r / factor)
    return f


def rotate(x, pos, f, layout, magnitude=1.0):
    """x fp64 [T][H][hd]: the rotated values, the error that its angles and cosines allow (fp32 and 16 bits)."""
    n = 2 * len(f)
    w = pos.astype(np.float64)[:, None] * f
    c, s = (np.cos(w) * magnitude)[:, None], (np.sin(w) * magnitude)[:, None]
    a, b = (slice(0, n // 2), slice(n // 2, n)) if layout == HALF else (slice(0, n, 2), slice(1, n, 2))
    y = x.copy()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    size = np.zeros_like(x)
    size[..., a] = size[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(magnitude)
    angle = np.zeros_like(x)
    angle[..., a] = angle[..., b] = (np.abs(w) * 2.0 ** -50 + np.abs(pos.astype(np.float64))[:, None] * 2 * math.pi * 2.0 ** -64)[:, None]  # in fp64: the least int32 has no absolute value of its type
    return y, (angle + 2.0 ** -40) * size, (angle + 2.0 ** -21) * size


def check_rotated(got, x, pos, f, layout, magnitude, kind, in_fp32=False):
    y, exact, fast = rotate(x.double().cpu().numpy(), pos, f, layout, magnitude)
    tol = (exact if kind == "fp32" or in_fp32 else fast) + ROUND[kind] * np.abs(y) + TINY[kind]
    if in_fp32:
        tol += 2.0 ** -24 * np.abs(y)
    err = np.abs(got.double().cpu().numpy() - y)
    assert np.all(err <= tol), (kind, float((err / tol).max()), np.unravel_index((err / tol).argmax(), err.shape))


SCALED = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="bands", factor=8.0, low=1.0, high=4.0, original=8192),
          dict(scaling="ramp", factor=10.0, low=1.0, high=32.0, original=2048)]


def kd_plan(kd, hd):
    return kd.kd_rope_plan(hd, 10000.0)


def make_plan(kd, hd, rot, theta, layout, magnitude=1.0, scaling="none", factor=1.0, low=1.0, high=4.0, original=8192):
    code = {"none": kd.KD_ROPE_UNSCALED, "linear": kd.KD_ROPE_LINEAR, "bands": kd.KD_ROPE_BANDS, "ramp": kd.KD_ROPE_RAMP}
    return kd.kd_rope_plan(hd, theta, rot_dim=rot, layout=layout, scaling=code[scaling], factor=factor, low=low, high=high,
                           original_ctx=original, magnitude=magnitude)


def normal(seed, shape, kind="fp32"):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32)).cuda().to(TYPES[kind])


@pytest.mark.parametrize("kind", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("layout", [HALF, PAIRS])
@pytest.mark.parametrize("hd,rot", [(128, 128), (128, 64), (64, 64), (64, 34), (128, 2), (256, 256), (24, 20), (96, 96),
                                    (16, 16), (2, 2), (7, 6), (250, 12), (128, 86), (80, 6), (192, 190)])
def test_rope_shapes(kdlib, kind, layout, hd, rot):
    for t, h in ((1, 1), (3, 5), (17, 33)):
        x = normal(hd + rot + t, (t, h, hd), kind)
        pos = np.random.default_rng(t).integers(-5, 100000, t).astype(np.int32)
        out = torch.full_like(x, float("nan"))
        kdlib.kd_rope(make_plan(kdlib, hd, rot, 10000.0, layout), x, torch.from_numpy(pos).cuda(), out)
        check_rotated(out, x, pos, frequencies(rot, 10000.0), layout, 1.0, kind)
        assert torch.equal(out[..., rot:], x[..., rot:])


@pytest.mark.parametrize("scaled", SCALED)
@pytest.mark.parametrize("layout", [HALF, PAIRS])
def test_rope_scaled_far_positions(kdlib, scaled, layout):
    pos = np.array([0, 1, -1, 2, 63, 64, 4095, 4096, 100000, -100000, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31], np.int32)
    for theta in (10000.0, 500000.0):
        f = frequencies(128, theta, **scaled)
        for magnitude in (1.0, 1.2302585092994046):
            plan = make_plan(kdlib, 128, 128, theta, layout, magnitude, **scaled)
            for kind in ("fp32", "fp16"):
                x = normal(7, (len(pos), 3, 128), kind)
                out = torch.empty_like(x)
                kdlib.kd_rope(plan, x, torch.from_numpy(pos).cuda(), out)
                check_rotated(out, x, pos, f, layout, magnitude, kind)


def test_rope_many_tokens_in_place_strided_and_back(kdlib):
    T, nh, nkv, hd = 2053, 8, 2, 128
    plan = make_plan(kdlib, hd, hd, 500000.0, HALF)
    f = frequencies(hd, 500000.0)
    for kind in ("fp32", "bf16"):
        fused = normal(3, (T, nh + 2 * nkv, hd), kind)
        before = fused.clone()
        pos = torch.arange(T, dtype=torch.int32, device="cuda") + 777
        q = fused[:, :nh]
        kdlib.kd_rope(plan, q, pos, q)  # in place, in the fused rows
        check_rotated(q, before[:, :nh], pos.cpu().numpy(), f, HALF, 1.0, kind)
        assert torch.equal(fused[:, nh:], before[:, nh:])
        kdlib.kd_rope(plan, q, -pos, q)
        err = (q.double() - before[:, :nh].double()).abs().max().item()
        assert err <= 5.0 * 4 * ROUND[kind] * 2, err  # |x| < 5 (seeded); two roundings of a sum of two, and of the pair


def test_rope_non_finite_values_and_positions_by_token(kdlib):
    plan = make_plan(kdlib, 64, 64, 10000.0, HALF)
    x = normal(1, (4, 2, 64))
    x[1, 0, 3] = float("inf")
    x[2, 1, 40] = float("nan")
    pos = torch.tensor([5, 0, 9, 5], dtype=torch.int32, device="cuda")
    out = torch.empty_like(x)
    kdlib.kd_rope(plan, x, pos, out)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[1, 0, [3, 35]] = True
    want[2, 1, [8, 40]] = True
    assert torch.equal(bad, want)
    assert out[1, 0, 3] == float("inf")
    assert torch.equal(out[1, 1], x[1, 1])  # position 0 is the identity


# -------------------------------------------------------------------- append ---
def values_of(quants, scales):
    q, s = quants.cpu().numpy().astype(np.float64) - 128, scales.cpu().numpy().astype(np.float64)
    return (q.reshape(*q.shape[:-1], 4, 32) * s[..., None]).reshape(q.shape)


class Pages:
    """A pool of pages (NaN, or NaN scales, everywhere) and a table of scattered pages for sessions of given lengths."""

    def __init__(self, q8, n_kv, hd, ps, lens, seed, spare=2):
        rng = np.random.default_rng(seed)
        self.q8, self.n_kv, self.hd, self.ps = q8, n_kv, hd, ps
        need = [-(-n // ps) for n in lens]
        self.n_pages = sum(need) + spare
        ids = rng.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((len(lens), max(need + [1]) + 1), 2 ** 30, np.int32)  # behind a session's pages: never looked up
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        shape = (self.n_pages, n_kv, ps)
        if q8:
            self.planes = [t for _ in range(2) for t in (torch.full((*shape, 128), 0x5A, dtype=torch.uint8, device="cuda"),
                                                         torch.full((*shape, 4), float("nan"), dtype=torch.float16, device="cuda"))]
        else:
            self.planes = [torch.full((*shape, hd), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2)]

    def device_table(self):
        return torch.from_numpy(self.table).cuda()

    def rows(self, part, b, t0, t1):
        """Rows t0 .. t1 of session b as they lie in the pages: [n][n_kv][...] per plane of the part."""
        t = np.arange(t0, t1)
        page, row = torch.from_numpy(self.table[b, t // self.ps].astype(np.int64)).cuda(), torch.from_numpy(t % self.ps).cuda()
        n = len(self.planes) // 2
        return [p[page, :, row] for p in self.planes[part * n:part * n + n]]


def bits(t):
    return t.view(torch.int16) if t.dtype == torch.float16 else t


@pytest.mark.parametrize("q8,hd", [(False, 128), (False, 64), (True, 128)])
@pytest.mark.parametrize("kind,layout,rot,nh,ps", [("fp32", HALF, None, 0, 16), ("fp16", HALF, 64, 4, 48), ("bf16", PAIRS, None, 16, 64),
                                                   ("fp32", HALF, 12, 2, 32), ("fp16", PAIRS, 34, 2, 256), ("fp32", None, None, 2, 16)])
def test_append(kdlib, q8, hd, kind, layout, rot, nh, ps):
    kd, nkv = kdlib, 2
    starts = np.array([0, 5, 61, 0, 1000, 15], np.int32)
    counts = np.array([1, 3, 70, 0, 129, 1], np.int32)
    T = int(counts.sum())
    pool = Pages(q8, nkv, hd, ps, list(starts + counts), 5)
    before = [p.clone() for p in pool.planes]
    rot = rot or hd
    plan = None if layout is None else make_plan(kd, hd, rot, 10000.0, layout, 1.25)
    fused = normal(11, (T, nh + 2 * nkv, hd), kind)
    q, k, v = fused.split([nh, nkv, nkv], 1)
    q_out = torch.full((T, nh, hd), float("nan"), device="cuda")
    fault = torch.zeros(1, dtype=torch.int32, device="cuda")
    extra = dict(q=q, q_out=q_out, n_heads=nh) if nh else {}
    if q8:
        kd.kd_paged_append_q8(plan, k, v, *pool.planes, pool.device_table(), starts, counts, nkv, pool.n_pages, ps, fault=fault, **extra)
    else:
        kd.kd_paged_append(plan, k, v, *pool.planes, pool.device_table(), starts, counts, nkv, hd, pool.n_pages, ps, fault=fault, **extra)
    assert fault.item() == 0
    pos = np.concatenate([np.arange(n) + s for s, n in zip(starts, counts)]).astype(np.int64)
    f = frequencies(rot, 10000.0) if plan else np.zeros(0)
    if nh:
        if plan:
            check_rotated(q_out, q, pos, f, layout, 1.25, "fp32")
        else:
            assert torch.equal(q_out, q.float())
    at = 0
    for b, (s, n) in enumerate(zip(starts, counts)):
        kb, vb, pb = k[at:at + n], v[at:at + n], pos[at:at + n]
        at += n
        if not n:
            continue
        if not q8:
            (gk,), (gv,) = pool.rows(0, b, s, s + n), pool.rows(1, b, s, s + n)
            assert torch.equal(gv, vb.float().half())
            if plan:
                check_rotated(gk, kb, pb, f, layout, 1.25, "fp16", in_fp32=True)
            else:
                assert torch.equal(gk, kb.float().half())
            continue
        y = kb.double().cpu().numpy()
        if plan:
            y = rotate(y, pb, f, layout, 1.25)[0]
        for part, x in ((0, y.astype(np.float32)), (1, vb.float().cpu().numpy())):
            blk = oracle.q8_0_quantize_f32(np.ascontiguousarray(x)).reshape(n, nkv, 4, 34)
            quant = (np.ascontiguousarray(blk[..., 2:]).view(np.int8).astype(np.int16) + 128).astype(np.uint8).reshape(n, nkv, 128)
            scale = np.ascontiguousarray(blk[..., :2]).view(np.uint16).reshape(n, nkv, 4)
            gq, gs = pool.rows(part, b, s, s + n)
            assert np.array_equal(gq.cpu().numpy(), quant)
            assert np.array_equal(gs.cpu().numpy().view(np.uint16), scale)
    # everything else is as it was
    for p, o in zip(pool.planes, before):
        touched = torch.zeros(p.shape[0], p.shape[2], dtype=torch.bool, device="cuda")
        for b, (s, n) in enumerate(zip(starts, counts)):
            t = np.arange(s, s + n)
            touched[torch.from_numpy(pool.table[b, t // ps].astype(np.int64)).cuda(), torch.from_numpy(t % ps).cuda()] = True
        keep = ~touched[:, None].expand(-1, nkv, -1)
        assert torch.equal(bits(p)[keep], bits(o)[keep])


def test_append_unaligned_inputs(kdlib):
    """Heads that start on odd elements, rows an odd distance apart."""
    for kind in ("fp32", "fp16"):
        T, nkv, hd = 9, 3, 64
        buf = normal(2, (T * 2 * (nkv * hd + 1) + 3,), kind)
        ld = 2 * nkv * hd + 1
        k = buf[1:].as_strided((T, nkv, hd), (ld, hd, 1))
        v = buf[1 + nkv * hd:].as_strided((T, nkv, hd), (ld, hd, 1))
        pool = Pages(False, nkv, hd, 16, [T], 1)
        plan = make_plan(kdlib, hd, hd, 10000.0, HALF)
        kdlib.kd_paged_append(plan, k, v, *pool.planes, pool.device_table(), [0], [T], nkv, hd, pool.n_pages, 16)
        (gk,), (gv,) = pool.rows(0, 0, 0, T), pool.rows(1, 0, 0, T)
        assert torch.equal(gv, v.float().half())
        check_rotated(gk, k, np.arange(T), frequencies(hd, 10000.0), HALF, 1.0, "fp16", in_fp32=True)
        x = buf[1:].as_strided((T, nkv, hd), (ld, hd, 1))
        out = torch.empty(T, nkv, hd, dtype=buf.dtype, device="cuda")
        kdlib.kd_rope(plan, x, torch.arange(T, dtype=torch.int32, device="cuda"), out)
        check_rotated(out, x, np.arange(T), frequencies(hd, 10000.0), HALF, 1.0, kind)


def test_append_many_sessions_and_long_prompts(kdlib):
    kd, nkv, hd, ps = kdlib, 8, 128, 32
    rng = np.random.default_rng(0)
    plan = make_plan(kd, hd, hd, 500000.0, HALF)
    f = frequencies(hd, 500000.0)
    for n_seqs, most in ((256, 3), (3, 4001)):
        counts = rng.integers(0, most + 1, n_seqs).astype(np.int32)
        counts[-1] = most
        starts = rng.integers(0, 5000, n_seqs).astype(np.int32)
        T = int(counts.sum())
        pool = Pages(False, nkv, hd, ps, list(starts + counts), n_seqs)
        k, v = normal(1, (T, nkv, hd), "fp16"), normal(2, (T, nkv, hd), "fp16")
        kd.kd_paged_append(plan, k, v, *pool.planes, pool.device_table(), starts, counts, nkv, hd, pool.n_pages, ps)
        at = 0
        for b, (s, n) in enumerate(zip(starts, counts)):
            if n:
                (gk,), (gv,) = pool.rows(0, b, s, s + n), pool.rows(1, b, s, s + n)
                assert torch.equal(gv, v[at:at + n])
                check_rotated(gk, k[at:at + n], np.arange(s, s + n), f, HALF, 1.0, "fp16", in_fp32=True)
            at += n


@pytest.mark.parametrize("q8", [False, True])
def test_append_bad_pages(kdlib, q8):
    kd, nkv, hd, ps = kdlib, 2, 128, 16
    pool = Pages(q8, nkv, hd, ps, [40, 40], 3)
    good = pool.table.copy()
    pool.table[0, 1], pool.table[1, 2] = -1, pool.n_pages
    before = [p.clone() for p in pool.planes]
    k, v = normal(1, (80, nkv, hd)), normal(2, (80, nkv, hd))
    fault = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = (None, k, v, *pool.planes, pool.device_table(), [0, 0], [40, 40], nkv)
    if q8:
        kd.kd_paged_append_q8(*a, pool.n_pages, ps, fault=fault)
        kd.kd_paged_append_q8(*a, pool.n_pages, ps)  # nobody asks
    else:
        kd.kd_paged_append(*a, hd, pool.n_pages, ps, fault=fault)
        kd.kd_paged_append(*a, hd, pool.n_pages, ps)
    assert fault.item() == 1
    for p, o in zip(pool.planes, before):
        for page in (good[0, 1], good[1, 2]):
            assert torch.equal(bits(p[page]), bits(o[page]))
        assert not torch.equal(bits(p[int(good[0, 0])]), bits(o[int(good[0, 0])]))


# ----------------------------------------------------------------- attention ---
def reference(q, K, V):
    """q [group][hd], K, V [keys][hd] in fp64 -> outputs and their tolerances."""
    n, hd = K.shape
    if n == 0:
        return np.zeros_like(q), np.zeros_like(q)
    s = q @ K.T / np.sqrt(hd)
    S = (np.abs(q) @ np.abs(K).T).max(1, keepdims=True) / np.sqrt(hd)
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    o = p @ V
    eps = 2 * S * (2.0 ** -21 + 9 * 2.0 ** -23) + 2.0 ** -21 + (n / 32 + 20) * 2.0 ** -22
    return o, 2.0 ** -11 * np.abs(o) + 2.0 ** -25 + eps * (p @ np.abs(V))


class Attn:
    """Sessions over scattered pages, in groups (sizes, prefixes) that share the whole pages of their prefixes."""

    def __init__(self, q8, nh, nkv, hd, ps, lens, groups=(), seed=0, kscale=1.0, vscale=1.0):
        rng = np.random.default_rng(seed)
        self.q8, self.nh, self.nkv, self.hd, self.ps = q8, nh, nkv, hd, ps
        self.lens = np.array(lens, np.int32)
        self.rows = np.array([g[0] for g in groups], np.int32)
        self.prefix = np.array([g[1] for g in groups], np.int32)
        self.pool = Pages(q8, nkv, hd, ps, lens, seed)
        B = len(lens)
        self.q = (rng.standard_normal((B, nh, hd)) * kscale).astype(np.float32)
        self.kv = []  # per session K, V as fp64 values [nkv][len][hd]
        first = 0
        lead_of, shared = list(range(B)), [0] * B
        for size, prefix in groups:
            for b in range(first, first + size):
                lead_of[b], shared[b] = first, prefix
            first += size
        table = self.pool.table
        for b in range(B):
            n, lead, p = int(lens[b]), lead_of[b], shared[b]
            x = [rng.standard_normal((nkv, n, hd)) * s for s in (1.0, vscale)]
            if lead != b:
                for i in range(2):
                    x[i][:, :p] = self.kv[lead][i][:, :p]
            vals = []
            page = torch.from_numpy(table[b, np.arange(n) // ps].astype(np.int64)).cuda()
            row = torch.from_numpy(np.arange(n) % ps).cuda()
            for i in range(2):
                if q8:
                    blk = oracle.q8_0_quantize_f32(x[i].astype(np.float32)).reshape(nkv, n, 4, 34) if n else np.zeros((nkv, 0, 4, 34), np.uint8)
                    quant = np.ascontiguousarray(blk[..., 2:]).view(np.int8)
                    scale = np.ascontiguousarray(blk[..., :2]).view(np.float16).reshape(nkv, n, 4)
                    if lead != b and p:  # the very rows of the shared part, in the own copy of the page it ends in too
                        quant[:, :p], scale[:, :p] = self.raw[lead][i][0][:, :p], self.raw[lead][i][1][:, :p]
                    vals.append((quant.astype(np.float64) * scale.astype(np.float64)[..., None]).reshape(nkv, n, 128))
                    u = (quant.astype(np.int16) + 128).astype(np.uint8).reshape(nkv, n, 128)
                    self.pool.planes[2 * i][page, :, row] = torch.from_numpy(u).cuda().transpose(0, 1)
                    self.pool.planes[2 * i + 1][page, :, row] = torch.from_numpy(scale.copy()).cuda().transpose(0, 1)
                    self.raw = getattr(self, "raw", {})
                    self.raw.setdefault(b, []).append((quant, scale))
                else:
                    h = x[i].astype(np.float16)
                    vals.append(h.astype(np.float64))
                    self.pool.planes[i][page, :, row] = torch.from_numpy(h).cuda().transpose(0, 1)
            self.kv.append(vals)
        for b in range(B):  # the whole pages of a prefix are looked up in the first session's row only
            if lead_of[b] != b:
                table[b, :shared[b] // ps] = -7
        self.dq = torch.from_numpy(self.q).cuda()
        self.table = self.pool.device_table()

    def workspace(self, kd):
        return torch.empty(kd.kd_attn_paged_workspace_bytes(len(self.lens), self.nh, self.nkv, self.hd), dtype=torch.uint8, device="cuda")

    def call(self, kd, out, ws, fault=None, stream=None, q=None):
        groups = dict(group_rows=self.rows, group_prefix=self.prefix) if len(self.rows) else {}
        a = (self.dq if q is None else q, *self.pool.planes, self.table, self.lens, self.nh, self.nkv)
        b = (self.pool.n_pages, self.ps, out, ws)
        if self.q8:
            kd.kd_attn_paged_decode_q8(*a, *b, fault=fault, stream=stream, **groups)
        else:
            kd.kd_attn_paged_decode(*a, self.hd, *b, fault=fault, stream=stream, **groups)

    def new_out(self):
        return torch.full((len(self.lens), self.nh * self.hd), float("nan"), dtype=torch.float16, device="cuda")

    def run(self, kd, fault_is=0):
        out, ws = self.new_out(), self.workspace(kd)
        ws.fill_(0xFF)
        fault = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.call(kd, out, ws, fault)
        torch.cuda.synchronize()
        assert kd.kd_attn_device_status(ws) == 0
        assert fault.item() == fault_is
        return out.cpu().numpy()

    def check(self, got, seen=None):
        group = self.nh // self.nkv
        for b in range(len(self.lens)):
            keys = slice(None) if seen is None else seen[b]
            for h in range(self.nkv):
                o, tol = reference(self.q[b, h * group:(h + 1) * group].astype(np.float64), self.kv[b][0][h][keys], self.kv[b][1][h][keys])
                g = got[b].reshape(self.nh, self.hd)[h * group:(h + 1) * group].astype(np.float64)
                err = np.abs(g - o)
                assert np.all(err <= tol), (b, h, int(self.lens[b]), float((err / np.maximum(tol, 1e-300)).max()))


SHAPES = [(False, 32, 8, 128), (False, 8, 8, 128), (False, 6, 3, 128), (False, 16, 2, 128), (False, 4, 4, 64), (False, 14, 7, 64),
          (False, 8, 2, 64), (False, 8, 1, 64), (True, 32, 8, 128), (True, 3, 3, 128), (True, 4, 2, 128), (True, 8, 1, 128)]


@pytest.mark.parametrize("q8,nh,nkv,hd", SHAPES)
@pytest.mark.parametrize("ps,lens", [(16, [37]), (16, [0, 1, 15, 16, 17, 31, 32, 33]), (48, [127, 128, 129, 0, 300, 47, 48, 49]),
                                     (64, [1500, 3, 700]), (256, [255, 256, 257, 1000]), (16, [0]), (4096, [4099, 1])])
def test_private_keys(kdlib, q8, nh, nkv, hd, ps, lens):
    c = Attn(q8, nh, nkv, hd, ps, lens, seed=len(lens) + ps + nh)
    c.check(c.run(kdlib))


@pytest.mark.parametrize("q8,nh,nkv,hd", [SHAPES[0], SHAPES[3], SHAPES[5], SHAPES[8]])
def test_many_sessions(kdlib, q8, nh, nkv, hd):
    rng = np.random.default_rng(nh)
    c = Attn(q8, nh, nkv, hd, 16, rng.integers(0, 90, 256).tolist(), seed=1)
    c.check(c.run(kdlib))
    c = Attn(q8, nh, nkv, hd, 32, [int(6000 ** u) for u in rng.random(19)] + [9001], seed=2)
    c.check(c.run(kdlib))


GROUPS = [
    (16, [300, 290, 280], [(3, 272)]),                        # a page boundary
    (16, [300, 290, 280], [(3, 277)]),                        # within a page
    (64, [200, 201, 330, 129, 128, 700], [(2, 200), (1, 100), (3, 128)]),
    (32, [50, 50], [(2, 50)]),                                # no key of their own but the rest of a page
    (32, [64, 64, 64], [(3, 64)]),                            # none at all
    (16, [0, 0, 5], [(2, 0), (1, 5)]),
    (48, [1100 + 3 * i for i in range(9)], [(9, 1000)]),
    (16, [2100 + i for i in range(33)] + [40], [(33, 2048), (1, 0)]),
    (128, [1300 + 7 * i for i in range(20)], [(16, 1290), (4, 1024)]),
]


@pytest.mark.parametrize("q8,nh,nkv,hd", SHAPES)
@pytest.mark.parametrize("ps,lens,groups", GROUPS)
def test_shared_prefixes(kdlib, q8, nh, nkv, hd, ps, lens, groups):
    c = Attn(q8, nh, nkv, hd, ps, lens, groups, seed=len(lens) + ps + nh)
    c.check(c.run(kdlib))


@pytest.mark.parametrize("q8,nh,nkv,hd", [SHAPES[0], SHAPES[3], SHAPES[7], SHAPES[8], SHAPES[11]])
def test_large_groups(kdlib, q8, nh, nkv, hd):
    rng = np.random.default_rng(5)
    for sizes, prefix in (([100, 3], 700), ([256], 515), ([64, 64], 1024)):
        groups = [(n, prefix + 16 * i) for i, n in enumerate(sizes)]
        lens = [p + int(rng.integers(0, 60)) for n, p in groups for _ in range(n)]
        c = Attn(q8, nh, nkv, hd, 16, lens, groups, seed=3)
        c.check(c.run(kdlib))


# Prefixes whose reading for every session would cost more than 24 MB (Q8_0: 16): taken once, on the tensor
# cores.  Tiles of 128 keys and 128 (Q8_0: 64) queries with nothing, one 16-key run or nearly all left over, pages
# smaller and larger than a tile, one tile of queries and many, groups of which only some qualify.
@pytest.mark.parametrize("q8,nh,nkv,hd,ps,groups,own", [
    (False, 32, 8, 128, 16, [(9, 1024)], 40), (False, 32, 8, 128, 48, [(9, 1010), (2, 48)], 100), (False, 32, 8, 128, 256, [(20, 769), (1, 300)], 30),
    (False, 6, 3, 128, 16, [(60, 528), (50, 656)], 9), (False, 16, 2, 128, 64, [(70, 460), (3, 128), (128, 512)], 20), (False, 8, 8, 128, 128, [(33, 256)], 0),
    (False, 8, 1, 64, 16, [(200, 656)], 5), (False, 4, 4, 64, 32, [(64, 530), (64, 416)], 33), (False, 14, 7, 64, 48, [(40, 400), (17, 1100)], 60),
    (True, 32, 8, 128, 16, [(12, 1104)], 40), (True, 3, 3, 128, 32, [(64, 600), (90, 417)], 17), (True, 8, 1, 128, 48, [(150, 700), (100, 1000)], 3),
    (True, 4, 2, 128, 256, [(80, 600), (120, 512), (2, 256)], 12), (True, 16, 4, 128, 16, [(160, 160)], 7),
])
def test_prefixes_read_once(kdlib, q8, nh, nkv, hd, ps, groups, own):
    rng = np.random.default_rng(nh + ps)
    lens = [p + int(rng.integers(0, own + 1)) for n, p in groups for _ in range(n)]
    c = Attn(q8, nh, nkv, hd, ps, lens, groups, seed=nh + ps)
    assert max((n - 1) * (p // ps * ps) * nkv * (272 if q8 else 4 * hd) for n, p in groups) >= 24 << 20
    c.check(c.run(kdlib))


@pytest.mark.parametrize("q8", [False, True])
def test_prefixes_read_once_far_scores(kdlib, q8):
    """Maxima that grow from tile to tile: the sums are rescaled; large and tiny values; small scores."""
    for kscale, vscale in ((30.0, 1.0), (1.0, 200.0), (0.01, 1e-3)):
        c = Attn(q8, 32, 8, 128, 32, [1300 + i for i in range(12)], [(12, 1290)], seed=4, kscale=kscale, vscale=vscale)
        c.check(c.run(kdlib))
    # keys in growing order: every tile has a new maximum for all queries
    c = Attn(False, 32, 8, 128, 32, [1300 + i for i in range(12)], [(12, 1280)], seed=4)
    lead = c.kv[0][0]
    for b in range(12):
        n = int(c.lens[b])
        grow = np.linspace(0.05, 40.0, 1280)[None, :, None]
        c.kv[b][0][:, :1280] = (lead[:, :1280] * grow if b == 0 else c.kv[0][0][:, :1280]).astype(np.float16)
        if b == 0:
            page, row = torch.from_numpy(c.pool.table[0, np.arange(1280) // 32].astype(np.int64)).cuda(), torch.from_numpy(np.arange(1280) % 32).cuda()
            c.pool.planes[0][page, :, row] = torch.from_numpy(c.kv[0][0][:, :1280].astype(np.float16)).cuda().transpose(0, 1)
    c.check(c.run(kdlib))


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("ps", [16, 64])
def test_prefixes_read_once_bad_pages(kdlib, q8, ps):
    """Pages of the shared part and of the sessions' own that do not exist, a whole tile of them among them."""
    c = Attn(q8, 32, 8, 128, ps, [1200 + 20 * i for i in range(14)], [(14, 1200 // ps * ps)], seed=6)
    bad = [2, *range(256 // ps, 384 // ps), 1088 // ps]
    for i, page in enumerate(bad):
        c.pool.table[0, page] = (-1, c.pool.n_pages, 2 ** 31 - 1, -2 ** 31)[i % 4]
    own = 1216 // ps
    c.pool.table[5, own] = -5
    c.table = c.pool.device_table()
    shared = 1200 // ps * ps
    seen = []
    for b in range(14):
        t = np.arange(int(c.lens[b]))
        hidden = np.isin(t // ps, bad) & (t < shared)
        if b == 5:
            hidden |= t // ps == own
        seen.append(t[~hidden])
    c.check(c.run(kdlib, fault_is=1), seen)


def test_prefixes_read_once_repeats_and_streams(kdlib):
    """Two streams at once with a workspace each, the same bits every time; smaller calls in between on the same workspace."""
    kd = kdlib
    cases = [Attn(False, 32, 8, 128, 16, [2000 + 9 * i for i in range(24)], [(14, 1800), (10, 1900)], seed=9),
             Attn(True, 16, 4, 128, 32, [1500 + i for i in range(40)], [(30, 1490), (10, 1000)], seed=10)]
    small = Attn(False, 32, 8, 128, 16, [50, 0, 300], seed=11)
    want, wanted = [c.run(kd) for c in cases], small.run(kd)
    for c, w in zip(cases, want):
        c.check(w)
    streams, outs, ws = [torch.cuda.Stream() for _ in cases], [c.new_out() for c in cases], [c.workspace(kd) for c in cases]
    out = small.new_out()
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s, o, w in zip(cases, streams, outs, ws):
            c.call(kd, o, w, stream=s)
        small.call(kd, out, ws[0], stream=streams[0])
    torch.cuda.synchronize()
    for w, o in zip(want + [wanted], outs + [out]):
        assert np.array_equal(w.view(np.int16), o.cpu().numpy().view(np.int16))
    assert kd.kd_attn_device_status(ws[0]) == 0 and kd.kd_attn_device_status(ws[1]) == 0


@pytest.mark.parametrize("q8", [False, True])
def test_far_scores_and_extreme_values(kdlib, q8):
    """Scores far apart (the running maximum moves), large and tiny values."""
    for kscale, vscale in ((30.0, 1.0), (1.0, 200.0), (0.01, 1e-3)):
        c = Attn(q8, 16, 4, 128, 32, [1000, 900, 64, 1], [(2, 512), (2, 0)], seed=4, kscale=kscale, vscale=vscale)
        c.check(c.run(kdlib))


@pytest.mark.parametrize("q8", [False, True])
def test_bad_pages_hide_their_keys(kdlib, q8):
    c = Attn(q8, 8, 2, 128, 16, [100, 64, 16, 300, 290], [(1, 0), (1, 0), (1, 0), (2, 256)], seed=6)
    c.pool.table[0, 2], c.pool.table[2, 0], c.pool.table[3, 4], c.pool.table[4, 17] = -1, c.pool.n_pages, 2 ** 31 - 1, -2 ** 31
    c.table = c.pool.device_table()
    seen = [np.r_[0:32, 48:100], np.r_[0:64], np.r_[0:0], np.r_[0:64, 80:300], np.r_[0:64, 80:272, 288:290]]
    c.check(c.run(kdlib, fault_is=1), seen)


def test_streams_graphs_and_repeats(kdlib):
    """The same call again, on another stream, and two captured graphs that share a workspace with eager calls."""
    kd = kdlib
    for q8 in (False, True):
        c = Attn(q8, 32, 8, 128, 16, [1300 + 31 * i for i in range(12)] + [0], [(12, 1290), (1, 0)], seed=8)
        want = c.run(kd)
        c.check(want)
        assert np.array_equal(want.view(np.int16), c.run(kd).view(np.int16))
        ws, side = c.workspace(kd), torch.cuda.Stream()
        out = c.new_out()
        side.wait_stream(torch.cuda.current_stream())
        c.call(kd, out, ws, stream=side)
        side.synchronize()
        assert np.array_equal(want.view(np.int16), out.cpu().numpy().view(np.int16))
        outs, graphs, q = [c.new_out(), c.new_out()], [], c.dq.clone()
        for o in outs:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                c.call(kd, o, ws, q=q)
            graphs.append(g)
        q.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert not np.array_equal(want.view(np.int16), outs[0].cpu().numpy().view(np.int16))
        q.copy_(c.dq)
        for _ in range(3):
            for g in graphs:
                g.replay()
        c.call(kd, out, ws)
        torch.cuda.synchronize()
        for o in outs + [out]:
            assert np.array_equal(want.view(np.int16), o.cpu().numpy().view(np.int16))


def test_two_calls_at_once(kdlib):
    """Calls on two streams, each with its own workspace."""
    kd = kdlib
    cases = [Attn(False, 32, 8, 128, 16, [2000, 1500, 900, 4000], [(4, 800)], seed=9),
             Attn(True, 16, 4, 128, 32, [3000, 3100, 2000], [(2, 2900), (1, 0)], seed=10)]
    want = [c.run(kd) for c in cases]
    streams, outs, ws = [torch.cuda.Stream() for _ in cases], [c.new_out() for c in cases], [c.workspace(kd) for c in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, o, w in zip(cases, streams, outs, ws):
            c.call(kd, o, w, stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert np.array_equal(w.view(np.int16), o.cpu().numpy().view(np.int16))


@pytest.mark.parametrize("q8", [False, True])
def test_one_page_many_times(kdlib, q8):
    """A page in every place of every table: each session sees its rows again and again, as it would see copies."""
    ps, B = 32, 12
    c = Attn(q8, 16, 4, 128, ps, [ps], seed=51)
    lens = [ps * 64 - 5 * b for b in range(B)]
    c.q = np.random.default_rng(5).standard_normal((B, 16, 128)).astype(np.float32)
    c.dq, c.lens = torch.from_numpy(c.q).cuda(), np.array(lens, np.int32)
    page = int(c.pool.table[0, 0])
    c.pool.table = np.full((B, 64), page, np.int32)
    c.table = c.pool.device_table()
    one = c.kv[0]
    c.kv = [[np.tile(x, (1, 64, 1))[:, :n] for x in one] for n in lens]
    c.check(c.run(kdlib))
    c.rows, c.prefix = np.array([B], np.int32), np.array([ps * 62], np.int32)
    c.check(c.run(kdlib))


@pytest.mark.parametrize("q8", [False, True])
def test_keys_appended_on_another_stream(kdlib, q8):
    """Rows appended on a stream that the attention's waits for, eager and in a graph of both."""
    kd = kdlib
    c = Attn(q8, 32, 8, 128, 16, [1300 + 31 * i for i in range(16)], [(16, 1290)], seed=61)
    new, plan = [normal(s, (16, 8, 128)) for s in (3, 4)], kd_plan(kd, 128)
    want, out, ws, side = c.run(kd), c.new_out(), c.workspace(kd), torch.cuda.Stream()

    def step(k, v):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        args = (plan, k, v, *c.pool.planes, c.table, c.lens - 1, [1] * 16, 8)
        if q8:
            kd.kd_paged_append_q8(*args, c.pool.n_pages, 16, stream=side)
        else:
            kd.kd_paged_append(*args, 128, c.pool.n_pages, 16, stream=side)
        main.wait_stream(side)
        c.call(kd, out, ws, stream=main)
    step(*new)
    torch.cuda.synchronize()
    with_new = out.cpu().numpy()
    assert np.array_equal(with_new, c.run(kd)) and not np.array_equal(with_new, want)
    k, v = (torch.zeros_like(x) for x in new)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(k, v)
    for _ in range(3):
        for x, y in ((k, new[0]), (v, new[1])):
            x.zero_()
        g.replay()
        k.copy_(new[0])
        v.copy_(new[1])
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(with_new, out.cpu().numpy())


@pytest.mark.parametrize("groups", [[], [(14, 1280), (2, 0)]])
@pytest.mark.parametrize("q8", [False, True])
def test_offsets_past_32_bits(kdlib, q8, groups):
    """Pages of planes of more than 4 GB, half of them at their ends: the bits that a small pool gives."""
    c = Attn(q8, 32, 8, 128, 64, [1290 + 11 * i for i in range(14)] + [300, 5], groups, seed=33)
    small, n, table = c.pool.planes, c.pool.n_pages, c.pool.table
    big_n = 70001 if q8 else 35001  # 2^32 bytes are 65536 and 32768 pages
    page = np.arange(n)
    page = np.where(page % 2, big_n - 1 - page, page)
    at = torch.from_numpy(page).cuda()
    big = [torch.empty((big_n, *p.shape[1:]), dtype=p.dtype, device="cuda") for p in small]
    assert max(p.nbytes for p in big) > 2 ** 32
    for b, p in zip(big, small):
        b[at] = p
    new = [normal(s, (16, 8, 128)) for s in (1, 2)]
    plan, got = kd_plan(kdlib, 128), []
    for planes, pages in ((small, n), (big, big_n)):
        if pages == big_n:
            c.pool.planes, c.pool.n_pages = big, big_n
            c.pool.table = np.where((table >= 0) & (table < n), page[np.clip(table, 0, n - 1)], table).astype(np.int32)
            c.table = c.pool.device_table()
        if q8:
            kdlib.kd_paged_append_q8(plan, *new, *planes, c.table, c.lens - 1, [1] * 16, 8, pages, 64)
        else:
            kdlib.kd_paged_append(plan, *new, *planes, c.table, c.lens - 1, [1] * 16, 8, 128, pages, 64)
        got.append(c.run(kdlib))
    assert all(torch.equal(b[at].view(torch.uint8), p.view(torch.uint8)) for b, p in zip(big, small))
    assert np.array_equal(got[0], got[1])


def test_rows_far_apart(kdlib):
    """Rows 2^31 elements apart: rotated from there, to there and in place, and appended, as rows that lie together."""
    far = torch.empty(2 * 2 ** 31 + 512, dtype=torch.float16, device="cuda").as_strided((3, 4, 128), (2 ** 31, 128, 1))
    x, pos, plan = normal(3, (3, 4, 128), "fp16"), torch.arange(7, 10, dtype=torch.int32, device="cuda"), kd_plan(kdlib, 128)
    want, got = torch.empty_like(x), torch.empty_like(x)
    kdlib.kd_rope(plan, x, pos, want)
    far.copy_(x)
    kdlib.kd_rope(plan, far, pos, got)
    assert torch.equal(got, want)
    kdlib.kd_rope(plan, far, pos, far)
    assert torch.equal(far, want)
    pools = [torch.zeros(4, 4, 16, 128, dtype=torch.float16, device="cuda") for _ in range(4)]
    table = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    q_out = [torch.empty(3, 4, 128, device="cuda") for _ in range(2)]
    for rows, planes, to in ((far, pools[:2], q_out[0]), (want, pools[2:], q_out[1])):
        kdlib.kd_paged_append(plan, rows, rows, *planes, table, [14], [3], 4, 128, 4, 16, q=rows, q_out=to, n_heads=4)
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3]) and torch.equal(*q_out)
    assert pools[1][2, :, 14:].abs().sum() > 0 and pools[1][0, :, :1].abs().sum() > 0


@pytest.mark.parametrize("groups", [[], [(14, 1200), (2, 0)]])
@pytest.mark.parametrize("q8", [False, True])
def test_not_a_number_stays_with_its_query(kdlib, q8, groups):
    """A NaN in one query's dims, and (fp16) in one key that a session sees: NaN there and nowhere else."""
    c = Attn(q8, 32, 8, 128, 16, [1290 + i for i in range(14)] + [300, 5], groups, seed=21)
    q = c.dq.clone()
    q[3, 17, 5] = float("nan")
    q[15, 2, 100] = float("nan")
    out, ws = c.new_out(), c.workspace(kdlib)
    c.call(kdlib, out, ws, q=q)
    bad = torch.isnan(out).view(16, 32, 128)
    want = torch.zeros(16, 32, dtype=torch.bool, device="cuda")
    want[3, 17] = want[15, 2] = True
    assert torch.equal(bad.all(-1), want) and torch.equal(bad.any(-1), want)
    if not q8:
        page = int(c.pool.table[14, 200 // 16])
        c.pool.planes[0][page, 6, 200 % 16, 3] = float("nan")
        c.call(kdlib, out, ws)
        want[:] = False
        want[14, 24:28] = True
        assert torch.equal(torch.isnan(out).view(16, 32, 128).all(-1), want)


FIRST = """
import numpy as np, torch
import session_decode_step_gb300 as kd
B, nh, nkv, hd, ps, n = 16, 32, 8, 128, 16, 1024
pages = n // ps + 2 * B
planes = {planes}
table = torch.zeros(B, n // ps + 2, dtype=torch.int32)
table[:, :n // ps] = torch.arange(n // ps)
table[:, n // ps:] = n // ps + torch.arange(2 * B).view(B, 2)
table = table.cuda()
q, k = torch.randn(B, nh, hd, device="cuda"), torch.randn(B, nkv, hd, device="cuda")
q_out, out = torch.empty_like(q), torch.zeros(B, nh * hd, dtype=torch.float16, device="cuda")
pos = torch.arange(B, dtype=torch.int32, device="cuda")
ws = torch.empty(kd.kd_attn_paged_workspace_bytes(B, nh, nkv, hd), dtype=torch.uint8, device="cuda")
plan = kd.kd_rope_plan(hd, 1e4)
def step():
    kd.kd_rope(plan, q, pos, q_out)
    {append}
    {attend}
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):  # nothing of these has run in this process
    step()
g.replay()
torch.cuda.synchronize()
first = out.clone()
assert kd.kd_attn_device_status(ws) == 0 and first.abs().sum() > 0
out.zero_()
step()
torch.cuda.synchronize()
assert torch.equal(first, out)
print("same")
"""


@pytest.mark.parametrize("q8", [False, True])
def test_first_calls_of_a_process_in_a_capture(kdlib, q8):
    if q8:
        parts = dict(planes='[torch.randint(1, 255, (pages, nkv, ps, 128), dtype=torch.uint8, device="cuda"), torch.rand(pages, nkv, ps, 4, device="cuda").half()] * 2',
                     append="kd.kd_paged_append_q8(plan, k, k, *planes, table, [n] * B, [1] * B, nkv, pages, ps, q=q, q_out=q_out, n_heads=nh)",
                     attend="kd.kd_attn_paged_decode_q8(q_out, *planes, table, [n + 1] * B, nh, nkv, pages, ps, out, ws, group_rows=[B], group_prefix=[n])")
    else:
        parts = dict(planes='[torch.randn(pages, nkv, ps, hd, device="cuda").half() for _ in range(2)]',
                     append="kd.kd_paged_append(plan, k, k, *planes, table, [n] * B, [1] * B, nkv, hd, pages, ps, q=q, q_out=q_out, n_heads=nh)",
                     attend="kd.kd_attn_paged_decode(q_out, *planes, table, [n + 1] * B, nh, nkv, hd, pages, ps, out, ws, group_rows=[B], group_prefix=[n])")
    r = subprocess.run([sys.executable, "-c", FIRST.format(**parts)], capture_output=True, text=True, timeout=300, cwd=Path(__file__).resolve().parents[1])
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


# ------------------------------------------------------------ used together ---
@pytest.mark.parametrize("q8", [False, True])
def test_a_prompt_shared_by_sessions_and_their_steps(kdlib, q8):
    """A prompt appended once, forked into sessions that share its whole pages (the page it ends in copied by
    kd_kv_reorder), then decode steps of rotate, append and attend, against the formulas on the rows read back."""
    kd, nh, nkv, hd, ps, B, n = kdlib, 16, 4, 128, 16, 5, 213
    plan = make_plan(kd, hd, hd, 10000.0, HALF, scaling="bands", factor=8.0)
    f = frequencies(hd, 10000.0, scaling="bands", factor=8.0)
    steps, whole = 6, n // ps
    pool = Pages(q8, nkv, hd, ps, [n + steps] + [(n + steps) - whole * ps] * (B - 1), 12)
    own = pool.table.copy()
    pool.table = np.full((B, own.shape[1]), 2 ** 30, np.int32)
    pool.table[0] = own[0]
    for b in range(1, B):
        pool.table[b, :whole] = own[0, :whole]
        pool.table[b, whole:whole + 2] = own[b, :2]
    table = pool.device_table()
    k, v = normal(20, (n, nkv, hd), "fp16"), normal(21, (n, nkv, hd), "fp16")
    append = (lambda p, k, v, s, c, **e: kd.kd_paged_append_q8(p, k, v, *pool.planes, table, s, c, nkv, pool.n_pages, ps, **e)) if q8 else \
             (lambda p, k, v, s, c, **e: kd.kd_paged_append(p, k, v, *pool.planes, table, s, c, nkv, hd, pool.n_pages, ps, **e))
    append(plan, k, v, [0] + [0] * (B - 1), [n] + [0] * (B - 1))
    last = pool.table[:, whole]
    kd.kd_kv_reorder(pool.planes, last[1:].copy(), [last[0]] * (B - 1), [n - whole * ps] * (B - 1), 1, pool.n_pages, nkv, ps)
    ws = torch.empty(kd.kd_attn_paged_workspace_bytes(B, nh, nkv, hd), dtype=torch.uint8, device="cuda")
    fault = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step in range(steps):
        q, kn, vn = (normal(100 * step + i, (B, h, hd)) for i, h in enumerate((nh, nkv, nkv)))
        q_rot = torch.empty_like(q)
        out = torch.empty(B, nh * hd, dtype=torch.float16, device="cuda")
        append(plan, kn, vn, [n + step] * B, [1] * B, q=q, q_out=q_rot, n_heads=nh, fault=fault)
        a = (q_rot, *pool.planes, table, [n + step + 1] * B, nh, nkv)
        e = dict(group_rows=[B], group_prefix=[n], fault=fault)
        if q8:
            kd.kd_attn_paged_decode_q8(*a, pool.n_pages, ps, out, ws, **e)
        else:
            kd.kd_attn_paged_decode(*a, hd, pool.n_pages, ps, out, ws, **e)
        check_rotated(q_rot, q, np.full(B, n + step), f, HALF, 1.0, "fp32")
        got = out.cpu().numpy().reshape(B, nh, hd).astype(np.float64)
        for b in range(B):
            K, V = ((values_of(*pool.rows(i, b, 0, n + step + 1)) if q8 else pool.rows(i, b, 0, n + step + 1)[0].double().cpu().numpy())
                    for i in range(2))
            if b and not step:  # the fork: the prompt's rows
                for i in range(2):
                    for x, y in zip(pool.rows(i, b, 0, n), pool.rows(i, 0, 0, n)):
                        assert torch.equal(bits(x), bits(y))
            for h in range(nkv):
                g = nh // nkv
                o, tol = reference(q_rot[b, h * g:(h + 1) * g].double().cpu().numpy(), K[:, h], V[:, h])
                assert np.all(np.abs(got[b, h * g:(h + 1) * g] - o) <= tol)
    assert fault.item() == 0 and kd.kd_attn_device_status(ws) == 0


# ------------------------------------------------- large scales of Q8_0 rows ---
def plant(c, part, t, h, scale, codes=None, block=0):
    """Another scale (and codes) for a block of row t of K (part 0) or V (1), a row that all sessions have from the first one's page."""
    page, row, dims = int(c.pool.table[0, t // c.ps]), t % c.ps, slice(32 * block, 32 * block + 32)
    quants, scales = c.pool.planes[2 * part:2 * part + 2]
    scales[page, h, row, block] = scale
    if codes is not None:
        quants[page, h, row, dims] = torch.as_tensor(codes + 128, dtype=torch.uint8, device="cuda")
    values = (quants[page, h, row, dims].cpu().numpy().astype(np.float64) - 128) * float(np.float16(scale))
    for K_V in c.kv:
        K_V[part][h, t, dims] = values


def check_rounded(c, got):
    """As Attn.check, where outputs may leave fp16's range: from 65520 on, the middle between its largest value and the
    next one, rounding gives an infinity."""
    group = c.nh // c.nkv
    for b in range(len(c.lens)):
        for h in range(c.nkv):
            o, tol = reference(c.q[b, h * group:(h + 1) * group].astype(np.float64), c.kv[b][0][h], c.kv[b][1][h])
            g = got[b].reshape(c.nh, c.hd)[h * group:(h + 1) * group].astype(np.float64)
            inf = np.isinf(g)
            assert np.all(inf | (np.abs(g - o) <= tol)) and np.all(~inf | ((np.abs(o) + tol >= 65520) & (np.sign(g) == np.sign(o)))), (b, h)


@pytest.mark.parametrize("B", [2, 12])  # a prefix that each session reads, and one that is read once
@pytest.mark.parametrize("scale", [511.5, 512.0, 516.0, 600.0, 1100.0, 9000.0, 65504.0])
def test_large_scales_in_a_shared_prefix(kdlib, B, scale):
    """Blocks whose values leave fp16's range, in rows of whole tiles and of the last one, in K, in V and in both."""
    for parts in ((0,), (1,), (0, 1)):
        c = Attn(True, 32, 8, 128, 16, [1310 + i for i in range(B)], [(B, 1300)], seed=71, kscale=0.3)
        rng = np.random.default_rng(B)
        if 0 in parts:
            # Query dims of block 0 that are whole pairs of fp16 (a few 2^-24 and more) and give scores of ordinary size.
            unit = 2.0 ** (-24 + math.floor(math.log2(65504 / scale)))
            c.q[..., :32] = rng.integers(-8, 9, (B, 32, 32)) * unit
            c.dq = torch.from_numpy(c.q).cuda()
        for part in parts:
            for h in range(8):
                for t in (5 + h, 67, 127, 128 + 33 * h % 128, 1279 - h, 1290):
                    plant(c, part, t, h, scale, rng.integers(-127, 128, 32))
                    plant(c, part, t, h, 2.0 ** -7, block=2)  # a small block beside it
        check_rounded(c, c.run(kdlib))


@pytest.mark.parametrize("B", [2, 12])
def test_large_scales_where_the_maximum_has_grown(kdlib, B):
    """A tile whose scores are e^3.4 above the first one's, in which values are far out of fp16's range."""
    c = Attn(True, 8, 8, 128, 16, [1310 + i for i in range(12)], [(12, 1300)], seed=72, kscale=0.05)
    if B == 2:  # the same sessions, every one with its own reading
        c.rows, c.prefix = np.array([2] * 6, np.int32), np.array([1300] * 6, np.int32)
        c.pool.table[:, :81] = c.pool.table[0, :81]
        c.table = c.pool.device_table()
    c.q[..., 96:] = 1.0
    c.dq = torch.from_numpy(c.q).cuda()
    rng = np.random.default_rng(5)
    for h in range(8):
        for t in range(1296):
            plant(c, 0, t, h, 1.2, np.full(32, 1 if 128 <= t < 256 else 0), block=3)
        for t in (130 + h, 200, 255):
            plant(c, 1, t, h, 40000.0, rng.integers(-127, 128, 32), block=1)
    check_rounded(c, c.run(kdlib))


# ------------------------------------------------ the bounds that kd.h states ---
def scale_keys(c, f):
    """K's values times f, a power of two, rounded as the cache holds them."""
    if c.q8:
        s = c.pool.planes[1]
        s.copy_((s.float() * f).half())
        for b, kv in enumerate(c.kv):
            quant, scale = c.raw[b][0]
            kv[0] = (quant.astype(np.float64) * (scale.astype(np.float32) * f).astype(np.float16).astype(np.float64)[..., None]).reshape(kv[0].shape)
    else:
        p = c.pool.planes[0]
        p.copy_((p.float() * f).half())
        for kv in c.kv:
            kv[0] = (kv[0] * f).astype(np.float16).astype(np.float64)


def check_bounds(c, got):
    """Attn.check with a query's least step: each of its values may be off by 2^-25, so a score by 2^-25 max_t sum_i |k_ti| /
    sqrt(hd), and weights by twice that."""
    group = c.nh // c.nkv
    for b in range(len(c.lens)):
        for h in range(c.nkv):
            K, V = c.kv[b][0][h], c.kv[b][1][h]
            q = c.q[b, h * group:(h + 1) * group].astype(np.float64)
            o, tol = reference(q, K, V)
            step = 2 * 2.0 ** -25 * np.abs(K).sum(1).max() / np.sqrt(c.hd)
            p = np.exp(q @ K.T / np.sqrt(c.hd) - (q @ K.T).max(1, keepdims=True) / np.sqrt(c.hd))
            tol = tol + step * ((p / p.sum(1, keepdims=True)) @ np.abs(V))
            g = got[b].reshape(c.nh, c.hd)[h * group:(h + 1) * group].astype(np.float64)
            assert np.all(np.abs(g - o) <= tol), (b, h, float((np.abs(g - o) / tol).max()))


@pytest.mark.parametrize("B", [2, 12])  # a prefix that each session reads, and one that is read once
@pytest.mark.parametrize("q8,nh,nkv,hd", [(False, 32, 8, 128), (False, 64, 8, 128), (False, 32, 8, 64), (True, 32, 8, 128), (True, 64, 8, 128)])
def test_queries_within_their_bounds(kdlib, q8, nh, nkv, hd, B):
    """Large queries of small keys, small queries of large keys: up to 65504 and down to a value's least step."""
    n = 2600 if hd == 64 else 1300  # in the larger group past the border of being read once
    for qscale, kscale in ((2.0 ** 13, 2.0 ** -12), (2.0 ** -7, 2.0 ** 7), (2.0 ** -12, 2.0 ** 12)):
        c = Attn(q8, nh, nkv, hd, 16, [n + 9 + i for i in range(B)], [(B, n)], seed=81)
        scale_keys(c, kscale)
        c.q = np.clip(c.q * np.float32(qscale), -65504, 65504).astype(np.float32)
        c.q[B - 1, 1] = 0.0
        c.q[0, 0, :2] = 65504.0 * min(1.0, qscale), -65504.0 * min(1.0, qscale)
        c.dq = torch.from_numpy(c.q).cuda()
        check_bounds(c, c.run(kdlib))


@pytest.mark.parametrize("B", [2, 12])
@pytest.mark.parametrize("q8", [False, True])
def test_scores_near_their_bound(kdlib, q8, B):
    """Scores of a few 10^6, up to 10^7 in size: the key with the largest one alone, whichever comes first."""
    c = Attn(q8, 32, 8, 128, 16, [1310 + i for i in range(B)], [(B, 1300)], seed=82)
    scale_keys(c, 2.0 ** 6)
    c.q *= np.float32(2.0 ** 15 / np.abs(c.q).max())
    c.dq = torch.from_numpy(c.q).cuda()
    got = c.run(kdlib).reshape(B, 32, 128).astype(np.float64)
    sure = 0
    for b in range(B):
        for h in range(32):
            q, K, V = c.q[b, h].astype(np.float64), c.kv[b][0][h // 4], c.kv[b][1][h // 4]
            s = K @ q / np.sqrt(128)
            assert 1e5 < np.abs(s).max() < 1e7
            # a score is off by (2^-21 + 9 2^-23) sum_i |q_i k_i| / sqrt(hd): the second one is e^-40 of the first at least then
            off = (2.0 ** -21 + 9 * 2.0 ** -23) * (np.abs(K) @ np.abs(q)).max() / np.sqrt(128)
            first = s.argmax()
            if np.sort(s)[-2] < s[first] - 2 * off - 40:
                sure += 1
                assert np.all(np.abs(got[b, h] - V[first]) <= 2.0 ** -11 * np.abs(V[first]) + 2.0 ** -19 * np.abs(V[first]) + 2.0 ** -25), (b, h)
    assert sure >= B * 32 * 9 // 10 and np.isfinite(got).all()


# ------------------------------------------------- steps behind a shared prefix ---
@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("q8", [False, True])
def test_steps_behind_a_prefix_read_once(kdlib, q8, graph):
    """Steps in one stream without a pause: each appends a key and a value, writes the queries that the attention behind it
    reads at once, and overwrites what the step before read; every step against the formula."""
    kd, B, nh, nkv, hd, ps, n, steps = kdlib, 12, 32, 8, 128, 16, 1300, 6
    c = Attn(q8, nh, nkv, hd, ps, [n + 5 * i + steps for i in range(B)], [(B, n)], seed=91)
    base, ws = c.lens - steps, c.workspace(kd)
    for b in range(B):  # the last rows are the steps'
        base[b] = max(base[b], n)
    c.lens = base + steps
    fresh = [[normal(1000 * part + t, (B, h, hd)) for t in range(steps)] for part, h in enumerate((nh, nkv, nkv))]
    given = [[torch.zeros_like(x) for x in part] for part in fresh] if graph else fresh
    q_out, outs = torch.empty(B, nh, hd, device="cuda"), [c.new_out() for _ in range(steps)]
    full = c.lens.copy()

    def run():
        for t in range(steps):
            args = (None, given[1][t], given[2][t], *c.pool.planes, c.table, base + t, [1] * B, nkv)
            extra = dict(q=given[0][t], q_out=q_out, n_heads=nh)
            if q8:
                kd.kd_paged_append_q8(*args, c.pool.n_pages, ps, **extra)
            else:
                kd.kd_paged_append(*args, hd, c.pool.n_pages, ps, **extra)
            c.lens = (base + t + 1).astype(np.int32)
            c.call(kd, outs[t], ws, q=q_out)
    torch.cuda.synchronize()
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        g.replay()  # of zeros
        for part, new in zip(given, fresh):
            for x, y in zip(part, new):
                x.copy_(y)
        g.replay()
    else:
        run()
    torch.cuda.synchronize()
    assert kd.kd_attn_device_status(ws) == 0
    c.lens = full
    for b in range(B):  # the new rows as they lie in the pages (behind the prefix, in the session's own)
        for part in range(2):
            rows = c.pool.rows(part, b, int(base[b]), int(full[b]))
            values = values_of(*rows) if q8 else rows[0].double().cpu().numpy()
            c.kv[b][part][:, int(base[b]):int(full[b])] = values.transpose(1, 0, 2)
            x = torch.stack([fresh[1 + part][t][b] for t in range(steps)]).double().cpu().numpy()
            assert np.all(np.abs(values - x) <= (np.abs(x).max() / 250 if q8 else 2.0 ** -11 * np.abs(x) + 2.0 ** -25))
    kv = c.kv
    for t in range(steps):
        c.lens = (base + t + 1).astype(np.int32)
        c.q = fresh[0][t].cpu().numpy()
        c.kv = [[x[:, :int(c.lens[b])] for x in kv[b]] for b in range(B)]
        c.check(outs[t].cpu().numpy())


# --------------------------------------------------------- a wait that runs out ---
@pytest.mark.parametrize("part", [0, 1])
@pytest.mark.parametrize("q8", [False, True])
def test_a_wait_that_runs_out_is_reported(kdlib, q8, part):
    """One barrier of the prefix kernel waits for bytes that nothing delivers: reported, and the next calls on the same
    workspace, a smaller one and the same again, are right before the host has cleared anything."""
    kd = kdlib
    c = Attn(q8, 32, 8, 128, 16, [1310 + i for i in range(12)], [(12, 1300)], seed=95)
    small = Attn(q8, 32, 8, 128, 16, [50, 0, 300], seed=11)
    want, wanted = c.run(kd), small.run(kd)
    c.check(want)
    out, small_out, ws = c.new_out(), small.new_out(), c.workspace(kd)
    kd.kd_debug_attn_paged_inject_wait_timeout(part)
    small.call(kd, small_out, ws)  # has no prefix to wait for
    assert kd.kd_attn_device_status(ws) == 0
    c.call(kd, out, ws)
    with pytest.raises(kd.KdError) as e:
        kd.kd_attn_device_status(ws)
    assert e.value.name == "KD_ERR_DEVICE"
    kd.kd_debug_attn_paged_inject_wait_timeout(part)
    c.call(kd, out, ws)  # again, and nothing asked in between
    small.call(kd, small_out, ws)
    c.call(kd, out, ws)
    assert kd.kd_attn_device_status(ws) == 0
    assert np.array_equal(out.cpu().numpy().view(np.int16), want.view(np.int16))
    assert np.array_equal(small_out.cpu().numpy().view(np.int16), wanted.view(np.int16))


def test_the_wait_hook_has_two_parts(kdlib):
    for part in (-1, 2):
        with pytest.raises(kdlib.KdError):
            kdlib.kd_debug_attn_paged_inject_wait_timeout(part)


# ------------------------------------------------ which prefixes are read once ---
def test_the_cases_of_prefixes_read_once_are(kdlib):
    """The largest groups of the cases above that are meant for the tensor cores go there."""
    mark = next(m for m in test_prefixes_read_once.pytestmark if m.name == "parametrize")
    for q8, nh, nkv, hd, ps, groups, own in mark.args[1]:
        assert any(kdlib.kd_attn_paged_reads_once(n, p, nh, nkv, hd, ps, q8) for n, p in groups), (q8, nh, nkv, hd, groups)
    for rows, prefix, q8 in ((12, 1290, False), (12, 1300, False), (12, 1300, True), (14, 1280, False), (14, 1280, True)):
        assert kdlib.kd_attn_paged_reads_once(rows, prefix, 32, 8, 128, 16, q8)
        assert not kdlib.kd_attn_paged_reads_once(2, prefix, 32, 8, 128, 16, q8)


@pytest.mark.parametrize("q8,nh,nkv,hd,rows,mb", [(False, 32, 8, 128, 2, 24), (False, 8, 8, 128, 5, 24), (False, 16, 8, 64, 3, 24), (False, 64, 8, 64, 16, 24),
                                                  (True, 32, 8, 128, 4, 24), (True, 8, 8, 128, 11, 24), (True, 24, 24, 128, 12, 24), (True, 64, 8, 128, 2, 40),
                                                  (True, 64, 8, 128, 3, 16)])
def test_both_sides_of_the_reading_rule(kdlib, q8, nh, nkv, hd, rows, mb):
    """A prefix one page short of being read once, and the same with it: both as the formula has it."""
    row = nkv * (272 if q8 else 4 * hd)
    pages = -(-(mb << 20) // ((rows - 1) * row * 16))
    for p, once in ((16 * pages - 16, False), (16 * pages, True)):
        assert kdlib.kd_attn_paged_reads_once(rows, p, nh, nkv, hd, 16, q8) == once
        c = Attn(q8, nh, nkv, hd, 16, [p + 7 + 3 * i for i in range(rows)], [(rows, p + 5)], seed=rows + mb)
        c.check(c.run(kdlib))
