"""Sliding-window attention with sinks on the GPU against a plain fp64 softmax.

Op level: fp16 rows (head dims 64 and 128) and Q8_0 rows, every GQA group, ragged
positions around the 64-key items and the window's edges, windows and sinks that
hide nothing, one key, or all but a few; every cache row a session must not use is
NaN (fp16) or has NaN scales (Q8_0).  Model level: the tiny models' steps with a
window against a step written from the oracle's parts.

Tolerance of an output o = sum_t p_t v_t (derived, per element).  Scores: q as an
fp16 pair loses 2^-21 |q|, the products' fp32 sums at most hd/16 + 1 truncated adds
of 2^-23, so a score moves by at most S (2^-21 + 9 2^-23), S = max_t sum_i |q_i
k_ti| / sqrt(hd).  Weights: twice that (numerator and denominator) plus expf's and
the roundings of p, 2^-21, and the sums over items, (items + 10) 2^-23.  So o moves
by at most eps sum_t p_t |v_t|; then it is rounded to fp16 once: 2^-11 |o| (2^-25
below the normal range)."""
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest

import oracle
import synth

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

NAN16 = np.float16(np.nan)


def visible(pos, window, sinks):
    t = np.arange(pos + 1)
    return t[(t < sinks) | (t > pos - window)]


def reference(q, K, V):
    """q [group][hd], K, V [keys][hd] in fp64 -> outputs and their tolerances."""
    hd = q.shape[1]
    s = q @ K.T / np.sqrt(hd)
    S = (np.abs(q) @ np.abs(K).T).max(1, keepdims=True) / np.sqrt(hd)
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    o = p @ V
    eps = 2 * S * (2.0 ** -21 + 9 * 2.0 ** -23) + 2.0 ** -21 + (len(K) / 64 + 10) * 2.0 ** -23
    return o, 2.0 ** -11 * np.abs(o) + 2.0 ** -25 + eps * (p @ np.abs(V))


class Case:
    """Caches (device) with NaN in every row a session must not use, and the visible rows' values (host)."""

    def __init__(self, q8, seed, nh, nkv, hd, cap, pos, window, sinks, n_slots=None, kscale=1.0, last_slot=False):
        rng = np.random.default_rng(seed)
        self.q8, self.nh, self.nkv, self.hd, self.cap, self.window, self.sinks = q8, nh, nkv, hd, cap, window, sinks
        self.pos = np.array(pos, np.int32)
        B = len(pos)
        self.n_slots = n_slots or B + 2
        self.slots = rng.permutation(self.n_slots)[:B].astype(np.int32)
        if last_slot and self.n_slots - 1 not in self.slots:
            self.slots[0] = self.n_slots - 1
        self.q = (rng.standard_normal((B, nh, hd)) * kscale).astype(np.float32)
        self.kn = rng.standard_normal((B, nkv, hd)).astype(np.float32)
        self.vn = rng.standard_normal((B, nkv, hd)).astype(np.float32)
        shape = (self.n_slots, nkv, cap)
        if not q8:
            self.dev = [torch.full((*shape, hd), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2)]
        else:
            self.dev = []
            for _ in range(2):
                self.dev.append(torch.full((*shape, 128), 0x5A, dtype=torch.uint8, device="cuda"))
                self.dev.append(torch.full((*shape, 4), float("nan"), dtype=torch.float16, device="cuda"))
        self.rows = {}  # (b, which) -> [nkv][visible][hd] fp64, the new row last
        for b in range(B):
            t = visible(int(pos[b]), window, sinks)[:-1]
            dt = torch.from_numpy(t).cuda()
            slot = int(self.slots[b])
            for i, new in enumerate((self.kn, self.vn)):
                x = rng.standard_normal((nkv, len(t), hd)).astype(np.float32)
                both = np.concatenate([x, new[b][:, None]], 1)
                if not q8:
                    val = both.astype(np.float16)
                    self.dev[i][slot][:, dt] = torch.from_numpy(val[:, :-1]).cuda()
                    self.rows[b, i] = val.astype(np.float64)
                else:
                    blk = oracle.q8_0_quantize_f32(both).reshape(nkv, len(t) + 1, 4, 34)
                    quant = np.ascontiguousarray(blk[..., 2:]).view(np.int8)
                    scale = np.ascontiguousarray(blk[..., :2]).view(np.float16)
                    u = (quant.astype(np.int16) + 128).astype(np.uint8).reshape(nkv, -1, 128)[:, :-1]
                    self.dev[2 * i][slot][:, dt] = torch.from_numpy(np.ascontiguousarray(u)).cuda()
                    self.dev[2 * i + 1][slot][:, dt] = torch.from_numpy(scale.reshape(nkv, -1, 4)[:, :-1].copy()).cuda()
                    self.rows[b, i] = (quant.astype(np.float64) * scale.astype(np.float64)).reshape(nkv, -1, 128)
        self.dq, self.dk, self.dv = (torch.from_numpy(x).cuda() for x in (self.q, self.kn, self.vn))

    def workspace(self, kd, B):
        n = kd.kd_attn_window_workspace_bytes(B, self.nh, self.hd, self.cap, self.window, self.sinks)
        return torch.empty(n, dtype=torch.uint8, device="cuda")

    def call(self, kd, out, ws, rows=slice(None), stream=None):
        a = (self.dq[rows], self.dk[rows], self.dv[rows], *self.dev, self.slots[rows], self.pos[rows], self.nh, self.nkv)
        b = (self.n_slots, self.cap, self.window, self.sinks, out, ws, stream)
        if self.q8:
            kd.kd_attn_window_append_decode_q8(*a, *b)
        else:
            kd.kd_attn_window_append_decode(*a, self.hd, *b)

    def run(self, kd, rows=slice(None)):
        B = len(self.pos[rows])
        out = torch.full((B, self.nh * self.hd), -1, dtype=torch.int16, device="cuda")
        ws = self.workspace(kd, B)
        self.call(kd, out, ws, rows)
        torch.cuda.synchronize()
        assert kd.kd_attn_device_status(ws) == 0
        return out.cpu().numpy().view(np.float16)

    def check(self, got):
        group = self.nh // self.nkv
        for b in range(len(self.pos)):
            for h in range(self.nkv):
                o, tol = reference(self.q[b, h * group:(h + 1) * group].astype(np.float64), self.rows[b, 0][h],
                                   self.rows[b, 1][h])
                g = got[b].reshape(self.nh, self.hd)[h * group:(h + 1) * group].astype(np.float64)
                err = np.abs(g - o)
                assert np.all(err <= tol), (b, h, int(self.pos[b]), float((err / tol).max()))


SHAPES = [(32, 8, 128), (8, 8, 128), (6, 3, 128), (16, 2, 128), (4, 4, 64), (14, 7, 64), (8, 2, 64), (8, 1, 64)]
RANGES = [(1, 0), (1, 1), (7, 4), (64, 0), (65, 3), (100, 64), (130, 200), (500, 1), (2 ** 31 - 1, 2 ** 31 - 1)]


# cap: up to 2048 visible keys are shared out over 16 or 24 chains, more over 32 or 48
@pytest.mark.parametrize("nh,nkv,hd", SHAPES)
@pytest.mark.parametrize("window,sinks,cap", [(w, s, 601) for w, s in RANGES] + [
    (2 ** 31 - 1, 5, 2101), (2500, 0, 2600), (2040, 3, 2301), (2100, 70, 4001), (300, 2000, 2301), (2080, 300, 2500)])
def test_window_fp16(kdlib, nh, nkv, hd, window, sinks, cap):
    c = Case(False, window % 1000 + sinks % 1000 + nh, nh, nkv, hd, cap,
             [0, 1, 6, 63, 64, 127, 200, 263, cap - 1, cap * 5 // 9], window, sinks)
    got = c.run(kdlib)
    c.check(got)
    for i, new in ((0, c.kn), (1, c.vn)):  # the appended rows
        d = c.dev[i].cpu().numpy()
        for b in range(len(c.pos)):
            assert np.array_equal(d[c.slots[b], :, c.pos[b]], new[b].astype(np.float16))


@pytest.mark.parametrize("nh,nkv", [(32, 8), (3, 3), (6, 3), (16, 2)])
@pytest.mark.parametrize("window,sinks", RANGES)
def test_window_q8(kdlib, nh, nkv, window, sinks):
    c = Case(True, window % 1000 + sinks % 1000 + nh, nh, nkv, 128, 602, [0, 1, 6, 63, 64, 127, 200, 263, 601, 333],
             window, sinks)
    c.check(c.run(kdlib))


def test_window_of_everything_equals_the_plain_call(kdlib):
    """A wide Q8_0 window that hides nothing: the same items, so the same bits as kd_attn_append_decode_q8."""
    kd = kdlib
    c = Case(True, 5, 32, 8, 128, 2300, [0, 63, 64, 300, 2299], 2300, 0)
    got = c.run(kd)
    out = torch.empty(5, 32 * 128, dtype=torch.int16, device="cuda")
    ws = torch.empty(kd.kd_attn_workspace_bytes(5, 32, 128, 2300), dtype=torch.uint8, device="cuda")
    kd.kd_attn_append_decode_q8(c.dq, c.dk, c.dv, *c.dev, c.slots, c.pos, 32, 8, c.n_slots, 2300, out, ws)
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), got.view(np.int16))


# windows run on one to eight CTAs per row and KV head, by the batch
@pytest.mark.parametrize("q8,nh,nkv,hd,window", [(False, 16, 4, 128, 700), (True, 16, 4, 128, 700), (False, 32, 8, 128, 1300),
                                                 (False, 8, 8, 64, 1990), (False, 64, 8, 128, 1024), (False, 8, 8, 128, 3000)])
def test_window_rows_do_not_depend_on_the_batch(kdlib, q8, nh, nkv, hd, window):
    c = Case(q8, 11, nh, nkv, hd, 5000, list(range(17, 4900, 305))[:16], window, 9)
    got = c.run(kdlib)
    c.check(got)
    for b in (0, 1, 7, 15):
        one = c.run(kdlib, slice(b, b + 1))
        assert np.array_equal(one[0].view(np.int16), got[b].view(np.int16)), b


@pytest.mark.parametrize("nh,nkv,window", [(32, 8, 4500), (8, 8, 2200), (16, 2, 4990), (8, 4, 2500)])
@pytest.mark.parametrize("hd", [64, 128])
def test_wide_window_rows_in_batches_of_every_size(kdlib, hd, nh, nkv, window):
    c = Case(False, 12, nh, nkv, hd, 5000, [4999, 4500, 4321, 60, 2048, 0, 1500, 3001] + list(range(17, 4900, 700)), window, 9)
    got = c.run(kdlib)
    c.check(got)
    for n in (1, 2, 3, 4, 8):
        some = c.run(kdlib, slice(0, n))
        assert np.array_equal(some.view(np.int16), got[:n].view(np.int16)), n


@pytest.mark.parametrize("q8", [False, True])
def test_window_long_cache(kdlib, q8):
    """65536-position slots, 32-warp merges, the last position; byte offsets past 2^32 (the last of 70 slots)."""
    c = Case(q8, 3, 16, 4, 128, 65536, [65535, 40001, 8190], 8190, 70, n_slots=70 if not q8 else 140, last_slot=True)
    assert c.dev[0].numel() * c.dev[0].element_size() > 2 ** 32
    c.check(c.run(kdlib))


def test_window_large_scores(kdlib):
    """Scores of several hundred: one key takes nearly all of the weight."""
    c = Case(False, 8, 8, 2, 128, 300, [5, 130, 299], 100, 4, kscale=60.0)
    c.check(c.run(kdlib))


@pytest.mark.parametrize("q8,cap,window", [(False, 400, 90), (True, 400, 90), (False, 4000, 3500)])
def test_window_captured_graphs_share_a_workspace(kdlib, q8, cap, window):
    """Two captured calls on one workspace, replayed in turn on a side stream, each with its own inputs."""
    kd = kdlib
    cs = [Case(q8, 40 + i, 8, 2, 128, cap, [cap - 1 - i, 70 + i, 3], window, 5) for i in range(2)]
    want = [c.run(kd) for c in cs]
    ws = cs[0].workspace(kd, 3)
    outs = [torch.zeros(3, 8 * 128, dtype=torch.int16, device="cuda") for _ in cs]
    s = torch.cuda.Stream()
    graphs = []
    torch.cuda.synchronize()
    for c, o in zip(cs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.call(kd, o, ws)
        graphs.append(g)
    with torch.cuda.stream(s):
        for _ in range(3):
            for g in graphs:
                g.replay()
    s.synchronize()
    for o, w in zip(outs, want):
        assert np.array_equal(o.cpu().numpy(), w.view(np.int16))


# ------------------------------------------------------------------ the model's step ---
def windowed_step(shape, w, tok, pos, cache, window, sinks, q8):
    """One session's step from the oracle's parts.  cache: K, V, [L][nkv][cap] rows of fp16 bits or Q8_0 blocks."""
    s, group = shape, shape.n_heads // shape.n_kv_heads
    seen = visible(pos, window, sinks)
    x = oracle.q8_0_dequant_row(w["tok_embd"][tok], s.hidden)
    for l in range(s.n_layers):
        xn = oracle.rmsnorm_f16(x, w[f"blk.{l}.attn_norm"], s.rms_eps)
        q, k, v = (oracle.matvec_q8_0(w[f"blk.{l}.attn_{n}"], xn).reshape(-1, s.head_dim) for n in "qkv")
        for h in range(s.n_kv_heads):
            for c, row in ((cache[0], oracle.rope_neox(k[h], pos, s.rope_theta)), (cache[1], v[h])):
                if q8:
                    c[l, h, pos] = oracle.q8_0_quantize_f32(row.astype(np.float32)).reshape(-1, 34)
                else:
                    c[l, h, pos] = row.astype(np.float16).view(np.uint16)
        att = []
        for h in range(s.n_heads):
            K, V = (np.ascontiguousarray(c[l, h // group][seen]) for c in cache)
            head = oracle.attention_head_q8 if q8 else oracle.attention_head
            att.append(head(oracle.rope_neox(q[h], pos, s.rope_theta), K, V))
        att = np.concatenate(att).astype(np.float16).astype(np.float64)
        x = (x + oracle.matvec_q8_0(w[f"blk.{l}.attn_output"], att)).astype(np.float32).astype(np.float64)
        z = oracle.rmsnorm_f16(x, w[f"blk.{l}.ffn_norm"], s.rms_eps)
        g, u = (oracle.matvec_q8_0(w[f"blk.{l}.ffn_{n}"], z) for n in ("gate", "up"))
        act = (np.array([oracle.silu(y) for y in g]) * u).astype(np.float16).astype(np.float64)
        x = (x + oracle.matvec_q8_0(w[f"blk.{l}.ffn_down"], act)).astype(np.float32).astype(np.float64)
    return oracle.matvec_q8_0(w["output"], oracle.rmsnorm_f16(x, w["output_norm"], s.rms_eps))


@pytest.mark.parametrize("name,flags", [("hd64", 0), ("hd64", 1), ("hd64", 64), ("hd128", 0), ("wide", 0), ("q8", 0), ("q8", 1)])
def test_model_window_steps(kdlib, name, flags):
    """Steps with a window, teacher-forced, logits within the step's gate (5e-2); then each session alone (the
    same bits), and with the window off again the plain step's bits."""
    kd = kdlib
    q8 = name == "q8"
    shape = synth.TINY if name == "hd64" else synth.TINY_HD128
    w = dict(synth.model_weights(shape, 0), **synth.norm_weights(shape, 5))
    cap, lens, window, sinks = (256, (150, 20, 201), 70, 3) if name != "wide" else (2600, (2450, 20, 2201), 2150, 3)
    flags |= kd.KD_FLAG_KV_Q8_0 if q8 else 0

    def load(which):
        m = kd.kd_model_load(kd.make_config(shape, 4, cap, flags), w)
        ids = []
        for i in which:
            k, v = synth.kv_prefill(shape, 0, i, lens[i])
            sid = kd.kd_session_bind(m)
            kd.kd_session_load_kv(m, sid, k, v, lens[i])
            ids.append(sid)
        return m, ids

    def step(m, ids, tok, pos):
        lg = torch.empty(len(ids), shape.vocab, device="cuda")
        kd.kd_decode_step(m, ids, tok, pos, lg, None)
        torch.cuda.synchronize()
        return lg.cpu().numpy()

    om = oracle.OracleModel(shape, w, kv_q8_0=q8)
    caches = [om.new_cache(cap, *synth.kv_prefill(shape, 0, i, n)) for i, n in enumerate(lens)]
    toks = [synth.tokens(t, "win", 3, shape.vocab) for t in range(4)]
    m, ids = load((0, 1, 2))
    plain, _ = load(())
    try:
        step(m, ids, toks[3], [n - 1 for n in lens])  # a plain step first (captured without the window)
        for i, n in enumerate(lens):  # restore the overwritten row
            kd.kd_session_load_kv(m, ids[i], *synth.kv_prefill(shape, 0, i, n), n)
        kd.kd_model_set_window(m, window, sinks)
        got = []
        for t in range(3):
            pos = [n + t for n in lens]
            got.append(step(m, ids, toks[t], pos))
            for b in range(3):
                ref = windowed_step(shape, w, int(toks[t][b]), pos[b], caches[b], window, sinks, q8)
                assert np.abs(got[t][b] - ref).max() <= 5e-2, (t, b)
        assert kd.kd_device_status(m) == 0
        for b in (0, 2):
            m1, id1 = load((b,))
            try:
                kd.kd_model_set_window(m1, window, sinks)
                for t in range(3):
                    one = step(m1, id1, toks[t][b:b + 1], [lens[b] + t])
                    assert np.array_equal(one[0], got[t][b]), (b, t)
            finally:
                kd.kd_model_free(m1)
        kd.kd_model_set_window(m, 0)
        k, v = synth.kv_prefill(shape, 0, 0, lens[0])
        kd.kd_session_load_kv(m, ids[0], k, v, lens[0])
        sid = kd.kd_session_bind(plain)
        kd.kd_session_load_kv(plain, sid, k, v, lens[0])
        a, b = step(m, ids[:1], toks[0][:1], [lens[0]]), step(plain, [sid], toks[0][:1], [lens[0]])
        assert np.array_equal(a, b)
    finally:
        kd.kd_model_free(m)
        kd.kd_model_free(plain)


def test_window_wait_timeout_is_reported(kdlib):
    """A bounded wait of the windowed attention made to run out: KD_ERR_DEVICE once, then correct steps again.
    Over an fp16 cache it waits on no barrier, and the hook says so."""
    kd = kdlib
    w = synth.model_weights(synth.TINY, 0)
    m = kd.kd_model_load(kd.make_config(synth.TINY, 2, 4096), w)
    try:
        kd.kd_debug_inject_wait_timeout(m, "qkv")
        kd.kd_model_set_window(m, 3500, 3)
        with pytest.raises(kd.KdError) as e:
            kd.kd_debug_inject_wait_timeout(m, "attn_split")
        assert e.value.name == "KD_ERR_INVALID_ARG"
    finally:
        kd.kd_model_free(m)
    shape = synth.TINY_HD128
    w = synth.model_weights(shape, 0)
    m = kd.kd_model_load(kd.make_config(shape, 2, 4096, kd.KD_FLAG_KV_Q8_0), w)
    try:
        kd.kd_model_set_window(m, 3500, 3)
        sid = kd.kd_session_bind(m)
        kd.kd_session_load_kv(m, sid, *synth.kv_prefill(shape, 0, 0, 150), 150)
        lg = torch.empty(1, shape.vocab, device="cuda")

        def step():
            kd.kd_decode_step(m, [sid], [7], [150], lg, None)
            torch.cuda.synchronize()
            return lg.cpu().numpy().copy()
        want = step()
        kd.kd_debug_inject_wait_timeout(m, "attn_split")
        step()
        with pytest.raises(kd.KdError) as e:
            kd.kd_device_status(m)
        assert e.value.name == "KD_ERR_DEVICE"
        assert np.array_equal(step(), want)
        assert kd.kd_device_status(m) == 0
    finally:
        kd.kd_model_free(m)


@pytest.mark.parametrize("q8", [False, True])
def test_calls_on_two_streams_at_once(kdlib, q8):
    """Two callers, each with its own cache, workspace and stream, wide and short windows in turn."""
    kd = kdlib
    cs = [Case(q8, 60 + i, 16, 4, 128, 3000, [2999 - i, 1500, 70], w, 5) for i, w in enumerate((2600, 300))]
    want = [c.run(kd) for c in cs]
    ws = [c.workspace(kd, 3) for c in cs]
    outs = [torch.zeros(3, 16 * 128, dtype=torch.int16, device="cuda") for _ in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, o, w, s in zip(cs, outs, ws, streams):
            c.call(kd, o, w, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert np.array_equal(o.cpu().numpy(), w.view(np.int16))


@pytest.mark.parametrize("hd", [64, 128])
def test_wide_windows_of_groups_of_eight(kdlib, hd):
    """64 query heads over 8 KV heads, more than 2048 visible keys: a row and KV head on one CTA (12 rows; its records pass
    through the workspace), on clusters of two (5 and 9), four (3, 4) and eight (1, 2).  The same bits in each."""
    c = Case(False, 21, 64, 8, hd, 2700, [2699, 2500, 2050, 60, 2048, 0, 1500, 2301, 33, 1000, 2600, 2699], 2560, 9)
    got = c.run(kdlib)
    c.check(got)
    for n in (1, 2, 3, 4, 5, 9):
        some = c.run(kdlib, slice(0, n))
        assert np.array_equal(some.view(np.int16), got[:n].view(np.int16)), n


@pytest.mark.parametrize("name,flags", [("hd64", 0), ("hd64", 1), ("wide", 0), ("q8", 0)])
def test_model_window_steps_of_more_than_sixteen_sessions(kdlib, name, flags):
    """20 windowed sessions a step (rows in groups of 16 and 4), two steps: each session's logits are those of
    the session stepped alone, bit for bit."""
    kd = kdlib
    shape = synth.TINY if name == "hd64" else synth.TINY_HD128
    w = dict(synth.model_weights(shape, 0), **synth.norm_weights(shape, 5))
    n, cap, window, sinks = (20, 256, 70, 3) if name != "wide" else (20, 2600, 2150, 3)
    flags |= kd.KD_FLAG_KV_Q8_0 if name == "q8" else 0
    lens = [1 + 11 * i for i in range(n)] if name != "wide" else [2590 - 130 * i for i in range(n)]
    m = kd.kd_model_load(kd.make_config(shape, n, cap, flags), w)
    one = kd.kd_model_load(kd.make_config(shape, 1, cap, flags), w)
    try:
        for x in (m, one):
            kd.kd_model_set_window(x, window, sinks)
        rows = [synth.kv_prefill(shape, 0, i, lens[i]) for i in range(n)]
        ids = []
        for i in range(n):
            ids.append(kd.kd_session_bind(m))
            kd.kd_session_load_kv(m, ids[i], *rows[i], lens[i])
        toks = [synth.tokens(t, "many", n, shape.vocab) for t in range(2)]
        lg = torch.empty(n, shape.vocab, device="cuda")
        got = []
        for t in range(2):
            kd.kd_decode_step(m, ids, toks[t], [x + t for x in lens], lg, None)
            got.append(lg.cpu().numpy().copy())
        assert kd.kd_device_status(m) == 0
        sid = kd.kd_session_bind(one)
        for i in range(n):
            kd.kd_session_load_kv(one, sid, *rows[i], lens[i])
            for t in range(2):
                kd.kd_decode_step(one, [sid], toks[t][i:i + 1], [lens[i] + t], lg[:1], None)
                assert np.array_equal(lg[0].cpu().numpy(), got[t][i]), (i, t)
    finally:
        kd.kd_model_free(m)
        kd.kd_model_free(one)


FRESH = """
import numpy as np, torch
import session_decode_step_gb300 as kd
kd.lib()
x = torch.randn(1, 16, 128, device="cuda")
cache = torch.randn(2, 2, 4, 4096, 128, device="cuda", dtype=torch.float16)
out = torch.zeros(1, 16 * 128, device="cuda", dtype=torch.float16)
ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")

def window(hd, w, nkv=4):
    kd.kd_attn_window_append_decode(x, x, x, cache[0], cache[1], [1], [3000], 16, nkv, hd, 2, 4096, w, 3, out, ws)

def captured(call):
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        call()
    return g
"""


def fresh(code):
    """A process of its own, in which no kernel of the library has run."""
    r = subprocess.run([sys.executable, "-c", FRESH + code], capture_output=True, text=True, timeout=300,
                       cwd=Path(__file__).resolve().parent.parent)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


def test_a_first_call_sets_up_no_windowed_kernels(kdlib):
    """The device memory that a process's first call takes is the kernels of the plain path and the workspaces'
    (2.1 MB, in steps of 2 MB); the 64 windowed kernels of all shapes are another 4 MB."""
    took = fresh("""
torch.cuda.synchronize()
before = torch.cuda.mem_get_info()[0]
kd.kd_attn_append_decode(x, x, x, cache[0], cache[1], [1], [30], 16, 4, 128, 2, 4096, out, ws)
torch.cuda.synchronize()
print(before - torch.cuda.mem_get_info()[0])
""")
    assert int(took.split()[-1]) < 4 << 20, took


@pytest.mark.parametrize("hd,w,nkv", [(128, 40, 4), (128, 4000, 4), (64, 4000, 2), (64, 1000, 8)])
def test_a_first_windowed_call_may_be_captured(kdlib, hd, w, nkv):
    """Captured without any call before it, or after another shape's; replayed, and compared with the call itself."""
    for before in ("", "window(128, 7)"):
        fresh(f"""
{before}
g = captured(lambda: window({hd}, {w}, {nkv}))
out.zero_()
g.replay()
torch.cuda.synchronize()
got = out.clone()
window({hd}, {w}, {nkv})
torch.cuda.synchronize()
assert torch.isfinite(got).all() and got.abs().sum() > 0 and torch.equal(got, out)
""")
