"""Measured cases of the operators around paged sessions.

- rotary positions: half and interleaved pairs, part of a head, scaled for long contexts;
- paged append: new keys (rotated on the way) and values into the pages of fp16 or Q8_0
  caches, a token per session or whole prompts, with the queries rotated alongside;
- paged attention: a decode step's attention through page tables, a prefix that a group of
  sessions shares taken once for all of them.

`run` computes an operator in its plain form with elementary torch operations, or, with
`own` true, calls the framework.  `exact` gives the same outputs in 64 bits from the
operator's definition.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # Eight sessions' query heads of one decode step at far-apart positions: what a layer waits for.
        dict(name="rope step", op="rope", T=8, heads=32, hd=128, rot=128, layout="half", type="fp32", theta=500000.0,
             scaling="bands", factor=8.0, low=1.0, high=4.0, original=8192, far=32768, mix=1),
        # A long prompt's queries and keys together, positions past the trained context.
        dict(name="rope prompt", op="rope", T=8191, heads=40, hd=128, rot=128, layout="half", type="fp16",
             theta=500000.0, scaling="ramp", factor=4.0, low=1.0, high=32.0, original=32768, far=0, mix=2),
        # One token for each of eight sessions: queries rotated, keys rotated and written, values written.
        dict(name="append step", op="append", B=8, lo=1, hi=1, first=1238, nh=32, n_kv=8, hd=128, page=16, rot=128,
             layout="half", type="fp32", theta=500000.0, scaling="none", factor=1.0, low=1.0, high=4.0, original=8192,
             fused=False, mix=3),
        # Four prompts arriving together out of one fused projection, 64 of 128 dims in interleaved pairs.
        dict(name="append prompts", op="append", B=4, lo=1238, hi=4096, first=0, nh=32, n_kv=8, hd=128, page=64, rot=64,
             layout="pairs", type="bf16", theta=10000.0, scaling="linear", factor=4.0, low=1.0, high=4.0, original=8192,
             fused=True, mix=4),
        # Turns of ragged conversations continued on the Q8_0 cache, at odd places within pages of 32.
        dict(name="append q8 turns", op="append_q8", B=11, lo=3, hi=2001, first=25704, nh=0, n_kv=8, hd=128, page=32,
             rot=128, layout="half", type="fp16", theta=500000.0, scaling="bands", factor=8.0, low=1.0, high=4.0,
             original=8192, fused=False, mix=5),
        # One short session: pure latency.
        dict(name="paged B1 short", op="attn", B=1, groups=0, prefix=0, step=0, lo=37, hi=37, nh=32, n_kv=8, hd=128, page=16,
             mix=6),
        # Eight chats around 1238 positions and beyond: the ordinary decode step.
        dict(name="paged B8", op="attn", B=8, groups=0, prefix=0, step=0, lo=1238, hi=1365, nh=32, n_kv=8, hd=128, page=16,
             mix=7),
        # A full server: sessions of all ages, one of them empty; the caches' bytes dominate.
        dict(name="paged B48 ragged", op="attn", B=48, groups=0, prefix=0, step=0, lo=0, hi=16384, nh=32, n_kv=8, hd=128,
             page=64, mix=8),
        # Sixteen beams of one long prompt, each a little way on.
        dict(name="shared beams", op="attn", B=16, groups=1, prefix=8111, step=0, lo=1, hi=200, nh=32, n_kv=8, hd=128,
             page=16, mix=9),
        # 64-wide heads in pairs, three few-shot prompts, odd lengths, pages of 48.
        dict(name="shared hd64 odd", op="attn", B=15, groups=3, prefix=1013, step=77, lo=0, hi=333, nh=14, n_kv=7, hd=64,
             page=48, mix=10),
        # Sixty-four chats behind two long system prompts.
        dict(name="shared 64", op="attn", B=64, groups=2, prefix=16384, step=-1001, lo=60, hi=1000, nh=32, n_kv=8, hd=128,
             page=64, mix=11),
        # Questions about three long documents on the Q8_0 cache.
        dict(name="shared q8 long", op="attn_q8", B=24, groups=3, prefix=25704, step=1000, lo=20, hi=1000, nh=32, n_kv=8,
             hd=128, page=32, mix=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_rope(rng, hd):
    scaling = rng.choice(("none", "linear", "bands", "ramp"))
    low, high = (1.0, 32.0) if scaling == "ramp" else (1.0, 4.0)
    return dict(hd=hd, rot=rng.choice((hd, hd, hd // 2, 2 * rng.randint(1, hd // 2))), layout=rng.choice(("half", "pairs")),
                type=rng.choice(("fp32", "fp16", "bf16")), theta=rng.choice((10000.0, 500000.0)), scaling=scaling,
                factor=1.0 if scaling == "none" else rng.choice((2.0, 4.0, 8.0, 10.0)), low=low, high=high,
                original=rng.choice((2048, 8192, 32768)), mix=rng.randrange(1 << 20))


def _draw(rng):
    op = rng.choice(("rope", "rope", "append", "append", "append_q8", "attn", "attn", "attn", "attn_q8"))
    if op == "rope":
        c = _draw_rope(rng, rng.choice((64, 128, 128, 8 * rng.randint(2, 32))))
        return dict(op=op, T=_log_int(rng, 1, 16384), heads=_log_int(rng, 1, 64), far=rng.choice((0, 2048, 100000)), **c)
    n_kv = rng.randint(1, 8)
    page = rng.choice((16, 16, 32, 48, 64, 128, 256))
    if op.startswith("append"):
        c = _draw_rope(rng, 128 if op == "append_q8" else rng.choice((64, 128)))
        lo = rng.choice((1, 1, _log_int(rng, 1, 512)))
        return dict(op=op, B=_log_int(rng, 1, 64), lo=lo, hi=lo if rng.random() < 0.4 else _log_int(rng, lo, 4096),
                    first=rng.choice((0, _log_int(rng, 1, 32768))), nh=n_kv * rng.choice((0, 1, 2, 4, 8)), n_kv=n_kv,
                    page=page, fused=rng.random() < 0.5, **c)
    B = _log_int(rng, 1, 64)
    groups = rng.choice((0, rng.randint(1, max(1, min(B, 6)))))
    lo = _log_int(rng, 1, 2048) - 1
    hi = _log_int(rng, max(1, lo), 16384)
    prefix = _log_int(rng, 16, 32768) if groups else 0
    return dict(op=op, B=B, groups=groups, prefix=prefix, step=rng.randint(0, prefix // 8) if groups > 1 else 0, lo=lo,
                hi=max(lo, hi), nh=n_kv * rng.choice((1, 2, 4, 8)), n_kv=n_kv,
                hd=128 if op == "attn_q8" else rng.choice((64, 128, 128)), page=page, mix=rng.randrange(1 << 20))


def _gathered(c):
    """Values that the plain attention gathers: every session padded to the longest."""
    lens, _, _ = _lens(c)
    return int(lens.max()) * c["B"] * c["n_kv"] * c["hd"]


def draw(rng):
    most = {}
    for c in listed():
        kind = c["op"].split("_")[0]
        w = work(c)
        old = most.get(kind, (0, 0, 0))
        most[kind] = (max(old[0], w["bytes"]), max(old[1], w["flops"]),
                      max(old[2], _gathered(c) if kind == "attn" else 0))
    while True:
        c = _draw(rng)
        kind = c["op"].split("_")[0]
        w = work(c)
        if w["bytes"] <= most[kind][0] and w["flops"] <= most[kind][1] and (kind != "attn" or _gathered(c) <= most[kind][2]):
            return c


# ---------------------------------------------------------------- the cases' plans ---
def _spread(c, n):
    """n lengths between lo and hi, spread over their logarithm, the ends among them where there is room."""
    r = random.Random(c["mix"])
    v = [round((c["hi"] + 1) ** u * (c["lo"] + 1) ** (1 - u)) - 1 for u in (r.random() for _ in range(n))]
    if n >= 4:
        v[n // 2], v[n // 3] = c["lo"], c["hi"]
    return [min(max(x, c["lo"]), c["hi"]) for x in v]


def _tokens(c):
    """Appending: each session's first new position and its number of new tokens."""
    counts = np.array(_spread(c, c["B"]), np.int32)
    r = random.Random(c["mix"] + 1)
    starts = np.array([c["first"] + (r.randrange(max(1, c["first"])) if c["first"] else 0) for _ in range(c["B"])], np.int32)
    return starts, counts


def _lens(c):
    """Attention: each session's keys, the groups' sizes and their shared prefixes."""
    own_keys = np.array(_spread(c, c["B"]), np.int32)
    if not c["groups"]:
        return own_keys, np.zeros(0, np.int32), np.zeros(0, np.int32)
    n = c["groups"]
    rows = np.array([c["B"] // n + (g < c["B"] % n) for g in range(n)], np.int32)
    prefix = np.array([c["prefix"] + g * c["step"] for g in range(n)], np.int32)
    return own_keys + np.repeat(prefix, rows), rows, prefix


def work(case):
    c = case
    if c["op"] == "rope":
        size = 4 if c["type"] == "fp32" else 2
        return {"bytes": 2 * size * c["T"] * c["heads"] * c["hd"] + 4 * c["T"], "flops": 3 * c["T"] * c["heads"] * c["rot"]}
    if c["op"].startswith("append"):
        starts, counts = _tokens(c)
        t, size = int(counts.sum()), 4 if c["type"] == "fp32" else 2
        row = 136 if c["op"] == "append_q8" else 2 * c["hd"]
        pages = int((-(-(starts + counts) // c["page"]) - starts // c["page"]).sum())
        return {"bytes": t * (2 * c["n_kv"] * (size * c["hd"] + row) + c["nh"] * c["hd"] * (size + 4)) + 4 * pages,
                "flops": 3 * t * (c["n_kv"] + c["nh"]) * c["rot"]}
    lens, rows, prefix = _lens(c)
    shared = int(prefix.sum()) - int((np.repeat(prefix, rows)).sum()) if c["groups"] else 0
    keys = int(lens.sum()) + shared
    row = 136 if c["op"] == "attn_q8" else 2 * c["hd"]
    return {"bytes": 2 * keys * c["n_kv"] * row + 6 * c["B"] * c["nh"] * c["hd"] + 4 * (keys // c["page"] + 1),
            "flops": 4 * int(lens.sum()) * c["nh"] * c["hd"]}


# ------------------------------------------------------------------------- inputs ---
def _normal(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _planes(g, q8, n_pages, c):
    """K's and V's pages: [fp16 rows] * 2, or [quants, scales] * 2."""
    shape = (n_pages, c["n_kv"], c["page"])
    if not q8:
        return [_normal(g, (*shape, c["hd"]), torch.float16) for _ in range(2)]
    planes = []
    for _ in range(2):
        planes.append(torch.randint(1, 256, (*shape, 128), generator=g, device="cuda", dtype=torch.uint8))
        planes.append((torch.rand((*shape, 4), generator=g, device="cuda", dtype=torch.float16) + 0.5) * (2.5 / 127))
    return planes


def _rope_plan(c):
    import session_decode_step_gb300 as kd
    layout = {"half": kd.KD_ROPE_HALF, "pairs": kd.KD_ROPE_PAIRS}[c["layout"]]
    scaling = {"none": kd.KD_ROPE_UNSCALED, "linear": kd.KD_ROPE_LINEAR, "bands": kd.KD_ROPE_BANDS, "ramp": kd.KD_ROPE_RAMP}
    return kd.kd_rope_plan(c["hd"], c["theta"], rot_dim=c["rot"], layout=layout, scaling=scaling[c["scaling"]],
                           factor=c["factor"], low=c["low"], high=c["high"], original_ctx=c["original"],
                           magnitude=_magnitude(c))


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = {"case": c}
    if c["op"] == "rope":
        s["x"] = _normal(g, (c["T"], c["heads"], c["hd"]), TYPES[c["type"]])
        pos = rng.integers(0, c["far"], c["T"]) if c["far"] else np.arange(c["T"]) + rng.integers(0, 100000)
        s["pos"] = torch.from_numpy(pos.astype(np.int32)).cuda()
        s["out"] = torch.empty_like(s["x"])
        if own:
            s["plan"] = _rope_plan(c)
        return s
    q8, ps = c["op"].endswith("q8"), c["page"]
    if c["op"].startswith("append"):
        s["starts"], s["counts"] = _tokens(c)
        T = int(s["counts"].sum())
        need = -(-(s["starts"] + s["counts"]) // ps)  # a session's pages; those before its new tokens are elsewhere
        skip = s["starts"] // ps
        used = need - skip
        s["n_pages"] = int(used.sum()) + 3
        ids = rng.permutation(s["n_pages"]).astype(np.int32)
        table = np.zeros((c["B"], int(need.max()) + 2), np.int32)
        at = 0
        for b in range(c["B"]):
            table[b, skip[b]:need[b]] = ids[at:at + used[b]]
            at += used[b]
        s["table"] = torch.from_numpy(table).cuda()
        s["planes"] = _planes(g, q8, s["n_pages"], c)
        widths = [c["nh"], c["n_kv"], c["n_kv"]]
        if c["fused"]:
            s["q"], s["k"], s["v"] = _normal(g, (T, sum(widths), c["hd"]), TYPES[c["type"]]).split(widths, 1)
        else:
            s["q"], s["k"], s["v"] = (_normal(g, (T, w, c["hd"]), TYPES[c["type"]]) for w in widths)
        s["q_out"] = torch.empty(T, c["nh"], c["hd"], device="cuda")
        seq = np.repeat(np.arange(c["B"]), s["counts"])
        pos = np.concatenate([np.arange(n) + p for p, n in zip(s["starts"], s["counts"])]).astype(np.int64)
        if q8:  # the appended rows, to be read back as values
            row = (table[seq, pos // ps].astype(np.int64)[:, None] * c["n_kv"] + np.arange(c["n_kv"])) * ps + (pos % ps)[:, None]
            s["new_rows"] = torch.from_numpy(row.reshape(-1)).cuda()
        if own:
            s["plan"] = _rope_plan(c)
        return s
    B = c["B"]
    s["lens"], s["rows"], s["prefix"] = _lens(c)
    need = -(-s["lens"] // ps)
    first = np.concatenate([[0], np.cumsum(s["rows"])]).astype(int)
    whole = np.zeros(B, int)  # leading pages that a session has from its group's first one
    for i, p in enumerate(s["prefix"]):
        whole[first[i] + 1:first[i + 1]] = p // ps
    s["n_pages"] = int((need - whole).sum()) + 2
    ids = rng.permutation(s["n_pages"]).astype(np.int32)
    table = np.zeros((B, max(1, int(need.max())) + 1), np.int32)
    at = 0
    for b in range(B):
        n = need[b] - whole[b]
        table[b, whole[b]:need[b]] = ids[at:at + n]
        at += n
    s["planes"] = _planes(g, q8, s["n_pages"], c)
    for i, p in enumerate(s["prefix"]):
        lead = first[i]
        for b in range(lead + 1, first[i + 1]):
            table[b, :p // ps] = table[lead, :p // ps]
            if p % ps:  # the page that the prefix ends in: a copy for each session
                for t in s["planes"]:
                    t[table[b, p // ps], :, :p % ps] = t[table[lead, p // ps], :, :p % ps]
    s["table"] = torch.from_numpy(table).cuda()
    s["q"] = _normal(g, (B, c["nh"], c["hd"]))
    s["out"] = torch.empty(B, c["nh"] * c["hd"], dtype=torch.float16, device="cuda")
    if own:
        import session_decode_step_gb300 as kd
        s["workspace"] = torch.empty(kd.kd_attn_paged_workspace_bytes(B, c["nh"], c["n_kv"], c["hd"]), dtype=torch.uint8,
                                     device="cuda")
    return s


# ---------------------------------------------------------------------------- run ---
def _magnitude(c):
    return 0.1 * math.log(c["factor"]) + 1 if c["scaling"] == "ramp" else 1.0


def _frequencies(c):
    """The angle per position of each pair, in 64 bits."""
    n = c["rot"]
    i = np.arange(n // 2, dtype=np.float64)
    f = c["theta"] ** (-2 * i / n)
    if c["scaling"] == "linear":
        f = f / c["factor"]
    elif c["scaling"] == "bands":  # long waves slowed down by the factor, short ones kept, a blend between
        turns = c["original"] * f / (2 * math.pi)
        keep = np.clip((turns - c["low"]) / (c["high"] - c["low"]), 0, 1)
        f = f * (keep + (1 - keep) / c["factor"])
    elif c["scaling"] == "ramp":   # the same with a blend that is linear over the pairs
        def pair(turns):
            return n * math.log(c["original"] / (turns * 2 * math.pi)) / (2 * math.log(c["theta"]))
        a, b = max(math.floor(pair(c["high"])), 0), min(math.ceil(pair(c["low"])), n - 1)
        slow = np.clip((i - a) / max(b - a, 0.001), 0, 1)
        f = f * (1 - slow + slow / c["factor"])
    return f


def _rotate(c, x, pos, dtype=torch.float32):
    """x [T][H][hd] rotated in `dtype`; the angles in 64 bits, as far positions need."""
    angle = pos.double()[:, None] * torch.from_numpy(_frequencies(c)).cuda()
    cos, sin = ((t * _magnitude(c)).to(dtype)[:, None] for t in (angle.cos(), angle.sin()))
    x = x.to(dtype)
    n = c["rot"]
    if c["layout"] == "half":
        a, b = x[..., :n // 2], x[..., n // 2:n]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., n:]], -1)
    a, b = x[..., 0:n:2], x[..., 1:n:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., n:]], -1)


def _quantise(x):
    """fp32 rows of 128 into Q8_0 codes (q + 128) and fp16 block scales: d = max|x| / 127 in fp32,
    q = x / d in fp32 rounded half away from zero."""
    x = x.view(*x.shape[:-1], 4, 32)
    d = x.abs().amax(-1)
    d = d / torch.full_like(d, 127)  # a division by a tensor is rounded once; by a number it is a product
    y = (x / torch.where(d > 0, d, 1)[..., None]).double()
    q = torch.sign(y) * torch.floor(y.abs() + 0.5)
    return (q.clamp(-127, 127) + 128).to(torch.uint8).flatten(-2), d.half()


def _values(quants, scales):
    """The values that Q8_0 rows stand for."""
    return ((quants.view(*quants.shape[:-1], 4, 32) - 128.0) * scales[..., None]).flatten(-2)


def _new_rows(s):
    """The appended rows as the values they stand for, read back from the pages: K's, then V's."""
    p, i = s["planes"], s["new_rows"]
    return [_values(p[j].view(-1, 128).index_select(0, i), p[j + 1].view(-1, 4).index_select(0, i)) for j in (0, 2)]


def _append_plain(s):
    c = s["case"]
    seq = torch.from_numpy(np.repeat(np.arange(c["B"]), s["counts"])).cuda()
    pos = torch.from_numpy(np.concatenate([np.arange(n) + p for p, n in zip(s["starts"], s["counts"])])).cuda().long()
    page, row = s["table"][seq, pos // c["page"]].long(), pos % c["page"]
    if c["op"] == "append":
        s["planes"][0][page, :, row] = _rotate(c, s["k"], pos).half()
        s["planes"][1][page, :, row] = s["v"].half()
    else:
        # in 64 bits and rounded to fp32: the codes' borders lie between neighbouring values
        for i, x in enumerate((_rotate(c, s["k"], pos, torch.float64).float(), s["v"].float())):
            s["planes"][2 * i][page, :, row], s["planes"][2 * i + 1][page, :, row] = _quantise(x)
    if c["nh"]:
        s["q_out"].copy_(_rotate(c, s["q"], pos))
    return _append_outputs(s)


def _append_outputs(s):
    c = s["case"]
    k, v = _new_rows(s) if c["op"] == "append_q8" else s["planes"]
    return {"k": k, "v": v, "q": s["q_out"]} if c["nh"] else {"k": k, "v": v}


def _attn_plain(s):
    c = s["case"]
    lens = torch.from_numpy(s["lens"]).cuda()
    t = torch.arange(max(1, int(s["lens"].max())), device="cuda")
    page = s["table"].long()[:, t // c["page"]]
    heads = torch.arange(c["n_kv"], device="cuda")[None, :, None]
    at = (page[:, None], heads, (t % c["page"])[None, None])
    if c["op"] == "attn":
        k, v = (p[at].float() for p in s["planes"])
    else:
        k, v = (_values(s["planes"][i][at], s["planes"][i + 1][at]) for i in (0, 2))
    hidden = t >= lens[:, None]
    q = s["q"].view(c["B"], c["n_kv"], -1, c["hd"])
    x = (q @ k.transpose(-1, -2)) / math.sqrt(c["hd"])
    x = x.masked_fill(hidden[:, None, None, :], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True)).masked_fill(hidden[:, None, None, :], 0)
    o = (p @ v) / p.sum(-1, keepdim=True).clamp(min=1)  # the largest weight is 1; a session without keys gives zeros
    return o.reshape(c["B"], -1).half()


def run(s):
    c = s["case"]
    if not own:
        if c["op"] == "rope":
            return _rotate(c, s["x"], s["pos"]).to(s["x"].dtype)
        return _append_plain(s) if c["op"].startswith("append") else _attn_plain(s)
    import session_decode_step_gb300 as kd
    if c["op"] == "rope":
        kd.kd_rope(s["plan"], s["x"], s["pos"], s["out"])
        return s["out"]
    if c["op"].startswith("append"):
        q = dict(q=s["q"], q_out=s["q_out"], n_heads=c["nh"]) if c["nh"] else {}
        if c["op"] == "append":
            kd.kd_paged_append(s["plan"], s["k"], s["v"], *s["planes"], s["table"], s["starts"], s["counts"], c["n_kv"],
                               c["hd"], s["n_pages"], c["page"], **q)
        else:
            kd.kd_paged_append_q8(s["plan"], s["k"], s["v"], *s["planes"], s["table"], s["starts"], s["counts"], c["n_kv"],
                                  s["n_pages"], c["page"], **q)
        return _append_outputs(s)
    groups = dict(group_rows=s["rows"], group_prefix=s["prefix"]) if c["groups"] else {}
    if c["op"] == "attn":
        kd.kd_attn_paged_decode(s["q"], *s["planes"], s["table"], s["lens"], c["nh"], c["n_kv"], c["hd"], s["n_pages"],
                                c["page"], s["out"], s["workspace"], **groups)
    else:
        kd.kd_attn_paged_decode_q8(s["q"], *s["planes"], s["table"], s["lens"], c["nh"], c["n_kv"], s["n_pages"],
                                   c["page"], s["out"], s["workspace"], **groups)
    return s["out"]


# -------------------------------------------------------------------------- exact ---
def _exact_angles(c):
    n, out = c["rot"], []
    for i in range(n // 2):
        f = math.pow(c["theta"], -2.0 * i / n)
        if c["scaling"] == "linear":
            f /= c["factor"]
        elif c["scaling"] == "bands":
            wave = 2 * math.pi / f
            if wave > c["original"] / c["low"]:
                f /= c["factor"]
            elif wave >= c["original"] / c["high"]:
                u = (c["original"] / wave - c["low"]) / (c["high"] - c["low"])
                f = (1 - u) * f / c["factor"] + u * f
        elif c["scaling"] == "ramp":
            ends = [n * math.log(c["original"] / (2 * math.pi * r)) / math.log(c["theta"]) / 2 for r in (c["high"], c["low"])]
            a, b = max(0, math.floor(ends[0])), min(n - 1, math.ceil(ends[1]))
            u = min(1.0, max(0.0, (i - a) / (b - a if b > a else 0.001)))
            f = u * f / c["factor"] + (1 - u) * f
        out.append(f)
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def _exact_rope(c, x, pos):
    w = torch.outer(pos.to(torch.float64), _exact_angles(c))
    scale = 1 + math.log(c["factor"]) / 10 if c["scaling"] == "ramp" else 1.0
    turn = torch.polar(torch.full_like(w, scale), w)[:, None]
    y = x.to(torch.float64).clone()
    n = c["rot"]
    a, b = (slice(0, n // 2), slice(n // 2, n)) if c["layout"] == "half" else (slice(0, n, 2), slice(1, n, 2))
    z = torch.complex(y[..., a].contiguous(), y[..., b].contiguous()) * turn
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_append(c, s):
    got = {}
    pos = torch.cat([torch.arange(int(p), int(p) + int(n)) for p, n in zip(s["starts"], s["counts"])]).cuda()
    k, v = _exact_rope(c, s["k"], pos), s["v"].to(torch.float64)
    if c["op"] == "append":
        planes = [p.double() for p in s["planes"]]
        table, at = s["table"].cpu().numpy(), 0
        for b, (p, n) in enumerate(zip(s["starts"], s["counts"])):
            for lo in range(int(p) // c["page"], -(-int(p + n) // c["page"])):
                t0, t1 = max(lo * c["page"], int(p)), min((lo + 1) * c["page"], int(p + n))
                i0, r0 = at + t0 - int(p), t0 - lo * c["page"]
                for plane, x in zip(planes, (k, v)):
                    plane[table[b, lo], :, r0:r0 + t1 - t0] = x[i0:i0 + t1 - t0].transpose(0, 1)
            at += int(n)
        got["k"], got["v"] = planes
    else:
        for name, x in (("k", k), ("v", v)):
            x = x.to(torch.float32).cpu().numpy().reshape(-1, 32)  # the row format: of fp32 values, scale and quotient in fp32
            d = (np.abs(x).max(1) / np.float32(127)).astype(np.float32)
            with np.errstate(invalid="ignore"):
                r = np.where(d[:, None] > 0, x / d[:, None], 0).astype(np.float32).astype(np.float64)
            q = np.where(r < 0, -np.floor(0.5 - r), np.floor(r + 0.5))
            got[name] = (q * d.astype(np.float16).astype(np.float64)[:, None]).reshape(-1, 128)
    if c["nh"]:
        got["q"] = _exact_rope(c, s["q"], pos)
    return got


def _exact_attn(c, s):
    out = torch.zeros(c["B"], c["n_kv"], c["nh"] // c["n_kv"], c["hd"], dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        if not n:
            continue
        pages = s["table"][b, :-(-n // c["page"])].long()
        rows = []
        for i in range(2):
            if c["op"] == "attn":
                x = s["planes"][i][pages].double()
            else:
                q, d = (s["planes"][2 * i + j][pages].double() for j in range(2))
                x = (q - 128) * d.repeat_interleave(32, -1)
            rows.append(x.transpose(0, 1).flatten(1, 2)[:, :n])
        z = torch.einsum("hgd,htd->hgt", s["q"][b].double().view(c["n_kv"], -1, c["hd"]), rows[0]) * c["hd"] ** -0.5
        out[b] = torch.einsum("hgt,htd->hgd", torch.softmax(z, -1), rows[1])
    return out.view(c["B"], -1)


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    if c["op"] == "rope":
        return _exact_rope(c, s["x"], s["pos"])
    return _exact_append(c, s) if c["op"].startswith("append") else _exact_attn(c, s)
