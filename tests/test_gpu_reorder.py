"""kd_kv_reorder and the sessions' reorder and fork: bytes moved exactly, in place.

Random maps (permutations, cycles of every length, parents taken many times,
unmoved slots, sources outside the destinations), ragged lengths, windows, fp16
and Q8_0 planes, odd row sizes; every byte of every plane compared with a copy
made on the host.  Model level: a forked or reordered session's steps give the
bits of a session that was loaded with the same rows."""
import re
import textwrap
from pathlib import Path

import numpy as np
import pytest

import synth

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def kept(n, window, sinks):
    t = np.arange(n)
    return t if not window else t[(t < sinks) | (t > n - window)]


def run(kd, rng, L, S, nkv, cap, widths, dst, src, lens, window=0, sinks=0, stream=None):
    host = [rng.integers(0, 256, (L, S, nkv, cap, w), dtype=np.uint8) for w in widths]
    dev = [torch.from_numpy(h).cuda() for h in host]
    want = [h.copy() for h in host]
    for d, s, n in zip(dst, src, lens):
        t = kept(n, window, sinks)
        for w, h in zip(want, host):
            w[:, d][:, :, t] = h[:, s][:, :, t]
    kd.kd_kv_reorder(dev, dst, src, lens, L, S, nkv, cap, window=window, sinks=sinks, stream=stream)
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(dev, want)):
        assert np.array_equal(a.cpu().numpy(), b), (i, list(dst), list(src), list(lens), window, sinks)


@pytest.mark.parametrize("k", [1, 2, 3, 7, 8, 9, 16, 17, 40, 64])
def test_cycles(kdlib, k):
    """One cycle of every batch-straddling length, with moves hanging off it where room is left."""
    rng = np.random.default_rng(k)
    S = 70
    slots = rng.permutation(S)
    dst = slots[:k].copy()
    src = np.roll(dst, 1) if k > 1 else slots[1:2]
    extra = min(64 - k, 5)
    dst = np.concatenate([dst, slots[k + 1:k + 1 + extra]])
    src = np.concatenate([src, rng.choice(slots[:k], extra)])
    order = rng.permutation(len(dst))
    run(kdlib, rng, 2, S, 2, 9, (32, 8), dst[order], src[order], np.full(len(dst), 9))


def connected_sets(rng, S, sets):
    """Moves of connected sets over distinct slots, in any order: (cycle, more) is a cycle of that many slots (0: one
    slot that nothing writes), then `more` slots that each continue one of the set's earlier."""
    free, dst, src = list(rng.permutation(S)), [], []
    for cycle, more in sets:
        nodes = [free.pop() for _ in range(max(cycle, 1))]
        if cycle:
            dst += nodes
            src += nodes[1:] + nodes[:1]
        for _ in range(more):
            nodes.append(free.pop())
            dst.append(nodes[-1])
            src.append(nodes[rng.integers(len(nodes) - 1)])
    order = rng.permutation(len(dst))
    return np.array(dst)[order], np.array(src)[order]


# Calls of more than 32 MB take sets four moves at a time, smaller ones eight.
@pytest.mark.parametrize("sets", [((0, 5), (0, 9)), ((5, 0), (9, 0)), ((5, 3), (2, 4)), ((9, 5),), ((0, 16),), ((6, 1), (0, 6)),
                                  ((0, 17), (9, 8), (5, 0)), ((17, 4), (0, 8), (3, 2)), ((40, 8),)])
@pytest.mark.parametrize("ragged,window", [(False, 0), (True, 0), (True, 1400)])
def test_large_calls_with_sets_of_many_moves(kdlib, sets, ragged, window):
    rng = np.random.default_rng(sum(map(sum, sets)) + window)
    S = sum(max(c, 1) + m for c, m in sets) + 2
    dst, src = connected_sets(rng, S, sets)
    widths, nkv = (256, 8, 128), 3
    cap = 1999 if len(dst) <= 16 else 1601
    at = rng.integers(cap * 3 // 4, cap + 1, S) if ragged else np.full(S, cap)
    lens, sinks = at[src], 33
    row = sum(widths) * nkv * sum(len(kept(int(n), window, sinks)) for n in lens)
    L = (32 << 20) // row + 1
    run(kdlib, rng, L, S, nkv, cap, widths, dst, src, lens, window, sinks)


@pytest.mark.parametrize("seed", range(30))
def test_random_maps(kdlib, seed):
    rng = np.random.default_rng(100 + seed)
    S = int(rng.integers(1, 40))
    n = int(rng.integers(1, S + 1))
    cap = int(rng.integers(1, 150))
    dst = rng.permutation(S)[:n]
    src = rng.choice(S, n) if seed % 3 else rng.permutation(dst)
    at = rng.integers(0, cap + 1, S)  # a length per slot, as sessions have
    lens = at[src] if seed % 2 else rng.integers(0, cap + 1, n)
    window = int(rng.choice([0, 1, 2, 5, 64, 1000]))
    widths = [(256, 256), (128, 8, 128, 8), (128, 128), (24,), (1024, 136, 16)][seed % 5]
    run(kdlib, rng, int(rng.integers(1, 4)), S, int(rng.integers(1, 4)), cap, widths, dst, src, lens, window,
        int(rng.choice([0, 1, 4, 200])))


def test_nothing_to_move(kdlib):
    rng = np.random.default_rng(0)
    run(kdlib, rng, 1, 4, 1, 8, (16,), [0, 2], [0, 2], [8, 3])
    run(kdlib, rng, 1, 4, 1, 8, (16,), [0, 2], [1, 3], [0, 0])
    run(kdlib, rng, 1, 4, 1, 8, (16,), [0], [1], [5], window=1)  # a window of one keeps nothing of the past


def test_many_layers_and_heads(kdlib):
    run(kdlib, np.random.default_rng(1), 40, 3, 9, 17, (64, 8), [0, 1, 2], [1, 2, 0], [17, 17, 17])


def test_offsets_past_32_bits(kdlib):
    """A plane of more than 2^32 bytes: the last slot of every layer swaps with the first."""
    kd = kdlib
    L, S, nkv, cap, w = 5, 5, 4, 65536, 1024
    t = torch.zeros(L, S, nkv, cap, w // 4, dtype=torch.int32, device="cuda")
    assert t.numel() * 4 > 2 ** 32
    t[:, 4] = torch.arange(cap, device="cuda", dtype=torch.int32)[None, None, :, None] + 1
    kd.kd_kv_reorder([t], [0, 4], [4, 0], [cap, cap], L, S, nkv, cap)
    torch.cuda.synchronize()
    col = torch.arange(cap, device="cuda", dtype=torch.int32)[:, None] + 1
    assert (t[:, 0] == col).all() and (t[:, 4] == 0).all() and (t[:, 1:4] == 0).all()


def test_captured_reorder_on_a_side_stream(kdlib):
    """A captured rotation of three slots, replayed three times, is the identity; replayed once more it is not."""
    kd = kdlib
    t = torch.randn(2, 4, 2, 50, 64, device="cuda", dtype=torch.float16)
    base = t.clone()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        kd.kd_kv_reorder([t], [0, 1, 2], [1, 2, 0], [50, 50, 50], 2, 4, 2, 50)
    with torch.cuda.stream(s):
        for _ in range(3):
            g.replay()
        s.synchronize()
        assert torch.equal(t, base)
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(t[:, 0], base[:, 1]) and torch.equal(t[:, 2], base[:, 0]) and torch.equal(t[:, 3], base[:, 3])


# ---------------------------------------------------------------------- sessions ---
SHAPES = {"hd64": (synth.TINY, 0), "q8": (synth.TINY_HD128, 128)}


@pytest.fixture(params=list(SHAPES))
def model(request, kdlib):
    kd = kdlib
    shape, flags = SHAPES[request.param]
    w = synth.model_weights(shape, 0)
    made = []

    def load(sessions=6, cap=256):
        m = kd.kd_model_load(kd.make_config(shape, sessions, cap, flags), w)
        made.append(m)
        return m
    yield kd, shape, load
    for m in made:
        kd.kd_model_free(m)


def fill(kd, m, shape, i, n):
    sid = kd.kd_session_bind(m)
    kd.kd_session_load_kv(m, sid, *synth.kv_prefill(shape, 0, i, n), n)
    return sid


def step(kd, m, shape, ids, tok, pos):
    lg = torch.empty(len(ids), shape.vocab, device="cuda")
    kd.kd_decode_step(m, ids, tok, pos, lg, None)
    torch.cuda.synchronize()
    return lg.cpu().numpy()


def refused(kd, m, shape, sid, pos):
    """True if the step is refused (for its position)."""
    try:
        step(kd, m, shape, [sid], [3], [pos])
    except kd.KdError as e:
        assert e.name == "KD_ERR_POSITION"
        return True
    return False


@pytest.mark.parametrize("window", [0, 50])
def test_sessions_reorder_and_fork(model, window):
    kd, shape, load = model
    lens = [90, 33, 120, 7]
    m = load()
    kd.kd_model_set_window(m, window, 4)
    ids = [fill(kd, m, shape, i, n) for i, n in enumerate(lens)]
    kd.kd_session_reorder(m, ids, [ids[2], ids[0], ids[1], ids[3]])  # a cycle of three, one unmoved
    of = [2, 0, 1, 3]
    assert [kd.kd_session_length(m, i) for i in ids] == [lens[p] for p in of]
    kd.kd_session_reorder(m, ids, [ids[0], ids[0], -1, ids[0]])  # one parent taken three times, one left alone
    of = [2, 2, 1, 2]
    fork = kd.kd_session_fork(m, ids[2])
    ids, of = ids + [fork], of + [1]
    assert [kd.kd_session_length(m, i) for i in ids] == [lens[p] for p in of]
    ref = load()
    kd.kd_model_set_window(ref, window, 4)
    rid = [fill(kd, ref, shape, p, lens[p]) for p in of]
    for t in range(3):
        tok = synth.tokens(t, "re", len(ids), shape.vocab)
        pos = [lens[p] + t for p in of]
        a, b = step(kd, m, shape, ids, tok, pos), step(kd, ref, shape, rid, tok, pos)
        assert np.array_equal(a, b), t
    assert kd.kd_device_status(m) == 0


def test_reorder_errors_change_nothing(model):
    kd, shape, load = model
    m = load(sessions=2)
    a, b = fill(kd, m, shape, 0, 20), fill(kd, m, shape, 1, 30)
    for ids, parents, name in (([a, 5], [b, a], "KD_ERR_BAD_SESSION"), ([a, a], [b, b], "KD_ERR_BAD_SESSION"),
                               ([a], [7], "KD_ERR_BAD_SESSION"), ([a], [-2], "KD_ERR_BAD_SESSION"),
                               ([], [], "KD_ERR_BATCH"), (list(range(65)), [0] * 65, "KD_ERR_BATCH")):
        with pytest.raises(kd.KdError) as e:
            kd.kd_session_reorder(m, ids, parents)
        assert e.value.name == name
    with pytest.raises(kd.KdError) as e:
        kd.kd_session_fork(m, a)
    assert e.value.name == "KD_ERR_NO_FREE_SLOT"
    assert [kd.kd_session_length(m, i) for i in (a, b)] == [20, 30]
    with pytest.raises(kd.KdError):
        kd.kd_model_set_window(m, -1, 0)


def test_rows_left_behind_are_refused(model):
    """Under a window a copy holds the sinks and the last window - 1 rows; a step that would attend another row
    of it is refused, and the session itself keeps everything."""
    kd, shape, load = model
    m = load()
    kd.kd_model_set_window(m, 20, 4)
    a = fill(kd, m, shape, 0, 100)
    f = kd.kd_session_fork(m, a)                      # rows 4..80 stay behind
    g = kd.kd_session_fork(m, f)
    for sid, pos in ((f, 99), (g, 99), (f, 50), (f, 5)):
        assert refused(kd, m, shape, sid, pos), pos
    assert kd.kd_session_length(m, f) == 100          # a refused step changed nothing
    assert not refused(kd, m, shape, a, 99)
    one = step(kd, m, shape, [f, g], [9, 9], [100, 100])
    assert np.array_equal(one[0], one[1])
    kd.kd_model_set_window(m, 22, 4)                  # wider: position 101 attends row 80
    assert refused(kd, m, shape, f, 101)
    kd.kd_model_set_window(m, 21, 4)                  # row 81 on: all there
    assert not refused(kd, m, shape, f, 101)
    kd.kd_model_set_window(m, 20, 5)                  # one more sink than was kept
    assert refused(kd, m, shape, f, 102)
    kd.kd_model_set_window(m, 0)
    assert refused(kd, m, shape, f, 102)
    assert not refused(kd, m, shape, a, 100)          # the original never lost a row
    kd.kd_model_set_window(m, 20, 4)
    assert not refused(kd, m, shape, f, 2)            # rewound in front of the gap: rows 0..1 only, whole again
    kd.kd_model_set_window(m, 0)
    assert not refused(kd, m, shape, f, 3)
    kd.kd_session_load_kv(m, g, *synth.kv_prefill(shape, 0, 1, 60), 60)
    assert not refused(kd, m, shape, g, 60)           # reloaded: whole


@pytest.mark.parametrize("window", [0, 24])
def test_beam_search_equals_replayed_hypotheses(model, window):
    """Six steps of beam search (decode step, selection, reorder) for two prompts of three beams.  At every
    step each hypothesis, replayed token by token in a session of its own, has the same logits bit for bit, and
    a selection made on the host from those logits picks the same beams, tokens and scores."""
    kd, shape, load = model
    prompts, W, V, eos, n = (70, 41), 3, shape.vocab, 17, 3
    G = len(prompts)
    m, ref = load(sessions=G * W), load(sessions=1)
    for x in (m, ref):
        kd.kd_model_set_window(x, window, 4)
    ids = [fill(kd, m, shape, g, prompts[g]) for g in range(G) for _ in range(W)]
    first = synth.tokens(1, "beam", G, V)
    hyps = [[int(first[g])] for g in range(G) for _ in range(W)]
    scores = torch.tensor([0.0 if w == 0 else -np.inf for _ in range(G) for w in range(W)], device="cuda")
    done = torch.zeros(G * W, dtype=torch.int32, device="cuda")
    par, tok, dn = (torch.empty(G, n, dtype=torch.int32, device="cuda") for _ in range(3))
    out = torch.empty(G, n, device="cuda")
    ws = torch.empty(kd.kd_beam_workspace_bytes(G, W, V, n), dtype=torch.uint8, device="cuda")
    logits = torch.empty(G * W, V, device="cuda")
    for t in range(6):
        pos = [prompts[r // W] + t for r in range(G * W)]
        kd.kd_decode_step(m, ids, [h[-1] for h in hyps], pos, logits, None)
        kd.kd_beam_select(logits, G, W, V, scores, n, par, tok, out, ws, done=done, done_out=dn, eos=eos)
        lg, old, od = logits.cpu().numpy(), scores.cpu().numpy().astype(np.float64), done.cpu().numpy()
        for r in range(G * W):  # the hypothesis from scratch
            sid = fill(kd, ref, shape, r // W, prompts[r // W])
            for j, token in enumerate(hyps[r]):
                one = step(kd, ref, shape, [sid], [token], [prompts[r // W] + j])
            kd.kd_session_free(ref, sid)
            assert np.array_equal(one[0], lg[r]), (t, r)
        new = []
        for g in range(G):
            cand = []
            for w in range(W):
                r = g * W + w
                if not old[r] > -np.inf:
                    continue
                if od[r]:
                    cand.append((-old[r], w, eos))
                    continue
                x = lg[r].astype(np.float64)
                s = old[r] + x - x.max() - np.log(np.exp(x - x.max()).sum())
                cand += [(-s[v], w, v) for v in range(V)]
            cand.sort()
            for j, (s, w, v) in enumerate(cand[:n]):
                assert (int(par[g, j]), int(tok[g, j])) == (w, v), (t, g, j)
                assert abs(float(out[g, j]) + s) <= 2.0 ** -24 * abs(s) + 20 * 2.0 ** -22
                assert int(dn[g, j]) == int(v == eos or od[g * W + w] != 0)
                new.append(hyps[g * W + w] + [int(v)])
        kd.kd_session_reorder(m, ids, [ids[g * W + int(par[g, j])] for g in range(G) for j in range(n)])
        hyps = new
        scores, done = out.flatten().clone(), dn.flatten().clone()
    assert len({(r // W, *h) for r, h in enumerate(hyps)}) == G * W  # the beams stay apart
    assert kd.kd_device_status(m) == 0


@pytest.mark.parametrize("groups,beams", [(3, 4), (10, 8)])
def test_the_readme_search_loop(model, groups, beams):
    """README's search step as it stands there, run three times, for up to 80 sessions.  Prompt 0 and prompt 1 have
    fewer candidates than beams in the first step, prompt 2 none at all in the second.  Every hypothesis that is
    left goes on with the logits of a session that was fed its tokens one by one."""
    kd, shape, load = model
    readme = (Path(__file__).resolve().parent.parent / "README.md").read_text()
    block, = [b for b in re.findall(r"```python\n(.*?)```", readme, re.S) if "kd_beam_select" in b]
    code = compile(textwrap.dedent(block), "README.md", "exec")
    V, n = shape.vocab, groups * beams
    prompts = [20 + 7 * g % 50 for g in range(groups)]
    m, ref = load(sessions=n), load(sessions=n)
    bound = [kd.kd_session_bind(m) for _ in range(n)]
    ids = np.random.default_rng(3).permutation(bound).astype(np.int32)
    rid = [kd.kd_session_bind(ref) for _ in range(n)]
    for r in range(n):
        rows = synth.kv_prefill(shape, 0, r // beams, prompts[r // beams])
        for x, sid in ((m, int(ids[r])), (ref, rid[r])):
            kd.kd_session_load_kv(x, sid, *rows, prompts[r // beams])
    t = 0
    allowed = {(0, 0): 3, (0, 1): 2, (1, 2): 0}  # (step, prompt): tokens that a grammar leaves

    class Masked:
        def __getattr__(self, name):
            return getattr(kd, name)

        def kd_decode_step(self, m, ids, tokens, positions, logits, argmax):
            kd.kd_decode_step(m, ids, tokens, positions, logits, argmax)
            for (step_, g), k in allowed.items():
                if step_ == t:
                    logits[g * beams:(g + 1) * beams, k:] = -np.inf

    first = np.repeat(synth.tokens(1, "loop", groups, V), beams)
    ns = dict(kd=Masked(), np=np, m=m, ids=ids, groups=groups, beams=beams, V=V, tokens=first,
              positions=np.repeat(np.array(prompts, np.int32), beams), logits=torch.empty(n, V, device="cuda"),
              scores=torch.tensor([0.0 if r % beams == 0 else -np.inf for r in range(n)], device="cuda"),
              parents=torch.empty(groups, beams, dtype=torch.int32, device="cuda"),
              new_tokens=torch.empty(groups, beams, dtype=torch.int32, device="cuda"),
              new_scores=torch.empty(groups, beams, device="cuda"),
              workspace=torch.empty(kd.kd_beam_workspace_bytes(groups, beams, V, beams), dtype=torch.uint8, device="cuda"))
    hyps = [[int(x)] for x in first]
    for t in range(3):
        exec(code, ns)
        par, tok = ns["parents"].cpu().numpy(), ns["new_tokens"].cpu().numpy()
        hyps = [hyps[r // beams * beams + par[r // beams, r % beams]] + [int(tok[r // beams, r % beams])]
                if par[r // beams, r % beams] >= 0 else None for r in range(n)]
        if t == 0:
            assert [sum(h is not None for h in hyps[g * beams:(g + 1) * beams]) for g in range(3)] == [3, 2, beams]
    live = [r for r in range(n) if hyps[r] is not None]
    assert len(live) == n - beams and not set(live) & set(range(2 * beams, 3 * beams))
    t = -1
    got = torch.empty(n, V, device="cuda")
    kd.kd_decode_step(m, ids, ns["tokens"], ns["positions"], got, None)
    want = torch.empty(n, V, device="cuda")
    for j in range(4):
        kd.kd_decode_step(ref, rid, [h[j] if h else 0 for h in hyps], [prompts[r // beams] + j for r in range(n)], want, None)
    assert np.array_equal(ns["positions"], [prompts[r // beams] + 3 for r in range(n)])
    assert torch.equal(got[live], want[live])
    assert torch.isfinite(ns["scores"].view(-1)[live]).all()
    assert kd.kd_device_status(m) == 0
