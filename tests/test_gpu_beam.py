"""kd_beam_select against a plain fp64 selection.

Rows of random logits over odd and even vocabularies (one token to the largest),
every beam count, padded and unaligned rows; rows with NaN, infinities, the type's
lowest value, planted ties, all equal, all masked; dead and finished beams; groups
with fewer candidates than asked for.  Parents, tokens and end marks must be equal
(ties included); scores within their rounding to fp32 (2^-24 |s|) plus the row
sums' error: each exponential is good to 2^-22 + 2^-23 |x - m| relative, weighted by
itself, and a block's sum is rounded a few times: (4 + E|x - m|) 2^-22."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

LOWEST = float(np.finfo(np.float32).min)


def plain(x, W, scores, done, eos, n_out):
    """x [rows][V] fp32 -> per group [(s, w, v, tolerance)] of the n_out best, in order."""
    rows, V = x.shape
    out = []
    for g in range(rows // W):
        found = []
        for w in range(W):
            r = g * W + w
            sc = float(scores[r])
            if not sc > -np.inf:
                continue
            if done is not None and done[r]:
                found.append((-sc, w, 0.0, eos, 2.0 ** -24 * abs(sc)))
                continue
            row = x[r].astype(np.float64)
            row[np.isnan(row)] = -np.inf
            m = row.max()
            if m == -np.inf:
                continue
            with np.errstate(invalid="ignore"):
                d = np.where(row == m, 0.0, row - m)
            e = np.exp(d)
            tot = e.sum()
            fin = e > 0
            spread = float((e[fin] * np.abs(d[fin])).sum() / tot)
            cand = np.flatnonzero(row > -np.inf)
            order = cand[np.lexsort((cand, -row[cand]))][:n_out]
            for v in order:
                s = sc + d[v] - np.log(tot)
                if s > -np.inf:
                    found.append((-s, w, -row[v], int(v), 2.0 ** -24 * abs(s) + (4 + spread) * 2.0 ** -22))
        found.sort(key=lambda f: f[:4])
        out.append([(-f[0], f[1], f[3], f[4]) for f in found[:n_out]])
    return out


class Call:
    def __init__(self, kd, x, W, n_out, scores=None, done=None, eos=-1, pad=0, shift=0, want_done=True):
        rows, V = x.shape
        self.kd, self.W, self.V, self.n_out, self.eos, self.ld = kd, W, V, n_out, eos, V + pad
        buf = torch.full((rows * self.ld + shift,), float("nan"), device="cuda")
        self.x = buf[shift:].view(rows, self.ld)
        self.x[:, :V] = torch.from_numpy(x).cuda()
        self.G = rows // W
        self.scores = None if scores is None else torch.from_numpy(np.asarray(scores, np.float32)).cuda()
        self.done = None if done is None else torch.from_numpy(np.asarray(done, np.int32)).cuda()
        n = self.G * n_out
        self.out = [torch.full((n + 3,), -77, dtype=torch.int32, device="cuda") for _ in range(3)]
        self.sc = torch.full((n + 3,), -77.0, device="cuda")
        self.want_done = want_done
        self.ws = torch.full((kd.kd_beam_workspace_bytes(self.G, W, V, n_out),), 0xAB, dtype=torch.uint8, device="cuda")

    def enqueue(self, ws=None):
        self.kd.kd_beam_select(self.x, self.G, self.W, self.V, self.scores, self.n_out, self.out[0], self.out[1], self.sc,
                               self.ws if ws is None else ws, done=self.done,
                               done_out=self.out[2] if self.want_done else None, eos=self.eos, ld=self.ld)

    def run(self):
        self.enqueue()
        return self.read()

    def read(self):
        torch.cuda.synchronize()
        n = self.G * self.n_out
        for t in (*self.out, self.sc):
            assert (t[n:] == -77).all()  # nothing past the outputs
        return [t[:n].cpu().numpy().reshape(self.G, self.n_out) for t in (*self.out, self.sc)]


def check(got, ref, done, eos, W, n_out):
    par, tok, dn, sc = got
    for g, best in enumerate(ref):
        for j in range(n_out):
            if j < len(best):
                s, w, v, tol = best[j]
                assert (par[g, j], tok[g, j]) == (w, v), (g, j, best[j], sc[g, j])
                assert abs(float(sc[g, j]) - s) <= tol or sc[g, j] == s, (g, j, s, sc[g, j])
                assert dn[g, j] == int(v == eos or (done is not None and done[g * W + w] != 0))
            else:
                assert (par[g, j], tok[g, j], sc[g, j], dn[g, j]) == (-1, -1, -np.inf, 0), (g, j)


def go(kd, x, W, n_out, scores=None, done=None, eos=-1, **kw):
    got = Call(kd, x, W, n_out, scores, done, eos, **kw).run()
    ref = plain(x, W, np.zeros(len(x)) if scores is None else np.asarray(scores, np.float32), done, eos, n_out)
    check(got, ref, done, eos, W, n_out)
    return got


@pytest.mark.parametrize("G,W,V,n_out,pad,shift", [
    (1, 1, 1, 1, 0, 0), (1, 1, 5, 32, 0, 1), (1, 4, 512, 8, 0, 0), (2, 3, 1000, 7, 3, 2), (1, 16, 4096, 32, 0, 0),
    (3, 5, 4097, 10, 1, 3), (4, 2, 8191, 4, 0, 0), (1, 16, 32000, 32, 0, 0), (3, 16, 32003, 32, 8, 1),
    (40, 4, 12289, 4, 0, 0), (2, 8, 128256, 16, 0, 0), (1, 2, 524288, 32, 0, 0), (300, 1, 999, 2, 0, 0)])
def test_random_rows(kdlib, G, W, V, n_out, pad, shift):
    rng = np.random.default_rng(V + W)
    x = (rng.standard_normal((G * W, V)) * 2.5).astype(np.float32)
    go(kdlib, x, W, n_out, scores=-20 - 3 * rng.random(G * W), pad=pad, shift=shift)
    go(kdlib, x, W, n_out, pad=pad, shift=shift)  # no scores: zeros


def special_rows(V, rng):
    base = (rng.standard_normal((16, V)) * 3).astype(np.float32)
    i = rng.permutation(V)
    base[0, i[:V // 2]] = -np.inf                      # half masked
    base[1, :] = -np.inf                               # all masked
    base[2, i[:40]] = np.nan
    base[3, :] = np.nan
    base[4, :] = 0.0                                   # all equal
    base[5, :] = LOWEST                                # masked by the type's lowest value, all of it
    base[6, i[3:]] = LOWEST                            # ... all but three
    base[7, i[5]] = np.inf                             # one infinity
    base[8, i[:6]] = np.inf                            # several share the row
    base[9, :] = base[10, :]                           # the same row twice: ties between beams
    base[11, i[:100]] = 9.0                            # a hundred-way tie for the lead
    base[12, :] = np.where(np.arange(V) % 2, -0.0, 0.0)  # -0 equals +0
    base[13, :] = -np.inf
    base[13, i[:5]] = 1.0                              # five candidates
    base[14, :] = np.sort(base[14])[::-1]              # descending, then
    base[15, :] = np.sort(base[15])                    # ascending
    return base


@pytest.mark.parametrize("V", [257, 4095, 9000, 32003])
def test_special_rows_together_and_alone(kdlib, V):
    rng = np.random.default_rng(V)
    x = special_rows(V, rng)
    scores = np.zeros(16) - 5
    go(kdlib, x, 16, 32, scores=scores)
    for r in range(16):
        for n_out in (1, 8, 32):
            go(kdlib, x[r:r + 1], 1, n_out, scores=scores[:1])


def test_one_thread_holds_the_best(kdlib):
    """The leading logits 256 apart, and all-equal rows with whole subsets of a block masked (many ties at once)."""
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((2, 8192)) * 0.1).astype(np.float32)
    x[0, 7::256] = 10 + np.arange(32, dtype=np.float32)[::-1]
    x[1, :] = 1.5
    x[1].reshape(32, 256)[:, :8] = -np.inf
    for n_out in (1, 9, 32):
        go(kdlib, x, 2, n_out)
        go(kdlib, x, 1, n_out)


def test_dead_and_finished_beams(kdlib):
    rng = np.random.default_rng(3)
    G, W, V, n = 5, 4, 3001, 6
    x = (rng.standard_normal((G * W, V)) * 2).astype(np.float32)
    scores = (-4 * rng.random(G * W)).astype(np.float32)
    done = np.zeros(G * W, np.int32)
    scores[0:4] = [0, -np.inf, -np.inf, -np.inf]        # the start of a search
    scores[4:8] = -np.inf                               # a dead group
    scores[8:12], done[8:12] = [-3, -2, -2, -9], 1      # all finished: they stand, two tied
    scores[12:16], done[12:16] = [np.nan, -1, -np.inf, -40], [0, 1, 1, 0]
    done[17] = 1
    for r in np.flatnonzero(~(scores > -np.inf) | (done != 0)):
        x[r] = np.nan if r % 2 else 1e30                # never used
    got = go(kdlib, x, W, n, scores=scores, done=done, eos=2)
    assert got[0][1].tolist() == [-1] * n
    assert got[0][2].tolist() == [1, 2, 0, 3, -1, -1] and got[1][2].tolist() == [2, 2, 2, 2, -1, -1]
    go(kdlib, x, W, n, scores=scores, done=done, eos=V - 1)


def test_without_done_output(kdlib):
    rng = np.random.default_rng(4)
    x = rng.standard_normal((4, 600)).astype(np.float32)
    c = Call(kdlib, x, 2, 4, eos=5, want_done=False)
    par, tok, dn, sc = c.run()
    assert (dn == -77).all()
    ref = plain(x, 2, np.zeros(4), None, 5, 4)
    assert [[(b[1], b[2]) for b in g] for g in ref] == [[(int(a), int(b)) for a, b in zip(*r)] for r in zip(par, tok)]


def test_groups_do_not_depend_on_each_other(kdlib):
    rng = np.random.default_rng(9)
    x = (rng.standard_normal((24, 20000)) * 2.5).astype(np.float32)
    sc = -10 * rng.random(24)
    both = Call(kdlib, x, 4, 8, scores=sc).run()
    for g in (0, 3, 5):
        one = Call(kdlib, x[4 * g:4 * g + 4], 4, 8, scores=sc[4 * g:4 * g + 4]).run()
        for a, b in zip(one, both):
            assert np.array_equal(a[0], b[g])  # scores bit for bit


def test_captured_calls_share_a_workspace(kdlib):
    rng = np.random.default_rng(10)
    xs = [(rng.standard_normal((8, 33000)) * 2.5).astype(np.float32) for _ in range(2)]
    calls = [Call(kdlib, x, 4, 8, scores=-rng.random(8)) for x in xs]
    want = [c.run() for c in calls]
    s = torch.cuda.Stream()
    graphs = []
    for c in calls:
        for t in (*c.out, c.sc):
            t.fill_(-77)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            c.enqueue(calls[0].ws)
        graphs.append(g)
    with torch.cuda.stream(s):
        for _ in range(3):
            for g in graphs:
                g.replay()
    for c, w in zip(calls, want):
        for a, b in zip(c.read(), w):
            assert np.array_equal(a, b)


def test_results_match_bitwise_between_runs(kdlib):
    rng = np.random.default_rng(12)
    x = (rng.standard_normal((64, 50001)) * 2.5).astype(np.float32)
    c = Call(kdlib, x, 16, 32, scores=-rng.random(64))
    first = c.run()
    for _ in range(5):
        for a, b in zip(c.run(), first):
            assert np.array_equal(a, b)


@pytest.mark.parametrize("G,W,dead", [(152, 1, 0.5), (39, 4, 0.3), (64, 16, 0.9), (1024, 1, 0.2), (1025, 1, 0.2),
                                      (40, 8, 1.0), (40, 8, 0.0)])
def test_many_rows_of_which_some_offer_nothing(kdlib, G, W, dead):
    rng = np.random.default_rng(G + W)
    V, n = 4100, 5
    x = (rng.standard_normal((G * W, V)) * 2.5).astype(np.float32)
    scores = (-4 * rng.random(G * W)).astype(np.float32)
    gone, done = rng.random(G * W) < dead, np.zeros(G * W, np.int32)
    done[gone & (rng.random(G * W) < 0.5)] = 1
    scores[gone & (done == 0)] = [-np.inf, np.nan][G % 2]
    x[gone] = np.nan  # never used
    go(kdlib, x, W, n, scores=scores, done=done, eos=7)
    if dead in (0.0, 1.0):
        go(kdlib, np.where(np.isnan(x), 1, x).astype(np.float32), W, n)  # neither scores nor end marks


@pytest.mark.parametrize("shift", [0, 1, 2, 3])
@pytest.mark.parametrize("V", [32768, 32771, 36864, 36861, 45053, 70001])
def test_long_rows_off_every_boundary(kdlib, V, shift):
    """Rows whose starts lie 0 to 3 elements past a 16-byte boundary, against the same rows on one: bit for bit."""
    rng = np.random.default_rng(V)
    x = (rng.standard_normal((5, V)) * 2.5).astype(np.float32)
    x[:, 0], x[:, -1] = [9, -np.inf, 30, np.nan, 9], [9, 30, -9, 31, np.nan]  # both ends count
    sc = -3 * rng.random(5)
    got = go(kdlib, x, 5, 9, scores=sc, shift=shift, pad=1)  # rows of V + 1: every offset in turn
    want = Call(kdlib, x, 5, 9, scores=sc, pad=-V % 4).run()
    for a, b in zip(got, want):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("W,n_out", [(1, 5), (2, 10), (2, 8), (4, 16), (8, 32), (16, 32)])
def test_logits_closer_than_the_scores_last_bits(kdlib, W, n_out):
    """Two adjacent logits on either side of where x - max changes its rounding to fp32: with about 2% of these scores
    the pair sums of the two come out the other way round.  Whatever their sums, every place of the output is
    written, no candidate appears twice, and a beam's larger logit comes before its smaller one: in the merge by
    counting (up to four beams here) and in the tree's."""
    G, V, top = 1500, 300, 3
    lo = np.float32(2.0 ** -17)
    hi = np.nextafter(lo, np.float32(1))
    row = np.full(V, -np.inf, np.float32)
    row[[9, 120, 280]] = 250.0  # e^-250 of the others vanishes: the sum is 3
    row[30], row[31] = lo, hi
    x = np.tile(row, (G * W, 1))
    scores = np.repeat((-3000 * np.random.default_rng(5).random(G)).astype(np.float32), W)
    par, tok, dn, sc = Call(kdlib, x, W, n_out, scores=scores).run()
    order = {9: 0, 120: 1, 280: 2, 31: 3, 30: 4}
    for g in range(G):
        got = list(zip(par[g].tolist(), tok[g].tolist()))
        n = min(n_out, 5 * W)
        lead = [(w, t) for w in range(W) for t in (9, 120, 280)][:n]
        assert got[:len(lead)] == lead, (g, got)
        near = got[len(lead):n]
        assert len(set(near)) == len(near) and all(0 <= w < W and t in (30, 31) for w, t in near), (g, got)
        for w in range(W):
            mine = [order[t] for b, t in near if b == w]
            assert mine in ([], [3], [3, 4]), (g, got)
        assert got[n:] == [(-1, -1)] * (n_out - n)
        assert np.all(np.diff(sc[g][:n]) <= 0)
        s0 = np.float64(scores[g * W])
        for j in range(n):
            s = s0 + np.float64(row[got[j][1]]) - 250.0 - np.log(3.0)
            assert abs(float(sc[g, j]) - s) <= 2.0 ** -24 * abs(s) + 4 * 2.0 ** -22, (g, j)


@pytest.mark.parametrize("W,V,n_out", [(1, 131072, 16), (2, 131072, 9), (2, 131072, 16), (3, 131071, 12), (2, 200003, 16),
                                       (2, 65536, 16), (4, 131072, 10)])
def test_many_equals_in_many_segments(kdlib, W, V, n_out):
    """Rows of few values: more than 64 keys of a row's segments are left after the bound, with 9 to 16 outputs."""
    rng = np.random.default_rng(V + n_out)
    go(kdlib, np.zeros((W, V), np.float32), W, n_out)
    x = rng.integers(0, 3, (W, V)).astype(np.float32)
    go(kdlib, x, W, n_out, scores=-rng.random(W))
    x[0] = np.arange(V)[::-1] // 5000  # the first segment holds them all
    x[-1, : V // 2] = -np.inf
    go(kdlib, x, W, n_out)
