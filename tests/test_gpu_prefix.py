"""Attention of sequences that share a prefix, on the GPU: cases of exact arithmetic (verify_exact.py) that show a single cell lost,
repeated or stale, ordinary values within the roundings, empty and uneven groups, reports, streams and graphs."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import dflash_block_drafter_gb300 as D  # noqa: E402
import gpu_helpers as H  # noqa: E402
import verify_exact as E  # noqa: E402
import verify_ref as V  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
LN2 = float(np.log(2))


@pytest.fixture(scope="module", autouse=True)
def R():
    H.need_gpu()
    H.build_lib()
    from dflash_block_drafter_gb300 import runtime
    return runtime


def ints(x):
    return torch.as_tensor(np.asarray(x, np.int32), device="cuda")


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


class Case:
    """groups: [(prefix cells, [(own cells, rows), ..]), ..].  Unused cells are NaN, unused table entries beyond the cache, and there are
    two rows behind the last sequence."""

    def __init__(self, R, seed, d, heads, G, groups, page, exact, kind="fp16", gain=1.0, spare=1):
        rng = np.random.default_rng(seed)
        self.d, self.heads, self.G, self.kind = d, heads, G, kind
        self.prefix = [p for p, _ in groups]
        self.own = [n for _, s in groups for n, _ in s]
        self.rows = [r for _, s in groups for _, r in s]
        self.of = [g for g, (_, s) in enumerate(groups) for _ in s]
        self.group_offsets = np.cumsum([0] + [len(s) for _, s in groups])
        self.offsets = np.cumsum([0] + self.rows)
        cells = [max(n, 0) for n in self.prefix + self.own]
        counts = [-(-n // page) for n in cells]
        order = rng.permutation(sum(counts) + 2)
        self.cache = R.kv4_cache(len(order), page, heads, d)
        self.cache.fill_(0xFF)
        self.tables, self.parts, at = [], [], 0
        for part in (counts[: len(groups)], counts[len(groups):]):
            table = np.full((len(part), max(part + [0]) + spare), 1 << 30, np.int32)
            for s, n in enumerate(part):
                table[s, :n] = order[at: at + n]
                at += n
                m = cells[len(self.parts)]
                k, v = E.cells(rng, m, heads, d) if exact else rng.standard_normal((2, m, heads, d))
                if m:
                    pos = np.arange(m)
                    slots = ints(table[s, pos // page] * page + pos % page)
                    R.kv4_write(self.cache, *(torch.as_tensor(x, device="cuda").half() for x in (k, v)), slots)
                    if not exact:
                        k, v = (x.double().cpu().numpy() for x in R.kv4_read(self.cache, slots))
                self.parts.append((k, v))
            self.tables.append(table)
        self.tokens = int(self.offsets[-1])
        q = E.queries(rng, self.tokens, heads * G, d) if exact else gain * rng.standard_normal((self.tokens, heads * G, d))
        self.q = torch.zeros((self.tokens + 2, heads * G, d), dtype=TYPES[kind], device="cuda")
        self.q[: self.tokens] = torch.as_tensor(q, device="cuda").to(TYPES[kind])
        self.q[self.tokens:] = float("nan")  # rows of no sequence are not read

    def args(self):
        return (self.cache, self.q, ints(self.tables[0]), ints(self.prefix), ints(self.group_offsets), ints(self.tables[1]), ints(self.own),
                ints(self.offsets), max(self.rows + [1]))

    def reference(self, causal, scale):
        """(o, spread, largest score, cells seen) in 64 bits."""
        q = self.q[: self.tokens].double().cpu().numpy()
        o, spread, top, seen = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
        for s, r in enumerate(self.rows):
            (pk, pv), (ok, ov) = self.parts[self.of[s]], self.parts[len(self.prefix) + s]
            k, v = np.concatenate([pk, ok]).astype(float), np.concatenate([pv, ov]).astype(float)
            n = len(ok)
            last = np.arange(n - r, n) if causal else np.full(r, n - 1)
            sees = np.concatenate([np.ones((r, len(pk)), bool), np.arange(n) <= last[:, None]], 1)
            if k.shape[0] == 0 or r == 0:
                continue
            mine = slice(self.offsets[s], self.offsets[s + 1])
            for h in range(self.heads):
                hs = slice(h * self.G, (h + 1) * self.G)
                x = np.where(sees[:, None], scale * np.einsum("rgd,nd->rgn", q[mine, hs], k[:, h]), -np.inf)
                m = x.max(-1, keepdims=True)
                p = np.exp(x - np.where(m > -np.inf, m, 0))
                total = np.maximum(p.sum(-1, keepdims=True), 1e-300)
                o[mine, hs], spread[mine, hs] = p @ v[:, h] / total, p @ np.abs(v[:, h]) / total
                top[mine, hs] = np.max(np.abs(np.where(sees[:, None], x, 0)), -1)
                seen[mine, hs] = sees.sum(-1)[:, None]
        return o, spread, top, seen

    def run(self, R, causal=True, scale=None, st=None, **kw):
        out = torch.full_like(self.q, 7.0)
        size = D.dflash_kv4_prefix_attention_workspace(R._kv4(self.cache), self.q.shape[0], self.heads * self.G, len(self.prefix),
                                                       self.tables[0].shape[1], len(self.own), max(self.rows + [1]), self.tables[1].shape[1])
        workspace = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")  # stale pieces would be NaN
        R.kv4_prefix_attention(*self.args(), causal=causal, scale=scale, out=out, workspace=workspace, status=st, **kw)
        assert bool((out[self.tokens:] == 7.0).all())  # rows of no sequence
        return out[: self.tokens]

    def check_exact(self, R, causal):
        st = status()
        got = self.run(R, causal, LN2, st).double().cpu().numpy()
        assert int(st) == 0
        o, spread, _, _ = self.reference(causal, LN2)
        worst = np.max(np.abs(got - o) / E.tolerance(o, spread, 2.0 ** -11))
        assert worst <= 1, worst

    def check(self, R, causal=True, scale=None, got=None):
        st = status()
        if got is None:
            got = self.run(R, causal, scale, st)
        assert int(st) == 0
        o, spread, top, seen = self.reference(causal, self.d ** -0.5 if scale is None else scale)
        # V and P to FP16: 2^-11 each; over the prefix K too: 2^-11 of each of a score's terms, at random, so that the score is off by 2^-11 of
        # the root of their squares, which the largest score of hundreds is not below; scores in FP32: 2^-16 of the largest, twice; P below
        # FP16's range: 2^-25 of the largest |v| a cell; the output's rounding
        eps = torch.finfo(TYPES[self.kind]).eps / 2
        tol = spread * (2.0 ** -10 + (2.0 ** -10 + 2.0 ** -16) * (1 + top)[..., None]) + seen[..., None] * 2.0 ** -25 * 8.0 * spread.max() \
            + eps * np.abs(o) + 1e-7
        err = np.abs(got.double().cpu().numpy() - o)
        assert np.all(err <= tol), f"worst {np.max(err / tol):.2f} x tolerance"


def uneven(rng, n, own, rows):
    return [(int(rng.integers(rows, own)), rows) for _ in range(n)]


@pytest.mark.parametrize("d,heads,G,rows", [(64, 2, 5, 8), (128, 1, 9, 8), (256, 2, 12, 8), (64, 2, 3, 8), (128, 2, 4, 8), (128, 4, 4, 1), (256, 2, 12, 1),
                                            (64, 1, 16, 1), (128, 1, 128, 1), (64, 1, 43, 2)])
@pytest.mark.parametrize("shape", ["long", "many"])
@pytest.mark.parametrize("causal", [True, False])
def test_every_cell_once(R, d, heads, G, rows, shape, causal):
    """Long prefixes over few sequences, many sequences over short ones: a single lost, repeated or stale tile shows."""
    rng = np.random.default_rng(d + G + rows)
    if shape == "long":
        groups = [(12000, uneven(rng, 5, 900, rows)), (77, uneven(rng, 1, 6000, rows)), (5001, uneven(rng, 14, 50, rows))]
    else:
        groups = [(int(rng.integers(1, 700)), uneven(rng, int(rng.integers(1, 20)), 200, rows)) for _ in range(12)]
    Case(R, d, d, heads, G, groups, 64, True).check_exact(R, causal)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("G,page", [(1, 16), (5, 32), (12, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_small_and_empty(R, d, kind, G, page, causal):
    """Prefixes of no cell, one, and ends inside a page and a tile; sequences without rows, without cells, with fewer cells than rows; a
    group without sequences, one without rows."""
    groups = [(1, [(1, 1)]), (0, [(5, 3), (64, 8), (17, 1)]), (33, []), (16, [(4, 0)]), (-4, [(0, 2), (2, 2)]), (65, [(0, 1), (0, 8), (3, 8), (200, 5)]),
              (130, [(1, 1)] * 9), (15, [(-2, 3)])]
    Case(R, d + G, d, 2, G, groups, page, False, kind).check(R, causal)


@pytest.mark.parametrize("d,heads,G,rows", [(64, 1, 16, 1), (128, 2, 4, 8), (256, 2, 12, 4)])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("gain", [0.01, 1.0, 6.0])
def test_ordinary_values(R, d, heads, G, rows, kind, gain):
    rng = np.random.default_rng(G)
    Case(R, 3 * d, d, heads, G, [(1500, uneven(rng, 6, 300, rows)), (401, uneven(rng, 3, 900, rows))], 32, False, kind, gain).check(R)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G,rows", [(4, 1), (5, 8)])
def test_one_side_outweighs_the_other(R, d, G, rows):
    """Scores so far apart that the prefix, or the own cells, have no weight at all beside the other."""
    c = Case(R, d, d, 1, G, [(300, [(40, rows)] * 3)], 16, False, "bf16", 1.0)
    for side in (0, 1):
        e = Case(R, d, d, 1, G, [(300, [(40, rows)] * 3)], 16, False, "bf16", 1.0)
        q = e.q[: e.tokens].double().cpu().numpy()
        far = 40 * q[0, 0] / np.linalg.norm(q[0, 0])  # all rows ask the same; one side's keys answer
        e.q[: e.tokens] = torch.as_tensor(far, device="cuda").to(e.q.dtype)
        for i, (k, v) in enumerate(e.parts):
            if (i == 0) == (side == 0):
                k = np.broadcast_to(far, k.shape).copy()
                table = e.tables[0][0] if i == 0 else e.tables[1][i - 1]
                pos = np.arange(len(k))
                slots = ints(table[pos // 16] * 16 + pos % 16)
                R.kv4_write(e.cache, torch.as_tensor(k, device="cuda").half(), torch.as_tensor(v, device="cuda").half(), slots)
                e.parts[i] = tuple(x.double().cpu().numpy() for x in R.kv4_read(e.cache, slots))
        e.check(R, causal=False)
    c.check(R)


@pytest.mark.parametrize("d,G,rows", [(64, 4, 1), (128, 5, 8), (256, 12, 8)])
def test_as_without_sharing(R, d, G, rows):
    """The same cells through tables that hold the prefix's pages before the own ones, where the prefix ends with a page."""
    rng = np.random.default_rng(d)
    c = Case(R, d, d, 2, G, [(640, uneven(rng, 7, 300, rows))], 64, False, "bf16")
    got = c.run(R)
    table = np.concatenate([np.repeat(c.tables[0][:, :10], 7, 0), c.tables[1]], 1)
    want = R.kv4_attention(c.cache, c.q, ints(table), ints(np.array(c.own) + 640), ints(c.offsets), rows)[: c.tokens]
    _, spread, top, _ = c.reference(True, d ** -0.5)
    tol = 2 * (spread * (2.0 ** -10 + 2.0 ** -10 * (1 + top)[..., None]) + 2.0 ** -8 * spread)
    assert np.all(np.abs((got.double() - want.double()).cpu().numpy()) <= tol)


@pytest.mark.parametrize("d,G,rows", [(64, 5, 8), (128, 4, 1), (256, 12, 8)])
def test_same_result_again(R, d, G, rows):
    rng = np.random.default_rng(d)
    c = Case(R, d, d, 2, G, [(3000, uneven(rng, 9, 400, rows)), (900, uneven(rng, 4, 400, rows))], 64, False)
    first = c.run(R)
    for _ in range(30):
        assert torch.equal(c.run(R), first)


def test_strided_rows(R):
    """Queries and outputs as parts of wider rows."""
    c = Case(R, 1, 128, 2, 4, [(200, [(30, 2), (9, 3)])], 16, False, "bf16")
    want = c.run(R)
    wide = torch.full((c.tokens + 2, 2, 12, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 0, 2:10] = c.q
    st = status()
    args = list(c.args())
    args[1] = wide[:, 0, 2:10]
    R.kv4_prefix_attention(*args, out=wide[:, 1, 2:10], status=st)
    assert int(st) == 0 and torch.equal(wide[: c.tokens, 1, 2:10], want)
    assert bool((wide[:, 1, :2] == 3).all()) and bool((wide[:, 1, 10:] == 3).all()) and bool((wide[c.tokens:, 1] == 3).all())


@pytest.mark.parametrize("G", [4, 9])
def test_reports(R, G):
    groups = [(100, [(20, 2), (5, 1)]), (40, [(9, 4)])]
    good = Case(R, 1, 64, 2, G, groups, 16, False)
    want = good.run(R)

    def report(rows=slice(0, 0), **kw):
        c = Case(R, 1, 64, 2, G, groups, 16, False)
        for name, (at, value) in kw.items():
            t = getattr(c, name) if name != "prefix_table" else c.tables[0]
            t[at] = value
        st = status()
        got = c.run(R, st=st)
        assert torch.equal(got[rows], want[rows])  # what has nothing to do with it
        return int(st)

    assert report(slice(None)) == 0
    # (the rows of a group that is refused, and of none, are unspecified: they join what the workspace held, here NaN, which is reported too)
    assert report(group_offsets=(1, 4)) & D.DFLASH_DEV_BAD_BLOCK
    assert report(group_offsets=(1, -1)) & D.DFLASH_DEV_BAD_BLOCK
    assert report(slice(0, 3), group_offsets=(2, 2)) & D.DFLASH_DEV_BAD_BLOCK  # a sequence of no group
    assert report(slice(3, 7), group_offsets=(0, 1)) & D.DFLASH_DEV_BAD_BLOCK
    assert report(slice(7, 7), offsets=(2, 30)) & D.DFLASH_DEV_BAD_BLOCK
    assert report(slice(0, 2), offsets=(3, 30)) & D.DFLASH_DEV_BAD_BLOCK
    assert report(slice(0, 3), prefix=(1, 10000)) & D.DFLASH_DEV_CAPACITY  # (its cells behind the table's pages are NaN or elsewhere)
    # a sequence of more rows than the call allows: what is not of it stays
    many = Case(R, 1, 64, 2, G, [(100, [(20, 8), (30, 8)]), (2000, uneven(np.random.default_rng(3), 9, 90, 2))], 16, False)
    first, st = many.run(R), status()
    args = list(many.args())
    args[8] = 2
    got = R.kv4_prefix_attention(*args, status=st)
    assert int(st) & D.DFLASH_DEV_BAD_BLOCK
    late = got[16: many.tokens].double(), first[16:].double()
    # another kernel's roundings: of P and V 2^-11 each, of K 2^-11 of scores below 5, all of sums of p |v| / sum p < 1, for both; the results spread by 0.03
    assert bool((late[0] - late[1]).abs().max() <= 2.0 ** -7)
    assert report(slice(3, 7), prefix_table=((0, 2), 1 << 20)) & D.DFLASH_DEV_CAPACITY
    assert report(slice(0, 3), prefix_table=((1, 0), -7)) & D.DFLASH_DEV_CAPACITY


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("G", [4, 9])
def test_queries_that_are_not_finite(R, bad, G):
    c = Case(R, 2, 128, 1, G, [(100, [(20, 1), (5, 1)]), (0, [(30, 1)])], 16, False)
    want = c.run(R)
    for row in range(3):
        q = c.q.clone()
        c.q[row, 1, 9] = bad
        st = status()
        got = c.run(R, st=st)
        others = [i for i in range(3) if i != row]
        assert int(st) == D.DFLASH_DEV_NONFINITE and torch.equal(got[others], want[others])
        c.q = q


def test_graphs_and_streams(R):
    """Two captured calls with workspaces of their own, replayed together with new lengths; a call on another stream."""
    rng = np.random.default_rng(8)
    cases = [Case(R, s, 128, 2, 6, [(500, uneven(rng, 5, 200, 2)), (90, uneven(rng, 3, 200, 2))], 16, False, "bf16") for s in (1, 2)]
    want = [c.run(R) for c in cases]
    held = [c.args() for c in cases]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(cases[0].run(R, stream=side), want[0])
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    for a in held:
        with torch.cuda.stream(side):
            R.kv4_prefix_attention(*a)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(R.kv4_prefix_attention(*a))
        graphs.append(g)
    other = torch.cuda.Stream()
    for _ in range(5):
        for s, g in zip((side, other), graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for c, o, w in zip(cases, outs, want):
            assert torch.equal(o[: c.tokens], w)
    c = cases[0]
    c.prefix[0], c.own[2] = 123, 3
    held[0][3].copy_(ints(c.prefix))
    held[0][6].copy_(ints(c.own))
    graphs[0].replay()
    c.parts[0] = tuple(x[:123] for x in c.parts[0])
    c.parts[4] = tuple(x[:3] for x in c.parts[4])
    c.check(R, got=outs[0][: c.tokens])


def test_calls_behind_one_another(R):
    """Different calls that share a workspace, one behind the other without a wait, calls without a prefix between them."""
    rng = np.random.default_rng(31)
    cases = [Case(R, 11, 128, 2, 4, [(3000, uneven(rng, 9, 500, 1))], 16, False, "bf16"),
             Case(R, 12, 128, 2, 4, [(40, [(3, 1)]), (0, uneven(rng, 3, 90, 5))], 16, False, "bf16"),
             Case(R, 13, 128, 2, 9, [(1200, uneven(rng, 12, 300, 8)), (700, uneven(rng, 30, 40, 8))], 16, False, "bf16"),
             Case(R, 14, 128, 2, 9, [(9000, [(0, 1)])], 16, False, "bf16")]
    want = [c.run(R) for c in cases]
    held = [c.args() for c in cases]
    space = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    got = []
    for i in range(40):
        k = int(rng.integers(4))
        got.append((k, R.kv4_prefix_attention(*held[k], workspace=space)))
        if i % 5 == 4:
            cache, q, _, _, _, table, own, off, most = held[k][:9]
            R.kv4_attention(cache, q, table, own, off, most, workspace=space)
    torch.cuda.synchronize()
    for k, o in got:
        assert torch.equal(o[: cases[k].tokens], want[k])


def test_most_groups_and_sequences(R):
    rng = np.random.default_rng(1)
    Case(R, 5, 64, 1, 2, [(int(rng.integers(0, 40)), [(int(rng.integers(1, 20)), 1)]) for _ in range(1024)], 16, False).check(R)
    Case(R, 6, 64, 1, 5, [(700, [(int(rng.integers(8, 20)), 8) for _ in range(1024)])], 16, False).check(R)
