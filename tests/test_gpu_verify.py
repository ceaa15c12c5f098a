"""The verify-step operators on the GPU against their 64-bit forms (verify_ref.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import dflash_block_drafter_gb300 as D  # noqa: E402
import gpu_helpers as H  # noqa: E402
import verify_ref as V  # noqa: E402

pytestmark = pytest.mark.gpu


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


TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------- page tables
def pages_case(rng, n_seq, page, width, most, spare, finished=0.1, out=0.1):
    lengths = rng.integers(0, most + 1, n_seq)
    new = rng.integers(0, 9, n_seq)
    held = -(-lengths // page)
    fresh = rng.random(n_seq) < 0.2  # prompts that arrive
    new[fresh], lengths[fresh], held[fresh] = rng.integers(1, most + 1, fresh.sum()), 0, 0
    done = rng.random(n_seq) < finished
    lengths[done] = new[done] = 0
    away = rng.random(n_seq) < out
    lengths[away] = -1
    n_pages = int(held.sum()) + spare
    order = rng.permutation(n_pages)
    table = np.full((n_seq, width), -5, np.int32)
    at = 0
    for s in range(n_seq):
        table[s, : held[s]] = order[at: at + held[s]]
        at += held[s]
    head = int(rng.integers(0, n_pages))
    ring = np.full(n_pages, -9, np.int32)
    ring[(head + np.arange(spare)) % n_pages] = order[at:]
    return lengths, new, held, table, ring, np.array([head, spare])


def check_pages(R, lengths, new, held, table, ring, state, page, cap, in_place):
    want = V.page_tables(lengths, new, held, table, ring, state, page, cap)
    t, r, h, rs, st = ints(table), ints(ring), ints(held), ints(state), status()
    ho, ro = (h, rs) if in_place else (torch.full_like(h, -3), torch.full_like(rs, -3))
    off, slots, pos = R.page_tables(ints(lengths), ints(new), h, t, r, rs, page, cap, held_out=ho, ring_state_out=ro, status=st)
    got = [x.cpu().numpy() for x in (ho, t, r, ro, off, slots, pos)]
    for name, g, w in zip(("held", "table", "ring", "ring state", "offsets", "slots", "positions"), got, want):
        assert np.array_equal(g, w), name
    assert (int(st) == D.DFLASH_DEV_CAPACITY) == bool(want[7]) and int(st) in (0, D.DFLASH_DEV_CAPACITY)
    if not in_place:
        assert np.array_equal(h.cpu().numpy(), held) and np.array_equal(rs.cpu().numpy(), state)
    return got


@pytest.mark.parametrize("n_seq,page,most,cap", [(1, 16, 5, 8), (1, 64, 40000, 50000), (5, 16, 70, 64), (16, 64, 3000, 128),
                                                 (33, 32, 500, 9000), (1000, 16, 60, 20000), (1025, 256, 900, 4096),
                                                 (4096, 16, 40, 70000), (3700, 128, 10, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_page_tables(R, n_seq, page, most, cap, in_place):
    rng = np.random.default_rng(n_seq + page)
    width = -(-(most + 8) // page) + 1
    lengths, new, held, table, ring, state = pages_case(rng, n_seq, page, width, most, spare=1)
    lengths2 = np.where(lengths < 0, 0, lengths)
    need = int(np.maximum(-(-(lengths2 + new) // page) * (lengths >= 0) - held, 0).sum())
    for spare in (need + 3, max(need, 1), max(need // 2, 1)):  # enough, just enough, too few
        args = pages_case(np.random.default_rng(n_seq + page), n_seq, page, width, most, spare)
        check_pages(R, *args, page, cap, in_place)


def test_page_tables_narrow_table_and_bad_pages(R):
    # request 1 does not fit the table's width, request 2's table names a page that does not exist
    got = check_pages(R, np.array([3, 90, 20]), np.array([2, 8, 2]), np.array([1, 2, 2]),
                      np.array([[0, -1], [1, 2], [3, 77]], np.int32), np.array([5, 4, -1, -1, -1, -1], np.int32), np.array([0, 2]), 16, 16, True)
    assert got[5].tolist()[:12] == [3, 4] + [-1] * 10


def test_page_tables_ring_out_of_range(R):
    t, st = ints([[0, -1]]), status()
    off, slots, _ = R.page_tables(ints([16]), ints([1]), ints([1]), t, ints([1, 2, 3, 0]), ints([7, 9]), 16, 4, status=st)
    assert int(st) == D.DFLASH_DEV_CAPACITY and off.tolist() == [0, 1]


def test_page_tables_steps_keep_every_page_once(R):
    """Many steps of requests that grow, shrink and finish, in place and captured as one graph."""
    rng = np.random.default_rng(7)
    n, page, width, n_pages, cap = 24, 16, 40, 500, 24 * 200
    lengths, new, held = ints(np.zeros(n)), ints(np.zeros(n)), ints(np.zeros(n))
    table, ring, state, st = ints(np.full((n, width), -1)), ints(np.arange(n_pages)), ints([0, n_pages]), status()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        R.page_tables(lengths, new, held, table, ring, state, page, cap, status=st)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        off, slots, pos = R.page_tables(lengths, new, held, table, ring, state, page, cap, status=st)
    ref = [np.zeros(n, int), np.full((n, width), -1, np.int32), np.arange(n_pages, dtype=np.int32), np.array([0, n_pages])]
    size = np.zeros(n, int)
    for step in range(40):
        add = rng.integers(0, 30, n)
        size = np.where(rng.random(n) < 0.2, 0, size)
        add = np.where(size + add > width * page, 0, add)
        lengths.copy_(ints(size))
        new.copy_(ints(add))
        graph.replay()
        w = V.page_tables(size, add, *ref, page, cap)
        ref = list(w[:4])
        for g, x in zip((held, table, ring, state, off, slots, pos), w):
            assert np.array_equal(g.cpu().numpy(), x), step
        size = size + add
        h, t, r, rs = ref
        free = r[(rs[0] + np.arange(rs[1])) % n_pages]
        owned = np.concatenate([t[s, : h[s]] for s in range(n)])
        assert np.array_equal(np.sort(np.concatenate([free, owned])), np.arange(n_pages))
    assert int(st) == 0


# ------------------------------------------------------------ write and read
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,heads,page,extra", [(1, 1, 16, 0), (7, 3, 32, 8), (130, 2, 256, 64)])
def test_write_read(R, d, kind, rows, heads, page, extra):
    rng = np.random.default_rng(rows * d)
    n_pages = rows // page + 2
    wide = rng.standard_normal((rows, 2 * heads * d + extra)) * np.exp(rng.standard_normal((rows, 1)) * 2)
    wide[0, :40] = 0  # a block of zeros, and part of the next
    if rows > 3:
        wide[1, :32] = np.tile([-2.0, 2.0], 16)  # ties of magnitude, both signs
        wide[2, :32] = 2.0 ** -30  # below FP16's smallest scale
        wide[3, :64] = np.arange(64) / 8.0  # quotients that lie on halves
    both = torch.as_tensor(wide, device="cuda").to(TYPES[kind])
    k = both[:, : heads * d].unflatten(1, (heads, d))
    v = both[:, heads * d: 2 * heads * d].unflatten(1, (heads, d))
    slots = rng.permutation(n_pages * page)[:rows].astype(np.int32)
    if rows > 3:
        slots[rng.integers(1, rows)] = -1
    before = rng.integers(0, 256, (n_pages, heads, page // 16, 18 * d), dtype=np.uint8)
    cache, st = torch.as_tensor(before, device="cuda"), status()
    R.kv4_write(cache, k, v, ints(slots), status=st)
    want = before.copy()
    kk, vv = k.double().cpu().numpy(), v.double().cpu().numpy()
    V.store(want, slots, kk, vv)
    got = cache.cpu().numpy()
    # the scale of a block of zeros may have either sign: compare values there, bytes everywhere else
    neg = want.copy()
    assert np.array_equal(np.isin(got ^ neg, (0, 0x80)), np.ones_like(got, bool))
    ck, cv = R.kv4_read(cache, ints(slots), status=st)
    for x, w in zip((ck, cv), V.load(want, slots)):
        assert np.array_equal(x.cpu().numpy().astype(np.float64), w)
    # cells that no slot names are as they were
    others = np.setdiff1d(np.arange(n_pages * page), slots)
    kc, vc, ks, vs = V.word_places(d)
    for at in (kc, vc, ks, ks + 1, vs, vs + 1):
        g = got.transpose(0, 2, 1, 3).reshape(-1, heads, 18 * d)[others // 16]
        b = before.transpose(0, 2, 1, 3).reshape(-1, heads, 18 * d)[others // 16]
        idx = np.broadcast_to(at[others % 16][:, None], (len(others), heads, at.shape[1]))
        assert np.array_equal(np.take_along_axis(g, idx, -1), np.take_along_axis(b, idx, -1))
    assert int(st) == 0


def test_write_reports_bad_slots_and_values(R):
    cache = torch.full((2, 1, 1, 18 * 64), 0x5A, dtype=torch.uint8, device="cuda")
    k = torch.ones((4, 1, 64), dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    st = status()
    R.kv4_write(cache, k, v, ints([32, -1, -(2 ** 31), 2 ** 31 - 1]), status=st)
    assert int(st) == D.DFLASH_DEV_CAPACITY and bool((cache == 0x5A).all())
    st.zero_()
    kk, vv = R.kv4_read(cache, ints([32, -5]), status=st)
    assert int(st) == D.DFLASH_DEV_CAPACITY and not kk.any() and not vv.any()
    for bad in (float("nan"), float("inf"), -float("inf"), 1e6):
        st.zero_()
        k = torch.ones((1, 1, 64), dtype=torch.bfloat16, device="cuda")
        k[0, 0, 5] = bad
        R.kv4_write(cache, k, v[:1], ints([3]), status=st)
        kk, vv = R.kv4_read(cache, ints([3]))
        assert int(st) == D.DFLASH_DEV_NONFINITE
        assert not kk[0, 0, :32].any() and bool((kk[0, 0, 32:] == 1).all()) and bool((vv == 1).all())


def test_write_largest_fp16(R):
    cache, st = R.kv4_cache(1, 16, 1, 64), status()
    k = torch.full((1, 1, 64), 65504.0, dtype=torch.float16, device="cuda")
    R.kv4_write(cache, k, -k, ints([15]), status=st)
    kk, vv = R.kv4_read(cache, ints([15]))
    assert int(st) == 0 and bool((kk == 65504).all()) and bool((vv == -65504).all())


# ----------------------------------------------------------------- attention
def attn_case(seed, d, heads, G, lens, rows, page, kind, spare_width=1, gain=1.0, vgain=1.0):
    """A cache whose unused cells, unused table entries and rows behind the last sequence hold what must not be read."""
    rng = np.random.default_rng(seed)
    counts = [-(-max(n, 0) // page) for n in lens]
    n_pages, width = sum(counts) + 2, max(counts) + spare_width
    order = rng.permutation(n_pages)
    table = np.full((len(lens), width), 1 << 30, np.int32)
    cache = np.full((n_pages, heads, page // 16, 18 * d), 0xFF, np.uint8)  # scales are NaN
    at = 0
    for s, n in enumerate(lens):
        table[s, : counts[s]] = order[at: at + counts[s]]
        at += counts[s]
        pos = np.arange(max(n, 0))
        if n > 0:
            slots = table[s, pos // page].astype(np.int64) * page + pos % page
            V.store(cache, slots, rng.standard_normal((n, heads, d)), vgain * rng.standard_normal((n, heads, d)))
    offsets = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    q = torch.as_tensor(gain * rng.standard_normal((offsets[-1] + 2, heads * G, d)), device="cuda").to(TYPES[kind])
    return cache, q, table, np.asarray(lens, np.int32), offsets


def check_attn(R, case, causal, window=0, scale=None, max_rows=None, stream=None):
    cache, q, table, lens, offsets = case
    d = q.shape[2]
    st = status()
    sc = d ** -0.5 if scale is None else scale
    out = torch.full_like(q, 7.0)
    rows = int(np.max(np.diff(offsets))) if max_rows is None else max_rows
    R.kv4_attention(torch.as_tensor(cache, device="cuda"), q, ints(table), ints(lens), ints(offsets), max(rows, 1), causal=causal,
                    window=window, scale=scale, out=out, status=st)
    o, spread, top, seen = V.attention(cache, q.double().cpu().numpy(), table, lens, offsets, causal, window, sc)
    got = out.double().cpu().numpy()
    n = offsets[-1]
    assert np.all(got[n:] == 7.0)  # rows of no sequence
    assert int(st) == 0
    # |error| <= sum p |v| / l * (V to FP16: 2^-11, p to FP16: 2^-11, scores in FP32: the 8 FMAs and products of d terms with
    # magnitudes up to 16 times the score's terms -> e = 2^-17 per unit of the largest |score| sum, counted twice)
    # + 2^-25 max |v| per cell for p below FP16's normal range + half a step of the output's type
    eps = torch.finfo(q.dtype).eps / 2
    vmax = np.abs(spread).max() + np.abs(o[:n]).max() + 1e-30
    vall = max(vmax, 8.0 * spread.max())
    tol = spread * (2.0 ** -10 + 2.0 ** -16 * (1 + top)[..., None]) + seen[..., None] * 2.0 ** -25 * vall + eps * np.abs(np.nan_to_num(o)) \
        + torch.finfo(q.dtype).smallest_normal * eps * 2
    err = np.abs(got - o)
    assert np.all(err[:n] <= tol[:n]), f"worst {np.nanmax(err[:n] / tol[:n]):.2f} x tolerance"
    return got[:n]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,G,lens,rows,page", [
    (1, 1, [1], [1], 16), (2, 3, [17, 33, 2], [1, 1, 1], 16), (1, 8, [100], [1], 32), (2, 12, [40, 7, 300], [1, 2, 8], 64),
    (1, 16, [65, 64, 63], [8, 7, 1], 16), (3, 5, [1, 8, 9], [1, 8, 3], 128), (2, 4, [700], [4], 256)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention(R, d, kind, heads, G, lens, rows, page, causal):
    check_attn(R, attn_case(d + G, d, heads, G, lens, rows, page, kind), causal)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 5, 16, 33, 100, 2 ** 31 - 1])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_window(R, d, window, causal):
    check_attn(R, attn_case(d + window, d, 2, 4, [200, 31, 4, 64], [3, 1, 4, 8], 16, "bf16"), causal, window)


@pytest.mark.parametrize("d,G,rows", [(64, 16, 8), (128, 16, 8), (256, 12, 8), (256, 16, 8), (128, 128, 1), (256, 6, 1), (64, 3, 5)])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_attention_split_over_ctas(R, d, G, rows, kind):
    """Long contexts of uneven lengths: segments cross CTAs and are joined."""
    check_attn(R, attn_case(G, d, 1, G, [5000, 130, 9, 2500], [rows, 1, rows, 1], 64, kind), True)


@pytest.mark.parametrize("d,heads,G,rows", [(64, 2, 5, 8), (64, 1, 16, 8), (128, 2, 9, 4), (64, 2, 3, 8), (256, 2, 12, 8), (256, 2, 12, 1), (128, 4, 4, 1)])
def test_attention_many_tiles_per_cta(R, d, heads, G, rows):
    """More tiles than a CTA's buffers hold, with and without quarters of rows that are empty, and parts of several
    sequences in one CTA."""
    lens = [20000, 40, 700, 12000, 9000] if d == 256 else [30000, 100, 2000, 17000]
    check_attn(R, attn_case(d + rows, d, heads, G, lens, [rows] * len(lens), 128, "bf16"), True)


@pytest.mark.parametrize("d,G", [(64, 5), (128, 6), (256, 5), (128, 3)])
def test_attention_same_result_again(R, d, G):
    """Many parts of many sequences per CTA, over and over: the same bits each time, and the right ones."""
    rng = np.random.default_rng(d)
    lens = rng.integers(64, 2500 if d < 256 else 1200, 40).tolist()
    case = attn_case(d, d, 2, G, lens, rng.integers(2, 9, 40).tolist(), 64, "bf16")
    first = check_attn(R, case, True, max_rows=8)
    cache, q, table, ln, off = case
    c, t, ln, off = torch.as_tensor(cache, device="cuda"), ints(table), ints(ln), ints(off)
    n = first.shape[0]
    outs = [R.kv4_attention(c, q, t, ln, off, 8) for _ in range(100)]
    for o in outs:
        assert np.array_equal(o[:n].double().cpu().numpy(), first)


def test_attention_many_short(R):
    rng = np.random.default_rng(5)
    lens = rng.integers(1, 60, 700)
    check_attn(R, attn_case(9, 64, 1, 2, lens.tolist(), [1] * 700, 16, "fp16"), True)


def test_attention_rows_without_cells(R):
    """No cells at all, fewer cells than rows (a causal row before the first cell), no rows."""
    case = attn_case(3, 128, 2, 4, [0, 2, 5, 40, -3], [2, 4, 0, 1, 1], 16, "bf16")
    got = check_attn(R, case, True)
    assert not got[:4].any() and got[4:6].any() and not got[-1].any()
    check_attn(R, case, False)


@pytest.mark.parametrize("kind,gain,scale", [("bf16", 1e-20, 1e19), ("bf16", 1e20, 1e-21), ("fp16", 1e-5, 2e4), ("fp16", 2e3, 1e-4),
                                             ("bf16", 0.0, 1.0), ("fp16", 8.0, 0.5)])
def test_attention_ranges(R, kind, gain, scale):
    """Queries near the ends of their type's range, equal scores, and scores that leave one cell."""
    check_attn(R, attn_case(1, 128, 1, 4, [300], [2], 32, kind, gain=gain), True, scale=scale)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("G,rows", [(3, 8), (13, 8)])
def test_attention_rows_of_unequal_size(R, d, kind, G, rows):
    """Rows of very different magnitudes side by side, in both kernels."""
    cache, q, table, lens, offsets = attn_case(d + G, d, 1, G, [300, 90], [rows, 3], 16, kind)
    size = torch.tensor([2.0 ** 9, 1.0, 2.0 ** -5, 2.0 ** -12, 2.0 ** 7, 2.0 ** -8, 0.0], device="cuda")
    n = q.shape[0] * q.shape[1]
    q = (q.float() * size[torch.arange(n, device="cuda") % 7].view(q.shape[0], q.shape[1], 1)).to(q.dtype)
    check_attn(R, (cache, q, table, lens, offsets), True, scale=d ** -0.5 * 2.0 ** -9)


@pytest.mark.parametrize("d,G,rows,seed", [(64, 4, 1, 70), (128, 3, 4, 70), (256, 5, 8, 99)])
def test_attention_huge_queries(R, d, G, rows, seed):
    """Scores near FP32's largest value: all weight on one cell, which both kernels must find."""
    cache, q, table, lens, offsets = attn_case(seed, d, 1, G, [8], [rows], 16, "bf16", gain=1e36)
    st = status()
    out = R.kv4_attention(torch.as_tensor(cache, device="cuda"), q, ints(table), ints(lens), ints(offsets), rows, causal=False, status=st)
    n = offsets[-1]
    got, x = out[:n].double().cpu().numpy(), q[:n].double().cpu().numpy()
    k, v = V.load(cache, table[0, 0].astype(np.int64) * 16 + np.arange(8))
    s, size = np.einsum("rgd,cd->rgc", x, k[:, 0]), np.einsum("rgd,cd->rgc", np.abs(x), np.abs(k[:, 0]))
    two = np.sort(s, -1)[..., -2:]
    assert np.all(two[..., 1] - two[..., 0] > 2.0 ** -9 * size.max(-1))  # more than K's rounding moves two scores
    want = v[:, 0][s.argmax(-1)]
    assert int(st) == 0
    assert np.all(np.abs(got - want) <= np.abs(want) * (2.0 ** -11 + 2.0 ** -8))  # V to FP16, the output to BF16


@pytest.mark.parametrize("vgain", [1e-4, 3e3])
def test_attention_value_range(R, vgain):
    check_attn(R, attn_case(2, 64, 1, 4, [100], [1], 16, "bf16", vgain=vgain), True)


def test_attention_strided_rows(R):
    """q inside a wider row, out inside another."""
    cache, q, table, lens, offsets = attn_case(4, 128, 2, 3, [50, 20], [2, 1], 16, "bf16")
    st = status()
    plain = R.kv4_attention(torch.as_tensor(cache, device="cuda"), q, ints(table), ints(lens), ints(offsets), 2)
    wide = torch.zeros((q.shape[0], 8, 128), dtype=q.dtype, device="cuda")
    wide[:, 1:7] = q
    outw = torch.full((q.shape[0], 9, 128), 3.0, dtype=q.dtype, device="cuda")
    R.kv4_attention(torch.as_tensor(cache, device="cuda"), wide[:, 1:7], ints(table), ints(lens), ints(offsets), 2, out=outw[:, 2:8], status=st)
    assert torch.equal(outw[:3, 2:8], plain[:3]) and bool((outw[:, :2] == 3).all()) and bool((outw[:, 8:] == 3).all())
    assert int(st) == 0


def test_attention_reports(R):
    cache, q, table, lens, offsets = attn_case(6, 64, 1, 2, [40, 20], [2, 1], 16, "fp16")
    c = torch.as_tensor(cache, device="cuda")

    def call(table=table, lens=lens, offsets=offsets, q=q, rows=2):
        st, out = status(), torch.full_like(q, 7.0)
        R.kv4_attention(c, q, ints(table), ints(lens), ints(offsets), rows, out=out, status=st)
        return int(st), out

    good = call()
    assert good[0] == 0
    # sequence 0 has more rows than allowed: it is left alone, sequence 1 is as before
    st, out = call(rows=1)
    assert st == D.DFLASH_DEV_BAD_BLOCK and bool((out[:2] == 7).all()) and torch.equal(out[2], good[1][2])
    assert call(offsets=np.array([0, 2, 1]))[0] == D.DFLASH_DEV_BAD_BLOCK
    assert call(offsets=np.array([-1, 0, 1]))[0] == D.DFLASH_DEV_BAD_BLOCK
    assert call(offsets=np.array([0, 2, 99]), rows=8)[0] == D.DFLASH_DEV_BAD_BLOCK
    # more cells than the table is wide
    assert call(lens=np.array([1000, 20]))[0] & D.DFLASH_DEV_CAPACITY
    bad = table.copy()
    bad[0, 1] = -1
    assert call(table=bad)[0] & D.DFLASH_DEV_CAPACITY
    nan = q.clone()
    nan[0, 0, 3] = float("nan")
    st, out = call(q=nan)
    assert st == D.DFLASH_DEV_NONFINITE and torch.equal(out[1:3], good[1][1:3])


@pytest.mark.parametrize("G", [4, 17])
def test_attention_streams_and_graph(R, G):
    """Two calls at once on two streams, and a captured call replayed with other lengths; both kernels."""
    a = attn_case(8, 128, 2, G, [900, 30], [2, 1], 32, "bf16")
    cache, q, table, lens, offsets = a
    c, t = torch.as_tensor(cache, device="cuda"), ints(table)
    ln, off = ints(lens), ints(offsets)
    want = R.kv4_attention(c, q, t, ln, off, 2)[:3].clone()
    short = ints([450, 30])
    want2 = R.kv4_attention(c, q, t, short, off, 2)[:3].clone()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(s1):
            x = R.kv4_attention(c, q, t, ln, off, 2)
        y = R.kv4_attention(c, q, t, short, off, 2, stream=s2, workspace=torch.empty(1 << 24, dtype=torch.uint8, device="cuda"),
                            out=torch.zeros_like(q))
        torch.cuda.synchronize()
        assert torch.equal(x[:3], want) and torch.equal(y[:3], want2)
    ws, out = torch.empty(1 << 24, dtype=torch.uint8, device="cuda"), torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        R.kv4_attention(c, q, t, ln, off, 2, out=out, workspace=ws)
    for lengths, w in ((lens, want), ([450, 30], want2)):
        ln.copy_(ints(lengths))
        g.replay()
        assert torch.equal(out[:3], w)


def test_stream_argument(R):
    """A call on a stream that has not come to it yet: its workspace and outputs are not handed to the current stream."""
    cache, q, table, lens, offsets = attn_case(6, 128, 2, 4, [3000, 70], [1, 2], 64, "bf16")
    c, table, lens, offsets = torch.as_tensor(cache, device="cuda"), ints(table), ints(lens), ints(offsets)
    n = int(offsets[-1])
    plain = R.kv4_attention(c, q, table, lens, offsets, 2)[:n].clone()
    logits = q.flatten(1)
    scores = R.token_logprobs(logits, top_k=3)
    args = D.DflashKv4Cache(c.data_ptr(), c.shape[0], 64, 2, 128)
    size = D.dflash_kv4_attention_workspace(args, 8, 2, 2, table.shape[1]) + 16
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    out = R.kv4_attention(c, q, table, lens, offsets, 2, stream=side)
    mine = torch.full((size,), 0x7F, dtype=torch.uint8, device="cuda")
    again = R.token_logprobs(logits, top_k=3, stream=side)
    torch.cuda.synchronize()
    assert bool((mine == 0x7F).all())
    assert torch.equal(out[:n], plain)
    for x, y in zip(scores[1:], again[1:]):
        assert torch.equal(x, y)


def test_cells_beyond_4_gb(R):
    """Pages whose bytes lie beyond 32 bits: written, read back and attended to."""
    heads, d, page, n_pages = 8, 256, 256, 9000  # 5.3 GB
    cache = torch.empty((n_pages, heads, page // 16, 18 * d), dtype=torch.uint8, device="cuda")
    cache[-4:] = 0xFF
    cache[:4] = 0xFF
    rng = np.random.default_rng(1)
    n, rows = 300, 2
    pages = np.array([n_pages - 1, n_pages - 3], np.int32)
    slots = ints([int(pages[p // page]) * page + p % page for p in range(n)])
    k, v = (torch.as_tensor(rng.standard_normal((n, heads, d)), device="cuda").bfloat16() for _ in range(2))
    st = status()
    R.kv4_write(cache, k, v, slots, status=st)
    kk, vv = (x.double().cpu().numpy() for x in R.kv4_read(cache, slots, status=st))
    for x, y in ((k, kk), (v, vv)):
        assert np.array_equal(V.dequantise(*V.quantise(x.double().cpu().numpy())), y)
    for G in (1, 17):
        q = torch.as_tensor(rng.standard_normal((rows, heads * G, d)), device="cuda").bfloat16()
        o = R.kv4_attention(cache, q, ints([pages]), ints([n]), ints([0, rows]), rows, status=st).double().cpu().numpy()
        qq = q.double().cpu().numpy()
        for i in range(rows):
            for h in range(heads * G):
                m = n - rows + i + 1
                x = kk[:m, h // G] @ qq[i, h] / 16.0
                p = np.exp(x - x.max())
                want, spread = p @ vv[:m, h // G] / p.sum(), p @ np.abs(vv[:m, h // G]) / p.sum()
                tol = spread * (2.0 ** -10 + 2.0 ** -16 * (1 + np.abs(x).max())) + m * 2.0 ** -25 * 8 + 2.0 ** -8 * np.abs(want)
                assert np.all(np.abs(o[i, h] - want) <= tol)
    assert int(st) == 0


# ------------------------------------------------------------------ logprobs
def check_logprobs(R, x, tokens, k):
    st = status()
    lp, ent, ids, top = R.token_logprobs(x, None if tokens is None else ints(tokens), top_k=k, status=st)
    toks = np.full(x.shape[0], -1) if tokens is None else np.asarray(tokens)
    wl, we, wi, wt, spread = V.logprobs(x.double().cpu().numpy(), toks, k)
    # FP32 sums: a thread adds up to vocab / 256 + 64 terms one by one, each with 2^-21 from the power of two
    rel = (x.shape[1] / 256 + 64) * 2.0 ** -24 + 2.0 ** -20
    def near(g, w, scale):
        g, w = g.cpu().numpy().astype(np.float64), np.asarray(w)
        inf = np.isinf(w)
        assert np.array_equal(g[inf], w[inf])
        assert np.all(np.abs(g - w)[~inf] <= (rel * scale + 2.0 ** -22 * np.abs(np.where(inf, 0, w)))[~inf])
    if tokens is None:
        assert lp is None
    else:
        near(lp, wl, np.ones_like(wl))
    near(ent, we, 2 + 2 * spread)
    assert np.array_equal(ids.cpu().numpy(), wi)
    near(top, wt, np.ones_like(wt))
    assert int(st) == 0


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,vocab,k", [(1, 1, 0), (1, 1, 3), (3, 7, 7), (2, 33, 32), (5, 1023, 1), (8, 1024, 8), (1, 4099, 20),
                                          (4, 50001, 5), (400, 2500, 4), (1, 151936, 32), (9, 151936, 8)])
def test_logprobs(R, kind, rows, vocab, k):
    rng = np.random.default_rng(vocab + rows)
    x = torch.as_tensor(rng.standard_normal((rows, vocab)) * 3, device="cuda").to(TYPES[kind])
    tokens = rng.integers(0, vocab, rows)
    tokens[-1] = -1 if rows > 1 else tokens[-1]
    check_logprobs(R, x, tokens, k)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("stride,first", [(1000, 0), (1001, 1), (1003, 3), (1013, 5)])
def test_logprobs_strides(R, kind, stride, first):
    """Rows that start at any element of a 16-byte piece; what lies around a row must not count."""
    buf = torch.full((9 * stride + 16,), float("inf"), device="cuda", dtype=TYPES[kind])
    x = torch.as_strided(buf, (9, 997), (stride, 1), first)
    rng = np.random.default_rng(stride)
    x.copy_(torch.as_tensor(rng.standard_normal((9, 997)), device="cuda").to(buf.dtype))
    check_logprobs(R, x, rng.integers(0, 997, 9), 6)


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab", [300, 40000])
def test_logprobs_masks_and_ties(R, kind, vocab):
    rng = np.random.default_rng(3)
    low = torch.finfo(TYPES[kind]).min
    x = np.round(rng.standard_normal((9, vocab)) * 2) / 2  # many ties
    x[1] = 1.0                                  # all equal: ids 0, 1, 2, ..
    x[2] = -np.inf                              # nothing left
    x[3] = -np.inf
    x[3, vocab // 2] = -4.0                     # one token left
    x[4] = low                                  # the type's lowest everywhere
    x[5] = low
    x[5, 7], x[5, vocab - 1] = 2.0, 2.0
    x[6, : vocab - 3] = -np.inf
    x[7, ::2] = 0.0
    x[7, 1::2] = -0.0                           # zeros of both signs are equal
    x[8] = np.sort(x[8])                        # ascending: every batch brings new leaders
    tokens = [0, 1, 2, vocab // 2, 4, 7, 0, 3, vocab - 1]
    check_logprobs(R, torch.as_tensor(x, device="cuda").to(TYPES[kind]), tokens, 32)


def test_logprobs_large_values(R):
    rng = np.random.default_rng(4)
    x = torch.as_tensor(rng.standard_normal((4, 3000)) + 3e4, device="cuda").float()
    check_logprobs(R, x, rng.integers(0, 3000, 4), 3)
    check_logprobs(R, x.float() * -1e30, rng.integers(0, 3000, 4), 3)


def test_logprobs_reports(R):
    x = torch.zeros((3, 500), device="cuda")
    st = status()
    lp, _, _, _ = R.token_logprobs(x, ints([500, -1, -2]), status=st)
    assert int(st) == D.DFLASH_DEV_BAD_TOKEN and lp.tolist() == [0, 0, 0]
    want = R.token_logprobs(x, ints([1, 2, 3]), top_k=2)
    for bad in (float("nan"), float("inf")):
        y = x.clone()
        y[1, 77] = bad
        st.zero_()
        got = R.token_logprobs(y, ints([1, 2, 3]), top_k=2, status=st)
        assert int(st) == D.DFLASH_DEV_NONFINITE
        for g, w in zip(got, want):
            assert torch.equal(g[[0, 2]], w[[0, 2]])


# ------------------------------------------------------------- one step, whole
def test_verify_steps_together(R):
    """Steps of a served model: page tables, cells, attention, scores, acceptance, the next lengths on the device."""
    rng = np.random.default_rng(11)
    n, heads, G, d, page, B, vocab, steps = 5, 2, 4, 64, 16, 4, 900, 6
    n_pages, width = 120, 20
    cap = n * B
    cache = R.kv4_cache(n_pages, page, heads, d)
    held, table, ring, state = ints(np.zeros(n)), ints(np.full((n, width), -1)), ints(np.arange(n_pages)), ints([0, n_pages])
    length = ints(np.zeros(n))
    st = status()
    head = torch.as_tensor(rng.standard_normal((vocab, heads * G * d)), device="cuda").float()
    keys = [np.zeros((0, heads, d)) for _ in range(n)]
    vals = [np.zeros((0, heads, d)) for _ in range(n)]
    accepted, bonus = ints(np.zeros(n)), ints(np.zeros(n))
    for step in range(steps):
        rows = ints(np.full(n, B))
        k, v = (torch.as_tensor(rng.standard_normal((cap, heads, d)), device="cuda").bfloat16() for _ in range(2))
        q = torch.as_tensor(rng.standard_normal((cap, heads * G, d)), device="cuda").bfloat16()
        before = length.cpu().numpy()
        off, slots, pos = R.page_tables(length, rows, held, table, ring, state, page, cap, status=st)
        R.kv4_write(cache, k, v, slots, status=st)
        o = R.kv4_attention(cache, q, table, length + rows, off, B, causal=True, status=st)
        logits = o.float().flatten(1) @ head.t()
        drafts = rng.integers(0, vocab, (n, B - 1)).astype(np.int32)
        tokens = rng.integers(0, vocab, cap)
        lp, ent, ids, top = R.token_logprobs(logits, ints(tokens), top_k=1, status=st)
        drafts[:, 0] = ids.view(n, B)[:, 0].cpu().numpy()  # the first candidate is always right
        R.accept(ints(drafts), ids.view(n, B).contiguous(), rows, accepted, bonus, anchor_pos=length)
        # the same by hand
        assert pos.cpu().numpy().tolist() == [int(before[s]) + j for s in range(n) for j in range(B)]
        want_len = length.cpu().numpy()
        acc = accepted.cpu().numpy()
        assert np.array_equal(want_len, before + acc + 1) and np.all(acc >= 1)
        for s in range(n):
            new = slice(s * B, s * B + B)
            kq, vq = (V.dequantise(*V.quantise(x[new].double().cpu().numpy())) for x in (k, v))
            K, W = np.concatenate([keys[s][: before[s]], kq]), np.concatenate([vals[s][: before[s]], vq])
            keys[s], vals[s] = K, W
            for i in range(B):
                m = before[s] + i + 1
                for h in range(heads * G):
                    x = K[:m, h // G] @ q[s * B + i, h].double().cpu().numpy() / 8.0
                    p = np.exp(x - x.max())
                    want = p @ W[:m, h // G] / p.sum()
                    tol = (p @ np.abs(W[:m, h // G]) / p.sum()) * (2.0 ** -10 + 2.0 ** -16 * (1 + np.abs(x).max())) \
                        + m * 2.0 ** -25 * 8 + 2.0 ** -8 * np.abs(want)
                    assert np.all(np.abs(o[s * B + i, h].double().cpu().numpy() - want) <= tol)
        check_logprobs(R, logits, tokens, 1)
    assert int(st) == 0
