"""The verify-step operators on the GPU where their rules meet: pages given back before a window, rows and cells without
weight, far apart scores, and the edges of the tcgen05 attention kernel (more than 32 rows per kv head)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import dflash_block_drafter_gb300 as D  # noqa: E402
import verify_exact as E  # noqa: E402
import verify_ref as V  # noqa: E402
from test_gpu_verify import R, TYPES, attn_case, check_attn, ints, status  # noqa: E402,F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- windows
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads,G", [(2, 4), (1, 5)])  # 32 and 40 rows per kv head: the warp-level and the tcgen05 kernel
@pytest.mark.parametrize("page,window", [(16, 1), (16, 33), (16, 100), (32, 70), (128, 20)])
@pytest.mark.parametrize("causal", [True, False])
def test_window_with_pages_given_back(R, d, heads, G, page, window, causal):
    """Pages that lie wholly before the window are gone from the table: no report, and the right outputs."""
    case = attn_case(d + window, d, heads, G, [300, 31, 4, 650], [8, 1, 4, 2], page, "bf16")
    cache, q, table, lens, offsets = case
    for s, n in enumerate(lens):
        first = max(int(n) - (int(offsets[s + 1] - offsets[s]) - 1 if causal else 0) - window, 0)  # that any row sees
        table[s, : first // page] = -1
    assert (table[0, 0] == -1) and (table[3, 0] == -1)
    check_attn(R, case, causal, window)


# -------------------------------------------------------------- values, weights
def integer_cells(R, k, v, page):
    """A cache whose cells 0 .. n - 1 (in order, one kv head) hold the integers k, v [n, d] exactly, one for all of its heads: values of
    -8 .. 7 with a -8 in each block of 32 channels, whose scale then is 1."""
    n, d = k.shape
    cache = R.kv4_cache(-(-n // page), page, 1, d)
    R.kv4_write(cache, *(torch.as_tensor(x, device="cuda").half()[:, None] for x in (k, v)), ints(np.arange(n)))
    back = R.kv4_read(cache, ints(np.arange(n)))
    assert all(np.array_equal(b[:, 0].cpu().numpy(), x) for b, x in zip(back, (k, v)))
    return cache


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("G,rows", [(4, 2), (5, 8)])  # the warp-level and the tcgen05 kernel
@pytest.mark.parametrize("below", [24.5, 25.5, 20.25])
def test_long_tail_below_one_cell(R, d, G, rows, below):
    """One cell outweighs each of 32767 others by 2^below, and the others alone make the output: their sum must not be lost in
    P's smallest step.  So many sequences (over the same pages) that segments are hardly split."""
    n, page, n_seq = 32768, 64, 512
    k, v = np.zeros((n, d)), np.full((n, d), 4.0)
    k[:, 31::32] = v[:, 31::32] = -8
    k[0, 0], v[0, :] = 7, 0
    v[0, 31::32] = -8
    cache = integer_cells(R, k, v, page)
    q = torch.zeros((n_seq * rows, G, d), dtype=torch.float16, device="cuda")
    q[:, :, 0] = 1
    st = status()
    table = torch.arange(n // page, dtype=torch.int32, device="cuda").repeat(n_seq, 1)
    out = R.kv4_attention(cache, q, table, ints(np.full(n_seq, n)), ints(np.arange(n_seq + 1) * rows), rows, causal=False,
                          scale=below * np.log(2) / 7, status=st).double().cpu().numpy()
    tail = 4 * (n - 1) * 2.0 ** -below
    want = np.where(np.arange(d) % 32 == 31, -8.0, tail / (1 + tail / 4))
    # a weight to FP16: half of its smallest step, 2^-25 of 2^7 at the reference, a cell (or 2^-11 of it); the power of two and the
    # score in FP32: 2^-21 of the weight; the sum of n terms in FP32, 16 a step; the output to FP16
    tol = 4 * n * 2.0 ** -32 + tail * (2.0 ** -11 + 2.0 ** -21 + n / 16 * 2.0 ** -23) + np.abs(want) * 2.0 ** -11
    tol = np.where(np.arange(d) % 32 == 31, 8 * (2.0 ** -11 + n / 16 * 2.0 ** -23) + 8 * 2.0 ** -11, tol)
    assert int(st) == 0
    worst = np.max(np.abs(out - want) / tol)
    assert worst <= 1, worst


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("G,rows", [(3, 1), (4, 8), (5, 8)])
def test_small_part_of_a_query(R, d, kind, G, rows):
    """A query with one large and one small value, over cells whose values there are zeros with a large scale: all scores are 0."""
    k, v = np.zeros((2, d)), np.ones((2, d))
    v[1], v[:, 31::32] = -1, -8
    cache = integer_cells(R, np.where(np.arange(d) % 32 == 31, -8.0, k), v, 16)
    wide = np.zeros((2, 1, d))
    wide[0, 0, 31::32] = -512  # cell 0: scale 64; cell 1: no scale
    R.kv4_write(cache, torch.as_tensor(wide, device="cuda").half(), torch.as_tensor(v, device="cuda").half()[:, None], ints([0, 1]))
    q = torch.zeros((rows, G, d), dtype=TYPES[kind], device="cuda")
    q[:, :, 0::32], q[:, :, 2::32] = 1, 2.0 ** -16
    st = status()
    out = R.kv4_attention(cache, q, ints([[0]]), ints([2]), ints([0, rows]), rows, causal=False, scale=16.0, status=st).double().cpu().numpy()
    # the sum of a block of q is off by 2^-19 of the row's largest, 1; with the scale 64 and the codes' 8 a score is off by 2^-10 a
    # block, times 16; two weights that should be equal give half of that; each to FP16: 2^-11
    tol = d / 32 * 2.0 ** -7 + 2.0 ** -10
    assert int(st) == 0
    assert np.abs(out[..., :31]).max() <= tol, np.abs(out[..., :31]).max()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("G,rows", [(4, 8), (5, 8)])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("channel", [0, -2])
def test_queries_that_are_not_finite(R, d, kind, G, rows, bad, channel):
    """An infinity or a NaN in a row's query is reported, also where it makes all of the scores -infinity; other rows keep theirs."""
    k, v = np.full((90, d), 3.0), np.ones((90, d))
    k[:, 31::32] = v[:, 31::32] = -8
    cache = integer_cells(R, k, v, 16)
    q = torch.ones((rows, G, d), dtype=TYPES[kind], device="cuda")

    def call(q):
        st = status()
        return R.kv4_attention(cache, q, ints([np.arange(6)]), ints([90]), ints([0, rows]), rows, causal=False, status=st), int(st)

    want, st = call(q)
    assert st == 0
    q[1, 2, channel] = bad
    got, st = call(q)
    assert st == D.DFLASH_DEV_NONFINITE
    others = torch.ones((rows, G), dtype=torch.bool, device="cuda")
    others[1, 2] = False
    assert torch.equal(got[others], want[others])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("G,rows", [(4, 8), (5, 8)])
def test_queries_that_meet_no_cell(R, d, kind, G, rows):
    """Rows before the first cell have no scores, whatever their queries hold: zeros and no report."""
    cache, q, table, lens, offsets = attn_case(d, d, 1, G, [5, 70, 0], [rows, rows, 1], 16, kind)
    q[: rows - 5] = float("inf")  # causal: positions -3 .. -1
    q[2 * rows] = float("nan")
    st, out = status(), torch.full_like(q, 7.0)
    R.kv4_attention(torch.as_tensor(cache, device="cuda"), q, ints(table), ints(lens), ints(offsets), rows, out=out, status=st)
    assert int(st) == 0 and not out[: rows - 5].any() and not out[2 * rows].any()
    assert bool(out[rows - 5: 2 * rows].isfinite().all()) and bool((out[2 * rows + 1:] == 7).all())


# --------------------------------------------------------------- page tables
@pytest.mark.parametrize("held,nearest", [([-1, 1, 1], [0, 1, 1]), ([1, 5, 1], [1, 4, 1]), ([1, 1, 2 ** 31 - 1], [1, 1, 4]),
                                          ([1, 1, -(2 ** 31)], [1, 1, 0])])
@pytest.mark.parametrize("lengths", [[3, 60, 0], [3, 60, -1]])
def test_held_out_of_range(R, held, nearest, lengths):
    """A count of pages that no table row can hold is reported; the call goes on as with the nearer end."""
    def call(h):
        table, ring, st = ints(np.arange(12).reshape(3, 4)), ints(np.arange(12, 24).tolist() + [-1] * 12), status()
        h, rs = ints(h), ints([0, 12])
        out = R.page_tables(ints(lengths), ints([2, 2, 0]), h, table, ring, rs, 16, 8, status=st)
        return int(st), [x.tolist() for x in (h, table, ring, rs, *out)]

    st, got = call(held)
    assert st == D.DFLASH_DEV_CAPACITY
    assert call(nearest) == (0, got)


# ---------------------------------------------------------- every cell, once
def exact_cache(R, rng, lens, heads, d, page):
    """(cache, table, [(k, v)]) of sequences of exact cells."""
    counts = [-(-n // page) for n in lens]
    order = rng.permutation(sum(counts))
    cache = R.kv4_cache(len(order), page, heads, d)
    cache.fill_(0xFF)
    table = np.full((len(lens), max(counts)), -1, np.int32)
    parts, at = [], 0
    for s, n in enumerate(lens):
        table[s, : counts[s]] = order[at: at + counts[s]]
        at += counts[s]
        parts.append(E.cells(rng, n, heads, d))
        pos = np.arange(n)
        R.kv4_write(cache, *(torch.as_tensor(x, device="cuda").half() for x in parts[s]), ints(table[s, pos // page] * page + pos % page))
    return cache, table, parts


@pytest.mark.parametrize("d,heads,G,rows", [(64, 2, 5, 8), (128, 1, 9, 8), (256, 2, 12, 8), (256, 1, 5, 8), (64, 2, 3, 8), (128, 2, 4, 8),
                                            (128, 4, 4, 1), (256, 2, 12, 1), (64, 1, 16, 1)])
@pytest.mark.parametrize("lens", ["long", "many"])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1500)])
def test_every_cell_once(R, d, heads, G, rows, lens, causal, window):
    """Long and many sequences whose result shows a single tile that is lost, taken twice or stale."""
    rng = np.random.default_rng(d + G)
    lens = ([30000, 100, 2000, 17000] if d < 256 else [20000, 40, 700, 12000]) if lens == "long" else rng.integers(64, 2500, 40).tolist()
    cache, table, parts = exact_cache(R, rng, lens, heads, d, 64)
    q = E.queries(rng, rows * len(lens), heads * G, d)
    st = status()
    out = R.kv4_attention(cache, torch.as_tensor(q, device="cuda").half(), ints(table), ints(lens), ints(np.arange(len(lens) + 1) * rows), rows,
                          causal=causal, window=window, scale=float(np.log(2)), status=st).double().cpu().numpy()
    assert int(st) == 0
    for s, (k, v) in enumerate(parts):
        mine = slice(s * rows, s * rows + rows)
        o, spread = E.attend(k, v, q[mine], causal, window)
        worst = np.max(np.abs(out[mine] - o) / E.tolerance(o, spread, 2.0 ** -11))
        assert worst <= 1, (s, worst)


@pytest.mark.parametrize("d,G,rows", [(64, 5, 8), (128, 5, 8), (256, 5, 8), (64, 4, 1), (128, 4, 8), (256, 4, 1)])
def test_every_cell_once_unsplit(R, d, G, rows):
    """More segments than CTAs, all of them long, over the same pages."""
    rng = np.random.default_rng(d)
    n, n_seq = 12000, 400
    cache, table, parts = exact_cache(R, rng, [n], 2, d, 64)
    q = E.queries(rng, rows, 2 * G, d)
    out = R.kv4_attention(cache, torch.as_tensor(q, device="cuda").half().repeat(n_seq, 1, 1), ints(np.repeat(table, n_seq, 0)),
                          ints(np.full(n_seq, n)), ints(np.arange(n_seq + 1) * rows), rows, scale=float(np.log(2))).double().cpu().numpy()
    o, spread = E.attend(*parts[0], q, True)
    worst = np.max(np.abs(out.reshape(n_seq, *o.shape) - o) / E.tolerance(o, spread, 2.0 ** -11))
    assert worst <= 1, worst


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("G,rows,gain", [(4, 1, 1.0), (4, 8, 4.0), (5, 8, 1.0), (16, 8, 4.0)])
def test_stated_roundings(R, d, kind, G, rows, gain):
    """Ordinary values within the bound that follows from the roundings that the kernels state, K's in the tcgen05 kernel among them."""
    cache, q, table, lens, offsets = attn_case(d + G, d, 1, G, [1500, 90], [rows, 1], 32, kind, gain=gain)
    out = R.kv4_attention(torch.as_tensor(cache, device="cuda"), q, ints(table), ints(lens), ints(offsets), rows)
    n = offsets[-1]
    o, tol = E.rounded_attention(cache, q[:n].double().cpu().numpy(), table, lens, offsets, True, d ** -0.5,
                                 torch.finfo(TYPES[kind]).eps / 2, G * rows > 32)
    worst = np.max(np.abs(out[:n].double().cpu().numpy() - o) / tol)
    assert worst <= 1, worst


# ------------------------------------------- edges of the tcgen05 attention
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 5, 16, 33, 100, 2 ** 31 - 1])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_window_of_many_rows(R, d, window, causal, kind):
    check_attn(R, attn_case(d + window, d, 2, 5, [200, 31, 4, 64], [3, 1, 4, 8], 16, kind), causal, window)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 3])
def test_many_rows_without_cells(R, d, window):
    """No cells at all, fewer cells than rows, no rows; more than 32 rows per kv head."""
    case = attn_case(3, d, 2, 16, [0, 2, 5, 40, -3], [2, 4, 0, 3, 1], 16, "bf16")
    got = check_attn(R, case, True, window)
    assert not got[:4].any() and got[4:6].any() and not got[-1].any()
    check_attn(R, case, False, window)


@pytest.mark.parametrize("kind,gain,scale", [("bf16", 1e-20, 1e19), ("bf16", 1e20, 1e-21), ("fp16", 1e-5, 2e4), ("fp16", 2e3, 1e-4),
                                             ("bf16", 0.0, 1.0), ("fp16", 8.0, 0.5)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_ranges_of_many_rows(R, kind, gain, scale, d):
    """(check_attn's bound does not know that this kernel rounds K to FP16.  That moves a score by up to scale * 2^-11 * sum |q k|: with queries
    of size 8 and a scale of 1/2 over 128 channels by 0.5 * 2^-11 * 128 * 8 * 0.8 * 0.8 = 0.16, where that bound has 2^-16 of scores of
    100 or 200, 0.003.  The reference here takes K rounded.)"""
    cache, q, table, lens, offsets = attn_case(1, d, 1, 20, [300], [2], 32, kind, gain=gain)
    st = status()
    out = R.kv4_attention(torch.as_tensor(cache, device="cuda"), q, ints(table), ints(lens), ints(offsets), 2, scale=scale, status=st)
    o, tol = E.rounded_attention(cache, q[:2].double().cpu().numpy(), table, lens, offsets, True, scale, torch.finfo(TYPES[kind]).eps / 2, True)
    worst = np.max(np.abs(out[:2].double().cpu().numpy() - o) / tol)
    assert int(st) == 0 and worst <= 1, worst


@pytest.mark.parametrize("vgain", [1e-4, 3e3])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_value_range_of_many_rows(R, vgain, d):
    check_attn(R, attn_case(2, d, 1, 5, [100], [8], 16, "bf16", vgain=vgain), True)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_strided_many_rows(R, d):
    """q inside a wider row, out inside another, and a row's neighbours left as they were."""
    cache, q, table, lens, offsets = attn_case(4, d, 2, 5, [50, 20], [8, 3], 16, "bf16")
    c, args, st = torch.as_tensor(cache, device="cuda"), (ints(table), ints(lens), ints(offsets), 8), status()
    plain = R.kv4_attention(c, q, *args)
    wide = torch.zeros((q.shape[0], 12, d), dtype=q.dtype, device="cuda")
    wide[:, 1:11] = q
    outw = torch.full((q.shape[0], 13, d), 3.0, dtype=q.dtype, device="cuda")
    R.kv4_attention(c, wide[:, 1:11], *args, out=outw[:, 2:12], status=st)
    assert torch.equal(outw[:11, 2:12], plain[:11]) and bool((outw[:, :2] == 3).all()) and bool((outw[:, 12:] == 3).all())
    assert bool((outw[11:] == 3).all()) and int(st) == 0


def test_reports_of_many_rows(R):
    cache, q, table, lens, offsets = attn_case(6, 64, 1, 40, [40, 20], [2, 1], 16, "fp16")
    c = torch.as_tensor(cache, device="cuda")

    def call(table=table, lens=lens, offsets=offsets, q=q, rows=2):
        st, out = status(), torch.full_like(q, 7.0)
        R.kv4_attention(c, q, ints(table), ints(lens), ints(offsets), rows, out=out, status=st)
        return int(st), out

    good = call()
    assert good[0] == 0
    st, out = call(rows=1)
    assert st == D.DFLASH_DEV_BAD_BLOCK and bool((out[:2] == 7).all()) and torch.equal(out[2], good[1][2])
    assert call(offsets=np.array([0, 2, 1]))[0] == D.DFLASH_DEV_BAD_BLOCK
    assert call(offsets=np.array([-1, 0, 1]))[0] == D.DFLASH_DEV_BAD_BLOCK
    assert call(offsets=np.array([0, 2, 99]), rows=3)[0] == D.DFLASH_DEV_BAD_BLOCK
    assert call(lens=np.array([1000, 20]))[0] & D.DFLASH_DEV_CAPACITY
    bad = table.copy()
    bad[0, 1] = -1
    st, out = call(table=bad)
    assert st & D.DFLASH_DEV_CAPACITY and torch.equal(out[2], good[1][2])
    nan = q.clone()
    nan[0, 0, 3] = float("nan")
    st, out = call(q=nan)
    assert st == D.DFLASH_DEV_NONFINITE and torch.equal(out[1:3], good[1][1:3])
    assert torch.equal(out[0, 1:], good[1][0, 1:])


# ------------------------------------------------------------- written bytes
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_written_bytes(R, d, kind):
    """Every byte of a written cell, codes and scales; only the sign of a zero scale is free."""
    rng = np.random.default_rng(d)
    n, heads, page = 96, 2, 32
    x = torch.as_tensor(rng.standard_normal((2, n, heads, d)) * np.exp(2 * rng.standard_normal((2, n, heads, 1))), device="cuda").to(TYPES[kind])
    x[:, 0] = 0
    x[:, 1] = 2.0 ** -24  # a scale below FP16's smallest
    cache = R.kv4_cache(n // page, page, heads, d)
    slots = rng.permutation(n).astype(np.int32)
    R.kv4_write(cache, x[0], x[1], ints(slots))
    want = np.zeros(tuple(cache.shape), np.uint8)
    V.store(want, slots, x[0].double().cpu().numpy(), x[1].double().cpu().numpy())
    got = cache.cpu().numpy()
    scales = np.zeros(18 * d, bool)
    for at in V.word_places(d)[2:]:
        scales[at] = scales[at + 1] = True
    assert np.array_equal(got[..., ~scales], want[..., ~scales])
    a, b = (np.ascontiguousarray(y[..., scales]).view(np.uint16) for y in (got, want))
    assert np.array_equal(np.where(a == 0x8000, 0, a), np.where(b == 0x8000, 0, b))


# ------------------------------------------------------------- largest calls
@pytest.mark.parametrize("d,heads,G,rows", [(256, 1, 5, 8), (64, 1, 5, 8), (256, 1, 4, 8), (128, 2, 1, 1)])
def test_most_sequences(R, d, heads, G, rows):
    """1024 sequences, some without rows or cells, rows that begin behind others of no sequence."""
    rng = np.random.default_rng(d)
    lens = rng.integers(0, 24, 1024)
    many = rng.integers(0, rows + 1, 1024)
    cache, q, table, lens, offsets = attn_case(5, d, heads, G, lens.tolist(), many.tolist(), 16, "bf16")
    check_attn(R, (cache, q, table, lens, offsets), True, max_rows=rows)
    first = 3
    moved = torch.cat([torch.full_like(q[:first], float("nan")), q])
    st, out = status(), torch.full_like(moved, 7.0)
    args = torch.as_tensor(cache, device="cuda"), ints(table), ints(lens)
    want = R.kv4_attention(args[0], q, args[1], args[2], ints(offsets), rows)
    R.kv4_attention(args[0], moved, args[1], args[2], ints(offsets + first), rows, out=out, status=st)
    n = int(offsets[-1])
    assert int(st) == 0 and torch.equal(out[first: first + n], want[:n])
    assert bool((out[:first] == 7).all()) and bool((out[first + n:] == 7).all())


@pytest.mark.parametrize("d", [64, 256])
def test_most_heads(R, d):
    check_attn(R, attn_case(7, d, 256, 1, [20, 3], [1, 2], 16, "fp16"), True)


def test_cells_and_scores_in_a_graph(R):
    """Writing, reading back and scoring captured once and replayed with other inputs."""
    rng = np.random.default_rng(2)
    cache, st = R.kv4_cache(8, 16, 2, 64), status()
    both = torch.zeros((100, 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    x, tokens, slots = torch.zeros((3, 70001), device="cuda"), ints(np.zeros(3)), ints(np.zeros(100))
    k, v = both[:, 0], both[:, 1].contiguous()

    def step():
        R.kv4_write(cache, k, v, slots, status=st)
        return R.kv4_read(cache, slots, status=st) + R.token_logprobs(x, tokens, top_k=4, status=st)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    slots.copy_(ints(np.arange(100)))
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        both.copy_(torch.as_tensor(rng.standard_normal(both.shape), device="cuda"))
        v.copy_(both[:, 1])
        slots.copy_(ints(rng.permutation(128)[:100]))
        x.copy_(torch.as_tensor(rng.standard_normal(x.shape), device="cuda"))
        tokens.copy_(ints(rng.integers(0, 70001, 3)))
        graph.replay()
        for a, b in zip(got, (y.clone() for y in step())):
            assert torch.equal(a, b)
        for a, b in zip(got, (k, v)):
            assert np.array_equal(a.double().cpu().numpy(), V.dequantise(*V.quantise(b.double().cpu().numpy())))
        z = x.double()
        assert np.allclose(got[2].cpu().numpy(), (z.gather(1, tokens.long()[:, None])[:, 0] - z.logsumexp(1)).cpu().numpy(), rtol=2.0 ** -18, atol=0)
    assert int(st) == 0
