"""The verify-step operators on the GPU where their rules meet: pages given back before a window, rows and cells without
weight, far apart scores, and the edges of the tcgen05 attention kernel (more than 32 rows per kv head)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import dflash_block_drafter_gb300 as D  # noqa: E402
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
