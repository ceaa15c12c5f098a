"""Host-side checks of the verify-step operators beyond their plain refusals: sizes of more than 32 bits, the largest softmax
scale.  No GPU is used."""
import ctypes

import numpy as np
import pytest

import dflash_block_drafter_gb300 as D
import verify_exact as E
import verify_ref as V
from test_verify_host import _cache, lib  # noqa: F401

WIDE = 2 ** 32  # a size that 32 bits would cut to 0
FAR = 4096      # an address that is never read: the calls are refused before anything is enqueued


@pytest.mark.parametrize("size", [WIDE, WIDE + 8, 2 ** 31, -WIDE + 8])
def test_sizes_beyond_32_bits(lib, size):  # noqa: F811
    c = _cache()

    def pages(n_seq=1, page=16, n_pages=8, width=4, cap=8):
        D.dflash_page_tables(FAR, FAR, n_seq, page, n_pages, FAR, FAR, FAR, width, FAR, FAR, FAR, FAR, FAR, 0, cap)

    def attention(tokens=1, nq=8, n_seq=1, rows=1, width=4, window=0):
        D.dflash_kv4_attention(c, FAR, FAR, D.DFLASH_T_BF16, 1024, 1024, tokens, nq, n_seq, rows, FAR, FAR, FAR, width, True, window, 1.0, FAR,
                               1 << 30)

    calls = [lambda: pages(n_seq=size), lambda: pages(page=size), lambda: pages(n_pages=size), lambda: pages(width=size),
             lambda: pages(cap=size), lambda: attention(tokens=size), lambda: attention(nq=size), lambda: attention(n_seq=size),
             lambda: attention(rows=size), lambda: attention(width=size), lambda: attention(window=size),
             lambda: D.dflash_kv4_write(c, FAR, FAR, D.DFLASH_T_BF16, 256, 256, FAR, size),
             lambda: D.dflash_kv4_read(c, FAR, size, FAR, FAR),
             lambda: D.dflash_token_logprobs(FAR, D.DFLASH_T_BF16, WIDE * 2, size, 8, 0, 0, FAR, 0, 0, 0),
             lambda: D.dflash_token_logprobs(FAR, D.DFLASH_T_BF16, WIDE * 2, 1, size, 0, 0, FAR, 0, 0, 0),
             lambda: D.dflash_token_logprobs(FAR, D.DFLASH_T_BF16, WIDE * 2, 1, 8, 0, 0, FAR, size, FAR, FAR)]
    for i, call in enumerate(calls):
        with pytest.raises(D.DflashError) as e:
            call()
        assert e.value.status == D.DFLASH_ERR_INVALID_ARG, i
    for kw in ("n_pages", "page_size", "n_kv_heads", "head_dim"):
        assert D.dflash_kv4_bytes(**{**dict(n_pages=8, page_size=64, n_kv_heads=2, head_dim=128), kw: size}) == 0
    for kw in ("n_q_heads", "n_seq", "max_rows", "table_stride"):
        assert D.dflash_kv4_attention_workspace(c, **{**dict(n_q_heads=8, n_seq=1, max_rows=1, table_stride=4), kw: size}) == 0


def test_largest_scale(lib):  # noqa: F811
    """A scale whose product with log2(e) is infinite in FP32 would give every row the largest factor there is."""
    c, far = _cache(), ctypes.c_void_p(FAR)

    def call(scale):
        return lib.dflash_kv4_attention(ctypes.byref(c), far, far, D.DFLASH_T_BF16, 1024, 1024, 0, 8, 1, 1, far, far, far, 4, 1, 0, scale,
                                        None, 0, None, None)

    assert call(2.0 ** 127) == D.DFLASH_OK  # no tokens: nothing to do
    for scale in (2.0 ** 127 * (1 + 2.0 ** -20), 3e38):
        assert call(scale) == D.DFLASH_ERR_INVALID_ARG


# ---------------------------------------------------------- the exact cases
@pytest.mark.parametrize("d,n", [(64, 30000), (128, 30000), (256, 20000)])
@pytest.mark.parametrize("cells", [64, 16])
def test_exact_cases_show_a_lost_tile(d, n, cells):
    """A tile (or group) of cells left out, taken twice or replaced by an earlier one passes the bound by far, wherever it lies."""
    rng = np.random.default_rng(d)
    k, v = E.cells(rng, n, 1, d)
    q = E.queries(rng, 2, 2, d)
    o, spread = E.attend(k, v, q, False)
    tol = E.tolerance(o, spread, 2.0 ** -11)
    for at in (0, n // 3 // cells * cells, (n - 1) // cells * cells):
        mine = slice(at, at + cells)
        for weight in (-np.inf, 1.0):
            bias = np.zeros(n)
            bias[mine] = weight
            assert np.all(np.max(np.abs(E.attend(k, v, q, False, bias=bias)[0] - o) / tol, -1) > 5)
        early = slice(at - 3 * cells, at - 2 * cells) if at else slice(n - 5 * cells, n - 4 * cells)
        for x in (k, v):
            size = x[mine].shape[0]
            kept = x[mine].copy()
            x[mine] = x[early][:size]
            assert np.all(np.max(np.abs(E.attend(k, v, q, False)[0] - o) / tol, -1) > 2.5)
            x[mine] = kept


def test_exact_cases_are_exact():
    rng = np.random.default_rng(0)
    for d in (64, 128, 256):
        k, v = E.cells(rng, 40, 2, d)
        for x in (k, v):
            codes, scales = V.quantise(x.astype(np.float64))
            assert np.all(scales == 1) and np.array_equal(V.dequantise(codes, scales), x)
        s = np.einsum("thd,nd->thn", E.queries(rng, 3, 4, d), k[:, 0].astype(np.float64))
        assert s.min() >= -3 and s.max() <= 0
