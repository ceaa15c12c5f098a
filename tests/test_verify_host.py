"""Host-side checks of the verify-step operators: argument refusals of the C ABI and of the torch wrappers, and the
reference forms against simple facts.  No GPU is used."""
import ctypes
import os
import shutil

import numpy as np
import pytest

import dflash_block_drafter_gb300 as D
import verify_ref as V

P = ctypes.c_void_p
FAKE = P(4096)  # never read: the calls are refused before anything is enqueued


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(D.LIB_PATH):
        if not shutil.which("nvcc") and not os.path.exists("/usr/local/cuda/bin/nvcc"):
            pytest.skip("nvcc unavailable and libdflash not built")
    from dflash_block_drafter_gb300 import build
    build.build()
    return D.load_library()


def _cache(data=4096, n_pages=8, page_size=64, n_kv_heads=2, head_dim=128):
    return D.DflashKv4Cache(data, n_pages, page_size, n_kv_heads, head_dim)


BAD_CACHES = [
    (dict(data=0), D.DFLASH_ERR_INVALID_ARG), (dict(data=4104), D.DFLASH_ERR_INVALID_ARG),
    (dict(n_pages=0), D.DFLASH_ERR_INVALID_ARG), (dict(n_kv_heads=0), D.DFLASH_ERR_INVALID_ARG),
    (dict(n_kv_heads=257), D.DFLASH_ERR_INVALID_ARG), (dict(page_size=8), D.DFLASH_ERR_UNSUPPORTED),
    (dict(page_size=48), D.DFLASH_ERR_UNSUPPORTED), (dict(page_size=512), D.DFLASH_ERR_UNSUPPORTED),
    (dict(head_dim=96), D.DFLASH_ERR_UNSUPPORTED), (dict(n_pages=1 << 25), D.DFLASH_ERR_CAPACITY),
]


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_cache_check(lib, kw, want):
    c = _cache(**kw)
    assert D.dflash_kv4_check(c) == want
    r = ctypes.byref(c)
    assert lib.dflash_kv4_write(r, FAKE, FAKE, D.DFLASH_T_BF16, 256, 256, FAKE, 1, None, None) == want
    assert lib.dflash_kv4_read(r, FAKE, 1, FAKE, FAKE, None, None) == want
    assert lib.dflash_kv4_attention(r, FAKE, FAKE, D.DFLASH_T_BF16, 1024, 1024, 1, 8, 1, 1, FAKE, FAKE, FAKE, 1, 1, 0, 1.0,
                                    FAKE, 1 << 30, None, None) == want
    assert D.dflash_kv4_attention_workspace(c, 8, 1, 1, 1) == 0


def test_cache_sizes(lib):
    assert D.dflash_kv4_check(_cache()) == D.DFLASH_OK
    assert lib.dflash_kv4_check(None) == D.DFLASH_ERR_INVALID_ARG
    assert D.dflash_kv4_bytes(8, 64, 2, 128) == 8 * 64 * 2 * 144  # 144 bytes a cell and head: 1.125 per channel
    assert D.dflash_kv4_bytes(8, 40, 2, 128) == 0


def test_write_and_read_refusals(lib):
    c = ctypes.byref(_cache())
    inv, uns = D.DFLASH_ERR_INVALID_ARG, D.DFLASH_ERR_UNSUPPORTED
    w = lib.dflash_kv4_write
    assert w(c, FAKE, FAKE, D.DFLASH_T_FP32, 256, 256, FAKE, 1, None, None) == uns
    assert w(c, FAKE, FAKE, 9, 256, 256, FAKE, 1, None, None) == uns
    assert w(c, FAKE, FAKE, D.DFLASH_T_BF16, 256, 256, FAKE, -1, None, None) == inv
    for k, v, ks, vs, slots in ((None, FAKE, 256, 256, FAKE), (FAKE, None, 256, 256, FAKE), (FAKE, FAKE, 256, 256, None),
                                (FAKE, FAKE, 255, 256, FAKE), (FAKE, FAKE, 256, 248, FAKE), (FAKE, FAKE, 260, 256, FAKE),
                                (P(4098), FAKE, 256, 256, FAKE), (FAKE, P(4104), 256, 256, FAKE)):
        assert w(c, k, v, D.DFLASH_T_FP16, ks, vs, slots, 1, None, None) == inv
    assert w(c, None, None, D.DFLASH_T_FP16, 0, 0, None, 0, None, None) == D.DFLASH_OK  # no rows: nothing to do
    r = lib.dflash_kv4_read
    assert r(c, None, 1, FAKE, FAKE, None, None) == inv
    assert r(c, FAKE, 1, P(4112), FAKE, None, None) == inv
    assert r(c, FAKE, -1, FAKE, FAKE, None, None) == inv
    assert r(c, FAKE, 0, FAKE, FAKE, None, None) == D.DFLASH_OK
    assert r(c, FAKE, 3, None, None, None, None) == D.DFLASH_OK


def test_attention_refusals(lib):
    good = dict(c=ctypes.byref(_cache()), q=FAKE, out=FAKE, type=D.DFLASH_T_BF16, qs=1024, os=1024, tokens=1, nq=8, n_seq=1, rows=1,
                off=FAKE, kv=FAKE, table=FAKE, width=4, causal=1, window=0, scale=0.1, ws=FAKE, wsb=1 << 30, st=None, stream=None)

    def call(**kw):
        return lib.dflash_kv4_attention(*{**good, **kw}.values())

    inv = D.DFLASH_ERR_INVALID_ARG
    for kw in (dict(q=None), dict(out=None), dict(off=None), dict(kv=None), dict(table=None), dict(q=P(4104)), dict(out=P(4104)),
               dict(qs=1016), dict(os=1016), dict(qs=1028), dict(os=1028), dict(tokens=-1), dict(nq=7), dict(nq=0), dict(n_seq=0),
               dict(rows=0), dict(rows=9), dict(width=0), dict(window=-1), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(**kw) == inv, kw
    assert call(type=D.DFLASH_T_FP32) == D.DFLASH_ERR_UNSUPPORTED
    assert call(nq=34, rows=8, qs=34 * 128, os=34 * 128) == D.DFLASH_ERR_UNSUPPORTED  # 17 heads of a group x 8 rows > 128
    assert call(n_seq=1025) == D.DFLASH_ERR_CAPACITY
    assert call(width=1 << 25) == D.DFLASH_ERR_CAPACITY  # positions beyond 31 bits
    assert D.dflash_kv4_attention_workspace(_cache(), 8, 1, 1, 1 << 25) == 0
    assert call(tokens=0) == D.DFLASH_OK


def test_page_tables_refusals(lib):
    good = dict(lengths=FAKE, new=FAKE, n_seq=2, page=16, pages=8, hi=FAKE, ho=FAKE, table=FAKE, width=4, ring=FAKE, ri=FAKE, ro=FAKE,
                off=FAKE, slots=FAKE, pos=None, cap=8, st=None, stream=None)

    def call(**kw):
        return lib.dflash_page_tables(*{**good, **kw}.values())

    for name in ("lengths", "new", "hi", "ho", "table", "ring", "ri", "ro", "off", "slots"):
        assert call(**{name: None}) == D.DFLASH_ERR_INVALID_ARG, name
    for kw in (dict(n_seq=0), dict(width=0), dict(pages=0), dict(cap=-1)):
        assert call(**kw) == D.DFLASH_ERR_INVALID_ARG, kw
    for kw in (dict(page=8), dict(page=24), dict(page=512)):
        assert call(**kw) == D.DFLASH_ERR_UNSUPPORTED, kw
    assert call(n_seq=4097) == D.DFLASH_ERR_CAPACITY
    assert call(pages=1 << 27) == D.DFLASH_ERR_CAPACITY
    assert call(n_seq=4096, width=1 << 19) == D.DFLASH_ERR_CAPACITY


def test_logprobs_refusals(lib):
    good = dict(x=FAKE, type=D.DFLASH_T_FP32, stride=100, rows=1, vocab=100, tok=FAKE, lp=FAKE, ent=FAKE, k=4, ids=FAKE, top=FAKE,
                st=None, stream=None)

    def call(**kw):
        return lib.dflash_token_logprobs(*{**good, **kw}.values())

    inv = D.DFLASH_ERR_INVALID_ARG
    for kw in (dict(x=None), dict(x=P(4098)), dict(stride=99), dict(rows=-1), dict(vocab=0), dict(k=-1), dict(tok=None), dict(lp=None),
               dict(ids=None), dict(top=None), dict(tok=None, lp=None, ent=None, k=0)):
        assert call(**kw) == inv, kw
    assert call(type=7) == D.DFLASH_ERR_UNSUPPORTED
    assert call(k=33) == D.DFLASH_ERR_CAPACITY
    assert call(rows=0) == D.DFLASH_OK


def test_torch_wrappers_refuse():
    torch = pytest.importorskip("torch")
    from dflash_block_drafter_gb300 import runtime as R
    cache = torch.zeros((2, 1, 1, 18 * 64), dtype=torch.uint8)  # on the CPU
    rows = torch.zeros((1, 1, 64), dtype=torch.bfloat16)
    one = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: R.kv4_write(cache, rows, rows, one), lambda: R.kv4_read(cache, one),
                 lambda: R.kv4_attention(cache, rows, one[None], one, torch.zeros(2, dtype=torch.int32), 1),
                 lambda: R.token_logprobs(torch.zeros((1, 8))),
                 lambda: R.page_tables(one, one, one, one[None], one, torch.zeros(2, dtype=torch.int32), 16, 4)):
        with pytest.raises(D.DflashError) as e:
            call()
        assert e.value.status == D.DFLASH_ERR_INVALID_ARG


# ------------------------------------------------------ the reference forms
@pytest.mark.parametrize("d", [64, 128, 256])
def test_reference_places_fill_a_group(d):
    kc, vc, ks, vs = V.word_places(d)
    every = np.concatenate([kc.ravel(), vc.ravel(), ks.ravel(), ks.ravel() + 1, vs.ravel(), vs.ravel() + 1])
    assert np.array_equal(np.sort(every), np.arange(18 * d))


def test_reference_quantiser():
    x = np.zeros((1, 64))
    x[0, :4] = [-8, 8, 4, 0.5]  # the first of equals is negative: d = 1
    codes, d = V.quantise(x)
    assert d[0, 0] == 1 and codes[0, :4].tolist() == [0, 15, 12, 8]  # 8 is beyond code 15, 0.5 goes to the even 0
    assert d[0, 1] == 0 and set(codes[0, 32:].tolist()) == {8}
    rng = np.random.default_rng(0)
    y = rng.standard_normal((50, 64)).astype(np.float16)
    codes, d = V.quantise(y)
    err = np.abs(V.dequantise(codes, d) - y)
    assert np.all(err <= np.repeat(np.abs(d.astype(np.float64)), 32, -1) * (1 + 2.0 ** -8))  # half a step; a whole one at the clamp


def test_reference_store_and_load():
    rng = np.random.default_rng(1)
    cache = rng.integers(0, 256, (3, 2, 2, 18 * 64), dtype=np.uint8)
    k, v = rng.standard_normal((2, 5, 2, 64))
    slots = np.array([0, 95, -1, 17, 33])
    V.store(cache, slots, k, v)
    for x, y in zip((k, v), V.load(cache, slots)):
        codes, d = V.quantise(x)
        want = V.dequantise(codes, d)
        want[2] = 0
        assert np.array_equal(want, y)


def test_reference_pages():
    # two pages are left; request 1 needs one, request 2 needs two: request 2 gets none, request 3 needs none
    held, table, ring, state, off, slots, pos, flag = V.page_tables(
        [16, 15, 16, 5, 0], [1, 2, 32, 3, 0], np.array([2, 1, 1, 1, 2]), np.array([[4, 5, -1], [6, -1, -1], [7, -1, -1], [8, -1, -1], [9, 3, -1]]),
        np.array([0, 1, 2, -1, -1, -1, -1, -1, -1, -1]), np.array([0, 2]), 16, 40)
    assert flag and held.tolist() == [2, 2, 1, 1, 0] and table[1].tolist() == [6, 0, -1]
    assert state.tolist() == [1, 3] and ring[[1, 2, 3]].tolist() == [1, 9, 3]
    assert off.tolist() == [0, 1, 3, 35, 38, 38]
    assert slots[:4].tolist() == [5 * 16, 6 * 16 + 15, 0, -1] and slots[35:39].tolist() == [8 * 16 + 5, 8 * 16 + 6, 8 * 16 + 7, -1]
    assert pos[1:3].tolist() == [15, 16] and pos[38] == -1
