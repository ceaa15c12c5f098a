"""Host-side checks of the sampling step's operators: argument refusals of the C ABI and of the torch wrappers, the rotation
table.  No GPU is used."""
import ctypes
import math
from fractions import Fraction

import pytest

import dflash_block_drafter_gb300 as D
from test_verify_host import FAKE, P, _cache, lib  # noqa: F401

INV, UNS, CAP = D.DFLASH_ERR_INVALID_ARG, D.DFLASH_ERR_UNSUPPORTED, D.DFLASH_ERR_CAPACITY
WIDE = [2 ** 32, 2 ** 32 + 8, 2 ** 31, -2 ** 32 + 8]


def refused(call):
    with pytest.raises(D.DflashError) as e:
        call()
    return e.value.status


# ------------------------------------------------------------- norm and rotation
PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


def test_rotation_table(lib):  # noqa: F811
    freqs = [1e7 ** (-2.0 * j / 256) for j in range(128)] + [0.0, 6.2, 6.3, 1000.0, -0.25, 1e-300]
    for f, t in zip(freqs, D.dflash_rope_turns(freqs)):
        turn = Fraction(f) / (2 * PI)
        off = (Fraction(t, 1 << 64) - turn) % 1
        off = min(off, 1 - off)
        # the quotient and pi are off by 2^-53 each relative to the turns, the table by 2^-64, and where whole turns are taken off a negative one by 2^-53
        assert off <= Fraction(2) ** -52 * abs(turn) + Fraction(2) ** -53 * (f < 0) + Fraction(2) ** -64, f
    assert D.dflash_rope_turns([]) == []
    for bad in (math.inf, -math.inf, math.nan):
        assert refused(lambda: D.dflash_rope_turns([1.0, bad])) == INV
    assert lib.dflash_rope_turns(None, 1, FAKE) == INV and lib.dflash_rope_turns(None, -1, None) == INV


GOOD_ROPE = dict(q=FAKE, qo=FAKE, qs=1024, qos=1024, nq=8, k=FAKE, ko=FAKE, ks=256, kos=256, nk=2, d=128, type=D.DFLASH_T_BF16, n=4, qw=None, kw=None,
                 eps=1e-6, pos=FAKE, ps=4, n_axes=1, axes=None, turns=FAKE, rot=128, st=None, stream=None)


def test_norm_rope_refusals(lib):  # noqa: F811
    def call(**kw):
        return lib.dflash_qk_norm_rope(*{**GOOD_ROPE, **kw}.values())

    for kw in (dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(q=P(4104)), dict(qo=P(4104)), dict(k=P(4098)), dict(ko=P(4104)),
               dict(qs=1016), dict(qos=1016), dict(ks=248), dict(kos=248), dict(qs=1028), dict(kos=260), dict(n=-1), dict(nq=-1), dict(nk=-1),
               dict(eps=-1e-6), dict(eps=math.inf), dict(eps=math.nan), dict(pos=None), dict(turns=None), dict(turns=P(4100)), dict(rot=-16), dict(rot=144),
               dict(n_axes=2, axes=None), dict(n_axes=2, axes=FAKE, ps=3)):
        assert call(**kw) == INV, kw
    for kw in (dict(type=D.DFLASH_T_FP32), dict(type=7), dict(d=96), dict(d=512, qs=4096, qos=4096, ks=1024, kos=1024), dict(rot=24), dict(rot=8),
               dict(n_axes=0), dict(n_axes=5, axes=FAKE)):
        assert call(**kw) == UNS, kw
    assert call(nq=65537, qs=1 << 30, qos=1 << 30) == CAP
    assert call(n=0) == D.DFLASH_OK and call(nq=0, nk=0) == D.DFLASH_OK


@pytest.mark.parametrize("size", WIDE)
def test_norm_rope_sizes_beyond_32_bits(lib, size):  # noqa: F811
    for name in ("nq", "nk", "d", "n", "n_axes", "rot"):
        args = {**GOOD_ROPE, name: size}
        args = [a.value if isinstance(a, ctypes.c_void_p) else 0 if a is None else a for a in args.values()]
        assert refused(lambda: D.dflash_qk_norm_rope(*args)) == INV, name


# --------------------------------------------------------------- shared prefixes
GOOD_PREFIX = dict(c=ctypes.byref(_cache()), q=FAKE, out=FAKE, type=D.DFLASH_T_BF16, qs=1024, os=1024, tokens=4, nq=8, groups=1, goff=FAKE, plen=FAKE, ptable=FAKE,
                   pwidth=4, n_seq=2, rows=2, off=FAKE, kv=FAKE, table=FAKE, width=4, causal=1, scale=0.1, ws=FAKE, wsb=1 << 40, st=None, stream=None)


def test_prefix_attention_refusals(lib):  # noqa: F811
    def call(**kw):
        return lib.dflash_kv4_prefix_attention(*{**GOOD_PREFIX, **kw}.values())

    for kw in (dict(q=None), dict(out=None), dict(goff=None), dict(plen=None), dict(ptable=None), dict(off=None), dict(kv=None), dict(table=None),
               dict(q=P(4104)), dict(out=P(4104)), dict(qs=1016), dict(os=1016), dict(qs=1028), dict(os=1028), dict(tokens=-1), dict(nq=7), dict(nq=0),
               dict(groups=0), dict(groups=-1), dict(pwidth=0), dict(n_seq=0), dict(rows=0), dict(rows=9), dict(width=0), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=math.nan), dict(scale=math.inf), dict(scale=3e38)):
        assert call(**kw) == INV, kw
    assert call(type=D.DFLASH_T_FP32) == UNS
    assert call(nq=34, rows=8, qs=34 * 128, os=34 * 128) == UNS  # 17 heads of a group x 8 rows > 128
    for kw in (dict(groups=1025), dict(n_seq=1025), dict(pwidth=1 << 25), dict(width=1 << 25), dict(tokens=1 << 28)):
        assert call(**kw) == CAP, kw
    assert call(tokens=0) == D.DFLASH_OK
    work = dict(n_tokens=4, n_q_heads=8, n_groups=1, prefix_stride=4, n_seq=2, max_rows=2, table_stride=4)
    for kw in (dict(n_q_heads=7), dict(n_groups=0), dict(n_groups=1025), dict(prefix_stride=1 << 25), dict(n_tokens=-1)):
        assert D.dflash_kv4_prefix_attention_workspace(_cache(), **{**work, **kw}) == 0
    assert D.dflash_kv4_prefix_attention_workspace(_cache(head_dim=96), **work) == 0
    for bad, want in ((dict(data=4104), INV), (dict(head_dim=96), UNS)):
        assert call(c=ctypes.byref(_cache(**bad))) == want


@pytest.mark.parametrize("size", WIDE)
def test_prefix_attention_sizes_beyond_32_bits(lib, size):  # noqa: F811
    for name in ("tokens", "nq", "groups", "pwidth", "n_seq", "rows", "width"):
        args = {**GOOD_PREFIX, "c": _cache(), name: size}
        args = [a.value if isinstance(a, ctypes.c_void_p) else 0 if a is None else a for a in args.values()]
        assert refused(lambda: D.dflash_kv4_prefix_attention(*args)) == INV, name
    work = dict(n_tokens=4, n_q_heads=8, n_groups=1, prefix_stride=4, n_seq=2, max_rows=2, table_stride=4)
    for name in work:
        assert D.dflash_kv4_prefix_attention_workspace(_cache(), **{**work, name: size}) == 0


# --------------------------------------------------------------------- sampling
GOOD_SAMPLE = dict(x=FAKE, type=D.DFLASH_T_BF16, stride=100, n=2, vocab=100, u=FAKE, t=None, k=None, p=None, low=None, tokens=FAKE, lp=None, kept=None,
                   st=None, stream=None)


def test_sample_refusals(lib):  # noqa: F811
    def call(**kw):
        return lib.dflash_sample_tokens(*{**GOOD_SAMPLE, **kw}.values())

    for kw in (dict(x=None), dict(x=P(4097)), dict(type=D.DFLASH_T_FP32, x=P(4098)), dict(stride=99), dict(n=-1), dict(vocab=0), dict(u=None),
               dict(tokens=None)):
        assert call(**kw) == INV, kw
    assert call(type=3) == UNS
    assert call(vocab=(1 << 19) + 1, stride=1 << 20) == CAP and call(n=(1 << 24) + 1) == CAP
    assert call(n=0) == D.DFLASH_OK


@pytest.mark.parametrize("size", WIDE)
def test_sample_sizes_beyond_32_bits(lib, size):  # noqa: F811
    for name in ("n", "vocab"):
        args = {**GOOD_SAMPLE, "stride": 2 ** 34, name: size}
        args = [a.value if isinstance(a, ctypes.c_void_p) else 0 if a is None else a for a in args.values()]
        assert refused(lambda: D.dflash_sample_tokens(*args)) == INV, name


def test_torch_wrappers_refuse():
    torch = pytest.importorskip("torch")
    from dflash_block_drafter_gb300 import runtime as R
    rows = torch.zeros((1, 1, 64), dtype=torch.bfloat16)  # on the CPU
    one = torch.zeros(1, dtype=torch.int32)
    cache = torch.zeros((2, 1, 1, 18 * 64), dtype=torch.uint8)
    two = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: R.qk_norm_rope(rows, rows, one, torch.zeros(32, dtype=torch.int64)),
                 lambda: R.sample_tokens(torch.zeros((1, 8)), torch.zeros(1)),
                 lambda: R.kv4_prefix_attention(cache, rows, one[None], one, two, one[None], one, two, 1)):
        assert refused(call) == INV


def test_wrappers_ask_torch_for_the_current_device(monkeypatch):
    """By its public call: a private binding may be gone in another release."""
    torch = pytest.importorskip("torch")
    from dflash_block_drafter_gb300 import runtime as R
    monkeypatch.delattr(torch._C, "_cuda_getDevice", raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert R._elsewhere(torch.device("cuda", 1), None) is None
    assert isinstance(R._elsewhere(torch.device("cuda", 0), None), torch.cuda.device)
