"""Tokens drawn from logits on the GPU: ids and counts equal to the 64-bit form's (sampling_ref.py) on every row, whatever the filters."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import dflash_block_drafter_gb300 as D  # noqa: E402
import gpu_helpers as H  # noqa: E402
import sampling_ref as S  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def R():
    H.need_gpu()
    H.build_lib()
    from dflash_block_drafter_gb300 import runtime
    return runtime


def ints(x):
    return None if x is None else torch.as_tensor(np.asarray(x, np.int32), device="cuda")


def floats(x):
    return None if x is None else torch.as_tensor(np.asarray(x, np.float32), device="cuda")


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def f32(x):
    return None if x is None else np.asarray(x, np.float32)


def check(R, x, uniform, temperature=None, top_k=None, top_p=None, min_p=None, want_status=0, rows=slice(None)):
    """x: a tensor of logits on the device.  Weights are right to 2^-43 and the form above to 2^-50 or so: what a decision is about lies
    further apart in these inputs, which `near` shows, or is equal in both."""
    uniform, temperature, top_p, min_p = (f32(v) for v in (uniform, temperature, top_p, min_p))
    st = status()
    token, logp, kept = R.sample_tokens(x, floats(uniform), floats(temperature), ints(top_k), floats(top_p), floats(min_p), status=st)
    token, logp, kept = (v.cpu().numpy()[rows] for v in (token, logp, kept))
    assert int(st) == want_status
    pick = lambda v: None if v is None else np.asarray(v)[rows]  # noqa: E731
    t, lp, n, near = S.sample(x.double().cpu().numpy()[rows], *(pick(v) for v in (uniform, temperature, top_k, top_p, min_p)))
    clear = near > 2.0 ** -42
    assert clear.all() or near[~clear].max() == 0, near.min()
    assert np.array_equal(token, t), np.flatnonzero(token != t)
    assert np.array_equal(kept, n), (kept[kept != n], n[kept != n])
    # an FP32 difference of the logits, its product and a logarithm, 2^-22 each, of a part that may be larger than the result
    with np.errstate(invalid="ignore"):
        size = np.abs(lp) + np.abs(np.log(np.maximum(n, 1)))
        assert np.all((np.abs(logp - lp) <= 2.0 ** -21 * (1 + size)) | (logp == lp))
    return token, logp, kept


def logits(rng, rows, vocab, kind, spread=1.0):
    z = rng.standard_normal((rows, vocab))
    x = (2 * z + 0.25 * z ** 3) * spread
    return torch.as_tensor(x, device="cuda").to(TYPES[kind])


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (5, 7), (4, 33), (9, 1023), (3, 1024), (2, 4099), (70, 5000), (8, 40000), (3, 151936), (200, 30011)])
@pytest.mark.parametrize("mode", ["plain", "k", "p", "min", "all"])
def test_draws(R, kind, rows, vocab, mode):
    rng = np.random.default_rng(rows + vocab)
    x = logits(rng, rows, vocab, kind, rng.uniform(0.2, 1.0, (rows, 1)))
    t = rng.uniform(0.3, 1.5, rows)
    k = np.exp(rng.uniform(0, np.log(vocab + 2), rows)).astype(int) if mode in ("k", "all") else None
    p = rng.uniform(0.3, 1.0, rows) if mode in ("p", "all") else None
    low = np.exp(rng.uniform(-12, 0, rows)) if mode in ("min", "all") else None
    check(R, x, rng.random(rows), t, k, p, low)


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab", [600, 151936])
def test_settings_by_row(R, kind, vocab):
    """Each filter on for some rows and off for others, greedy rows among them; filters that keep one token, or all but one."""
    rng = np.random.default_rng(vocab)
    n = 48
    x = logits(rng, n, vocab, kind)
    t = np.where(rng.random(n) < 0.2, 0, rng.uniform(0.2, 2, n))
    k = rng.choice([0, -3, 1, 2, 50, vocab - 1, vocab, vocab + 1, 2 ** 31 - 1], n)
    p = rng.choice([1.0, 2.0, 0.0, -1.0, 1e-9, 0.5, 0.95, 1 - 2.0 ** -24], n)
    low = rng.choice([0.0, -1.0, 1.0, 1e-30, 0.05], n)
    check(R, x, rng.random(n), t, k, p, low)


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab", [1, 64, 1024, 32768, 2 ** 19])
def test_equal_logits(R, kind, vocab):
    """Weights of 1: the token is the whole part of u times the vocabulary, at its borders too, and no filter parts equals."""
    x = torch.full((9, vocab), -2.5, dtype=TYPES[kind], device="cuda")
    step = 1.0 / max(vocab, 4)
    u = np.array([0, step, 0.25, 0.5, 0.5 - step, 0.75, 1 - step, 1 - 2.0 ** -24, 2.0 ** -30])
    for kw in ({}, dict(top_k=[1] * 9), dict(top_p=[0.01] * 9), dict(min_p=[1.0] * 9), dict(top_k=[3] * 9, top_p=[0.5] * 9)):
        token, logp, kept = R.sample_tokens(x, floats(u), floats([0.7] * 9), ints(kw.get("top_k")), floats(kw.get("top_p")), floats(kw.get("min_p")))
        assert token.tolist() == np.floor(f32(u).astype(float) * vocab).astype(int).tolist()
        assert kept.tolist() == [vocab] * 9 and np.allclose(logp.cpu().numpy(), -np.log(vocab), rtol=2.0 ** -22, atol=0)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
def test_few_levels(R, kind):
    """Logits of a few values, hundreds of tokens each, zeros of both signs among them."""
    rng = np.random.default_rng(3)
    v = rng.choice([-4.0, -1.0, -0.0, 0.0, 0.5, 2.0], (24, 3001))
    x = torch.as_tensor(v, device="cuda").to(TYPES[kind])
    check(R, x, rng.random(24), rng.uniform(0.5, 2, 24), rng.integers(1, 3001, 24), rng.uniform(0.05, 1, 24), np.exp(-rng.uniform(0, 8, 24)))
    zeros = torch.as_tensor(np.where(rng.random((4, 100)) < 0.5, 0.0, -0.0), device="cuda").to(TYPES[kind])
    assert R.sample_tokens(zeros, floats([0.0] * 4), floats([0.0, 1, 1, 1]), top_k=ints([0, 1, 0, 5]))[0].tolist() == [0] * 4


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab", [90, 500, 5000, 100003])
@pytest.mark.parametrize("small", [20, 150, 600])
def test_smallest_numbers(R, kind, vocab, small):
    """Numbers about and below the weights of single tokens, 0 among them: in order of ids come tokens that weigh nothing in 64 bits, then tokens of
    2^-100 to 2^-45 of the largest, then those that carry the sum.  Each filter keeps the small ones, or none."""
    rng = np.random.default_rng(vocab + small)
    n, small = 24, min(small, vocab // 2)
    v = np.full((n, vocab), float(torch.finfo(TYPES[kind]).min))
    v[:, : vocab // 3: 3] = -2000.0
    for i in range(n):
        v[i, np.sort(rng.permutation(vocab - 40)[:small])] = np.sort(rng.uniform(-69, -31, small))
        v[i, rng.permutation(np.arange(vocab - 40, vocab))[:12]] = rng.uniform(-3, 0, 12)
    v[:, 1::4] = np.where(rng.random((n, 1)) < 0.3, -INF, v[:, 1::4])
    x = torch.as_tensor(v, device="cuda").to(TYPES[kind])
    row = x.double().cpu().numpy()
    u = f32(np.exp2(rng.uniform(-105, -20, n)))
    u[:8] = [0, 0, 1e-45, 2.0 ** -126, 1e-30, 1e-20, 2.0 ** -24, 2.0 ** -25]
    cover = small + 12
    for kw in ({}, dict(top_k=np.full(n, cover)), dict(top_k=np.full(n, vocab - 1)), dict(top_k=np.full(n, 12)), dict(min_p=np.full(n, 1e-36)),
               dict(top_p=np.full(n, 1 - 2.0 ** -24)), dict(top_k=np.full(n, cover), min_p=np.full(n, 1e-25), temperature=np.full(n, 1.25)),
               dict(temperature=np.full(n, 0.75))):
        kw = {k: (w if k == "top_k" else f32(w)) for k, w in kw.items()}
        token, logp, kept, _ = S.sample(row, u, **kw)
        # how near a border lies to the number, relative to the number: further than the sums are off, which is 2^-43 of the whole sum for numbers from
        # 2^-24 on, and 2^-42 of themselves (the whole sum's, and FP64 roundings) for those below
        t = kw.get("temperature", np.ones(n, np.float32)).astype(float)[:, None]
        for i in range(n):
            z = (row[i] - row[i].max()) / t[i]
            live = row[i] >= np.sort(row[i])[::-1][kept[i] - 1]
            upto = np.where(live, np.exp(z), 0).cumsum()
            at = float(u[i]) * upto[-1]
            assert at == 0 or np.abs(upto / at - 1).min() > (2.0 ** -18 if u[i] >= 2.0 ** -24 else 2.0 ** -41)
        got = [w.cpu().numpy() for w in R.sample_tokens(x, floats(u), floats(kw.get("temperature")), ints(kw.get("top_k")), floats(kw.get("top_p")),
                                                        floats(kw.get("min_p")))]
        assert got[0].tolist() == token.tolist(), kw
        assert got[2].tolist() == kept.tolist()
        assert np.allclose(got[1], logp, rtol=2.0 ** -20, atol=2.0 ** -20)


@pytest.mark.parametrize("vocab", [40, 3000])
def test_the_smallest_weights(R, vocab):
    """Weights at the end of FP64's range, which 0 draws if they are first: from half of 2^-1074 on they are some."""
    z = np.float32([-746.0, -745.5, -745.25, -745.1875, -745.125, -745.0625, -745.0, -744.0, -720.0, -709.0])
    x = torch.full((len(z), vocab), -800.0, device="cuda")
    x[:, 7] = torch.as_tensor(z, device="cuda")
    x[:, 30] = -1.0
    x[:, 31] = 0.0
    want = np.where(z > -745.1332, 7, 30)  # (e^-745.125 is 1.008 halves of 2^-1074)
    u = floats(np.zeros(len(z)))
    assert R.sample_tokens(x, u)[0].tolist() == want.tolist()
    assert R.sample_tokens(x, u, top_k=ints(np.full(len(z), vocab - 1)))[0].tolist() == want.tolist()


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab", [2000, 40000, 151936, 2 ** 19 - 3])
def test_flat_rows(R, kind, vocab):
    """Nuclei, numbers and least weights that keep hundreds of tokens to all but a few: lists of each length, and rows without one."""
    rng = np.random.default_rng(vocab)
    n = 24
    x = logits(rng, n, vocab, kind, np.exp(rng.uniform(np.log(0.02), np.log(0.5), (n, 1))))
    p = 1 - np.exp(rng.uniform(np.log(1e-8), np.log(0.9), n))
    k = np.exp(rng.uniform(np.log(100), np.log(vocab), n)).astype(int)
    low = np.exp(-np.exp(rng.uniform(np.log(0.02), np.log(12), n)))
    u, t = rng.random(n), rng.uniform(0.5, 2, n)
    for kw in (dict(top_p=p), dict(top_k=k), dict(min_p=low), dict(top_p=p, top_k=k), dict(top_p=p, min_p=low), dict(top_k=k, min_p=low),
               dict(top_p=p, top_k=k, min_p=low)):
        check(R, x, u, t, **kw)


@pytest.mark.parametrize("ctas,n", [(1, 153), (2, 77), (3, 51), (4, 39), (5, 31), (6, 26), (7, 22), (9, 17), (12, 13)])
def test_long_lists_by_ctas(R, ctas, n):
    """Rows of so many CTAs (as many as hold a row, where the rows are enough for all SMs), that find their thresholds digit by digit: shares of the
    ranges that end inside a warp among them."""
    rng = np.random.default_rng(ctas)
    x = logits(rng, n, 18500 * ctas, "fp32", rng.uniform(0.02, 0.1, (n, 1)))
    u, p, k = rng.random(n), rng.uniform(0.3, 0.99, n), rng.integers(2000, 15000, n)
    for kw in (dict(top_p=p), dict(top_k=k), dict(top_k=k, top_p=p, min_p=np.full(n, 0.1))):
        check(R, x, u, rng.uniform(0.7, 1.5, n), **kw)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("vocab,heavy", [(1500, 0), (1500, 1000), (40000, 0), (40000, 500), (40000, 1000)])
@pytest.mark.parametrize("mode", ["plain", "p", "k"])
def test_numbers_near_borders(R, kind, vocab, heavy, mode):
    """u as near to the border of two tokens as FP32 has it, and up to 100 steps of 2^-24 beside: about as far as FP32 sums may be off.  Where
    `heavy` neighbours have most of the weight (alike, so that all their roundings are), the largest logit is another's."""
    rng = np.random.default_rng(vocab + heavy)
    n = 120
    x = logits(rng, n, vocab, kind, np.exp(rng.uniform(-2.5, -0.5, (n, 1))))
    if heavy:
        x[:, :] = torch.as_tensor(rng.uniform(-30, -14, (n, vocab)), device="cuda").to(TYPES[kind])
        at = rng.integers(0, vocab - heavy, n)
        for i in range(n):
            x[i, at[i]: at[i] + heavy] = float(rng.uniform(-9, -1))
            x[i, (at[i] + vocab // 2) % vocab] = float(rng.uniform(-0.1, 0.1))
    t = f32(rng.uniform(0.6, 1.4, n))
    p = f32(rng.uniform(0.9, 0.9999, n)) if mode == "p" else None
    k = np.full(n, vocab - 3) if mode == "k" else None
    row = x.double().cpu().numpy()
    token, _, kept, _ = S.sample(row, rng.random(n), t, k, p)
    u = np.zeros(n, np.float32)
    for i in range(n):
        live = row[i] >= np.sort(row[i])[::-1][kept[i] - 1]
        upto = np.where(live, np.exp((row[i] - row[i].max()) / float(t[i])), 0).cumsum()
        u[i] = np.float32(upto[token[i]] / upto[-1]) + np.float32(rng.integers(-100, 101) * 2.0 ** -24 * (i % 3 > 0))
    u = np.clip(u, 0, f32(1 - 2.0 ** -24))
    check(R, x, u, t, k, p)


@pytest.mark.parametrize("sizes", [(1, 128), (129, 256), (257, 511), (512, 1024), (1025, 1400)])
def test_lists(R, sizes):
    """As many tokens as named stand out: those that a filter's list takes in."""
    rng = np.random.default_rng(sizes[0])
    n, vocab = 32, 60000
    v = rng.uniform(-30, -20, (n, vocab))
    for i, c in enumerate(np.linspace(*sizes, n).astype(int)):
        v[i, rng.permutation(vocab)[:c]] = rng.uniform(0, 1, c)
    x = torch.as_tensor(v, device="cuda").float()
    u = rng.random(n)
    size = np.linspace(*sizes, n).astype(int)
    for kw in (dict(top_p=np.full(n, 0.999)), dict(top_k=size), dict(min_p=np.full(n, 0.05)), dict(top_k=size, top_p=rng.uniform(0.5, 1, n)),
               dict(top_p=rng.uniform(0.5, 1, n), min_p=rng.uniform(0.3, 0.6, n)), dict(top_k=np.maximum(size - 1, 1), min_p=rng.uniform(0.3, 0.6, n))):
        _, _, kept = check(R, x, u, None, **kw)
        assert kept.max() <= sizes[1]


@pytest.mark.parametrize("offset", [-2.0 ** 13, 2.0 ** 13, 2.0 ** 16])
def test_logits_far_from_zero(R, offset):
    """A common addend that FP32 weights of 2^(x c + k) hardly bear: k is off by percents, or out of its range."""
    rng = np.random.default_rng(abs(int(offset)))
    n, vocab = 24, 30000
    x = (torch.as_tensor(rng.standard_normal((n, vocab)) * rng.uniform(0.02, 0.5, (n, 1)), device="cuda") + offset).float()
    t = np.exp(rng.uniform(np.log(0.012), np.log(0.3), n))
    p = 1 - np.exp(rng.uniform(np.log(1e-5), np.log(0.9), n))
    for kw in ({}, dict(top_p=p), dict(top_k=rng.integers(1, 3000, n), top_p=p), dict(min_p=np.exp(-rng.uniform(0, 12, n))),
               dict(top_p=p, min_p=np.exp(-rng.uniform(0, 12, n)))):
        check(R, x, rng.random(n), t, **kw)


@pytest.mark.parametrize("offset", [0.0, 2.0 ** 16])
def test_long_tails(R, offset):
    """One token has most of the weight, and what is decided lies among 2^19 small ones: weights far below the largest count."""
    rng = np.random.default_rng(41)
    n, vocab = 12, 2 ** 19 - 3
    # (steps of 2^-7 at 2^16; T 2^-6, so that the tail is 2^-29 .. 2^-35 of the largest)
    v = (rng.integers(-3, 1, (n, vocab)) - 41) * 2.0 ** -7
    v[np.arange(n), rng.integers(0, vocab, n)] = 0
    x = torch.as_tensor(v + offset, device="cuda").float()
    t = np.full(n, 2.0 ** -6 / 1.0)
    tail = np.exp(v / 2.0 ** -6).sum(1) - 1
    for part in (0.2, 0.5, 0.9):
        check(R, x, rng.random(n), t, top_p=1 - tail / (1 + tail) * part)
        check(R, x, 1 - tail / (1 + tail) * part, t, top_p=np.full(n, 1 - 1e-7), min_p=np.full(n, 1e-20))
        check(R, x, 1 - tail / (1 + tail) * part, t)


def test_draws_follow_the_distribution(R):
    """Evenly spaced numbers draw each token as often as its weight says, to one draw."""
    rng = np.random.default_rng(5)
    n, vocab = 8192, 500
    x = logits(rng, 1, vocab, "fp32").repeat(n, 1)
    u = (np.arange(n) + 0.5) / n
    token, _, _ = R.sample_tokens(x, floats(u), floats(np.full(n, 0.8)), top_p=floats(np.full(n, 0.9)))
    got = np.bincount(token.cpu().numpy(), minlength=vocab)
    _, _, kept, _ = S.sample(x[:1].double().cpu().numpy(), u[:1], [np.float32(0.8)], None, [np.float32(0.9)])
    row = x[0].double().cpu().numpy()
    live = row >= np.sort(row)[::-1][kept[0] - 1]
    w = np.where(live, np.exp((row - row.max()) / np.float64(np.float32(0.8))), 0)
    assert np.all(np.abs(got - n * w / w.sum()) <= 1)


@pytest.mark.parametrize("kind", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab", [300, 40000])
def test_masks(R, kind, vocab):
    """Masked tokens are never drawn, by -infinity or the type's lowest value; k counts more than are left; a row with one token, with none."""
    rng = np.random.default_rng(vocab)
    n = 12
    x = logits(rng, n, vocab, kind)
    for low in (-INF, float(torch.finfo(TYPES[kind]).min)):
        y = x.clone()
        y[:, torch.as_tensor(rng.random(vocab) < 0.7, device="cuda")] = low
        y[3] = low
        y[3, vocab // 3] = -7.0
        if low == -INF:
            y[5] = low
        t, k, p = rng.uniform(0.4, 1.2, n), rng.choice([0, vocab // 2, vocab - 1, 5], n), rng.uniform(0.5, 1.1, n)
        token, logp, kept = check(R, y, rng.random(n), t, k, p)
        assert token[3] == vocab // 3
        if low == -INF:
            assert token[5] == -1 and logp[5] == -INF and kept[5] == 0
        check(R, y, rng.random(n), np.where(np.arange(n) % 2, 0, 0.5))


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("stride,first", [(1000, 0), (1001, 1), (1003, 3), (1013, 5)])
def test_strides(R, kind, stride, first):
    """Rows that begin anywhere, beside values that are not theirs."""
    rng = np.random.default_rng(stride)
    wide = torch.full((11, stride), 1e30, dtype=TYPES[kind], device="cuda")
    x = wide.view(-1)[: 11 * stride].view(11, stride)[:, first: first + 990]
    x.copy_(logits(rng, 11, 990, kind))
    check(R, x, rng.random(11), rng.uniform(0.5, 1, 11), rng.choice([0, 40], 11), rng.choice([0.9, 1.0], 11))
    check(R, x, rng.random(11), np.zeros(11))


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_far_temperatures_and_values(R, kind):
    rng = np.random.default_rng(9)
    t = [1e-40, 1e-30, 1e-6, 0.01, 100.0, 1e10, 2.0 ** 64, 1.0]
    x = logits(rng, 8, 2000, kind)
    check(R, x, rng.random(8), t)
    check(R, x, rng.random(8), t, top_p=rng.uniform(0.1, 0.9, 8), top_k=rng.integers(1, 2000, 8))
    big = torch.as_tensor(rng.choice([-3e38, 3e38, 1e38, -1e38, 0.0], (8, 700)), device="cuda").to(TYPES[kind])
    check(R, big, rng.random(8), t, top_k=rng.integers(1, 700, 8))
    check(R, big, rng.random(8), t, top_p=rng.uniform(0.1, 0.9, 8), min_p=[0.1] * 8)


def test_smallest_temperatures(R):
    """Logits as far apart as the smallest temperature; those below act as it."""
    rng = np.random.default_rng(10)
    least = np.float32(2.0 ** -125)
    x = torch.as_tensor(rng.standard_normal((12, 3000)) * 2.0 ** -125 * rng.uniform(0.5, 4, (12, 1)), device="cuda").float()
    u, p, k = rng.random(12), rng.uniform(0.2, 1, 12), rng.integers(1, 3000, 12)
    t = np.concatenate([np.full(8, least), np.geomspace(2.0 ** -125, 2.0 ** -120, 4)])
    for kw in ({}, dict(top_p=p), dict(top_k=k), dict(top_k=k, top_p=p), dict(min_p=p)):
        check(R, x, u, t, **kw)
    small = np.float32([1e-45, 1e-40, 1e-39, 2.0 ** -126, 2.0 ** -125, 2e-38, 2e-38, 2e-38, 2e-38, 2e-38, 2e-38, 2e-38])
    for a, b in zip(R.sample_tokens(x, floats(u), floats(small)), R.sample_tokens(x, floats(u), floats(np.maximum(small, least)))):
        assert torch.equal(a, b)


def test_reports(R):
    rng = np.random.default_rng(2)
    x = logits(rng, 6, 3000, "fp32")
    u = rng.random(6)
    for bad in (INF, float("nan")):
        y = x.clone()
        y[2, 1234] = bad
        token, _, _ = check(R, y, u, want_status=D.DFLASH_DEV_NONFINITE, rows=np.array([0, 1, 3, 4, 5]))
        st = status()
        assert int(R.sample_tokens(y, floats(u), status=st)[0][2]) == -1 and int(st) == D.DFLASH_DEV_NONFINITE
    want = R.sample_tokens(x, floats(u), floats([0.8] * 6))[0]
    others = [0, 1, 3, 4, 5]

    def call(at, **kw):
        args = {**dict(uniform=u.copy(), temperature=np.full(6, 0.8), top_k=None, top_p=np.ones(6), min_p=np.zeros(6)), **kw}
        st = status()
        token = R.sample_tokens(x, floats(args["uniform"]), floats(args["temperature"]), None, floats(args["top_p"]), floats(args["min_p"]), status=st)[0]
        assert int(st) == D.DFLASH_DEV_BAD_VALUE and torch.equal(token[others], want[others])
        return int(token[at])

    def put(values, value):
        values = np.array(values, np.float32)
        values[2] = value
        return values

    best = int(x[2].argmax())
    for t in (-1.0, float("nan")):
        assert call(2, temperature=put(np.full(6, 0.8), t)) == best  # greedy
    call(2, temperature=put(np.full(6, 0.8), INF))
    for w, near in ((-0.5, 0.0), (float("nan"), 0.0), (1.0, 1 - 2.0 ** -24), (INF, 1 - 2.0 ** -24)):
        st = status()
        v = put(u, near)
        assert call(2, uniform=put(u, w)) == int(R.sample_tokens(x, floats(v), floats([0.8] * 6), status=st)[0][2]) and int(st) == 0
    assert call(2, top_p=put(np.ones(6), float("nan"))) == int(want[2])
    assert call(2, min_p=put(np.zeros(6), float("nan"))) == int(want[2])
    assert call(2, min_p=put(np.zeros(6), 1.5)) == best


def test_same_result_again(R):
    rng = np.random.default_rng(4)
    x = logits(rng, 40, 100003, "bf16")
    args = (floats(rng.random(40)), floats(rng.uniform(0.5, 1, 40)), ints(rng.choice([0, 30, 5000], 40)), floats(rng.uniform(0.7, 1.1, 40)))
    first = R.sample_tokens(x, *args)
    for _ in range(30):
        for a, b in zip(R.sample_tokens(x, *args), first):
            assert torch.equal(a, b)


def test_graph_and_stream(R):
    rng = np.random.default_rng(6)
    x, u, t, k = logits(rng, 16, 9000, "bf16"), floats(rng.random(16)), floats(rng.uniform(0.5, 1, 16)), ints(rng.integers(1, 100, 16))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = R.sample_tokens(x, u, t, k)
    got = R.sample_tokens(x, u, t, k, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = R.sample_tokens(x, u, t, k)
    for seed in range(3):
        rng = np.random.default_rng(seed)
        x.copy_(logits(rng, 16, 9000, "bf16"))
        u.copy_(floats(rng.random(16)))
        t.copy_(floats(np.where(rng.random(16) < 0.3, 0, rng.uniform(0.5, 1, 16))))
        k.copy_(ints(rng.choice([0, 10], 16)))
        graph.replay()
        token, _, kept, _ = S.sample(x.double().cpu().numpy(), u.cpu().numpy(), t.cpu().numpy(), k.cpu().numpy())
        assert out[0].tolist() == token.tolist() and out[2].tolist() == kept.tolist()


def raw(R, x, u, tokens, logprob=None, kept=None, **kw):
    at = lambda v: 0 if v is None else v.data_ptr()  # noqa: E731
    D.dflash_sample_tokens(x.data_ptr(), {torch.float32: D.DFLASH_T_FP32, torch.bfloat16: D.DFLASH_T_BF16, torch.float16: D.DFLASH_T_FP16}[x.dtype],
                           x.stride(0), x.shape[0], x.shape[1], u.data_ptr(), at(kw.get("temperature")), at(kw.get("top_k")), at(kw.get("top_p")),
                           at(kw.get("min_p")), at(tokens), at(logprob), at(kept), 0, torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("n,vocab", [(3000, 1024), (700, 32768), (40, 2 ** 18)])
def test_numbers_on_a_border(R, kind, n, vocab):
    """u on the border of two tokens in every row: 2^-k of equal weights is exact, and the token behind the border is the one.  With and
    without the outputs that may be left out."""
    x = torch.full((n, vocab), 1.5, dtype=TYPES[kind], device="cuda")
    want = torch.as_tensor(np.random.default_rng(n).integers(0, vocab, n), device="cuda").int()
    u = want.float() / vocab
    hot = x.clone()
    hot[:, ::2] = -INF  # half of them are left
    for y, factor in ((x, 1), (hot, 2)):
        token, logp, kept = R.sample_tokens(y, u)
        right = want if factor == 1 else want // 2 * 2 + 1
        assert torch.equal(token, right) and kept.tolist() == [vocab // factor] * n
        assert np.allclose(logp.cpu().numpy(), -np.log(vocab // factor), rtol=2.0 ** -22, atol=0)
        for outs in ({}, dict(logprob=logp), dict(kept=kept)):
            for o in outs.values():
                o.fill_(7)
            token.fill_(7)
            raw(R, y, u, token, **outs)
            assert torch.equal(token, right)
            assert all(not bool((o == 7).any()) for o in outs.values())


@pytest.mark.parametrize("kind", ["fp32", "fp16"])
def test_outputs_left_out(R, kind):
    rng = np.random.default_rng(21)
    x = logits(rng, 30, 20011, kind, np.exp(rng.uniform(-3, 0, (30, 1))))
    u = floats(rng.random(30))
    for kw in ({}, dict(top_k=ints(rng.integers(1, 3000, 30))), dict(top_p=floats(rng.uniform(0.5, 1, 30))), dict(min_p=floats(rng.uniform(0.01, 1, 30))),
               dict(temperature=floats(np.zeros(30)), top_k=ints(np.ones(30)))):
        token, logp, kept = R.sample_tokens(x, u, **kw)
        for outs in ({}, dict(logprob=torch.empty_like(logp)), dict(kept=torch.empty_like(kept))):
            t = torch.empty_like(token)
            raw(R, x, u, t, **outs, **kw)
            assert torch.equal(t, token)
            assert all(torch.equal(o, dict(logprob=logp, kept=kept)[k]) for k, o in outs.items())


def test_calls_at_once(R):
    """Calls with and without filters on three streams, and one behind the other on each."""
    rng = np.random.default_rng(17)
    cases = []
    for i, (n, vocab, kind) in enumerate([(300, 2 ** 15, "fp32"), (64, 50000, "bf16"), (9, 151936, "fp16")]):
        x = logits(rng, n, vocab, kind, np.exp(rng.uniform(-3, 0, (n, 1))))
        if i == 0:
            x[::2] = 0.5  # equal weights: u on a border
        u = floats(np.round(rng.random(n) * 2 ** 15 - 0.5) / 2 ** 15)
        for kw in ({}, dict(top_p=floats(rng.uniform(0.5, 1, n))), dict(top_k=ints(rng.integers(1, 4000, n)))):
            cases.append((x, u, kw, R.sample_tokens(x, u, **kw)))
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for i in range(len(cases)):
            x, u, kw, want = cases[(i * 4) % len(cases)]
            with torch.cuda.stream(streams[i % 3]):
                got.append((R.sample_tokens(x, u, **kw), want))
    torch.cuda.synchronize()
    for a, b in got:
        assert all(torch.equal(v, w) for v, w in zip(a, b))


def test_graph_without_filters(R):
    """Two captured calls replayed on two streams, rows that their second kernel decides among them."""
    rng = np.random.default_rng(23)
    held = []
    for n, vocab, kind in ((500, 4096, "fp32"), (20, 100003, "bf16")):
        x, u = logits(rng, n, vocab, kind), floats(rng.random(n))
        R.sample_tokens(x, u)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = R.sample_tokens(x, u)
        held.append((g, x, u, out))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for seed in range(4):
        rng = np.random.default_rng(seed)
        for g, x, u, out in held:
            x.copy_(logits(rng, *x.shape, "fp32"))
            x[::3] = -0.25
            u.copy_(floats(np.floor(rng.random(len(u)) * 4096) / 4096))
        torch.cuda.synchronize()
        for s, (g, *_) in zip(streams, held):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for g, x, u, out in held:
            token, _, kept, near = S.sample(x.double().cpu().numpy(), u.cpu().numpy())
            clear = near > 2.0 ** -42
            assert clear.sum() > len(u) // 2 and out[2].tolist() == kept.tolist()
            assert np.array_equal(out[0].cpu().numpy()[clear], token[clear])
        equal = held[0][1].shape[1]  # (a power of two: the token is known there too)
        assert held[0][3][0][::3].tolist() == (held[0][2][::3] * equal).int().tolist()


def test_no_rows(R):
    token, logp, kept = R.sample_tokens(torch.zeros((0, 50), device="cuda"), floats(np.zeros(0)))
    assert token.shape == logp.shape == kept.shape == (0,)


def test_offsets_beyond_32_bits(R):
    """A row that begins beyond 4 GB."""
    rng = np.random.default_rng(8)
    x = torch.full((9000, 2 ** 18), -1.0, dtype=torch.bfloat16, device="cuda")
    x[-2:] = logits(rng, 2, 2 ** 18, "bf16")
    u = rng.random(9000)
    token, _, kept = R.sample_tokens(x, floats(u), top_k=ints(np.full(9000, 64)))
    t, _, n, _ = S.sample(x[-2:].double().cpu().numpy(), f32(u)[-2:], None, [64, 64])
    assert token[-2:].tolist() == t.tolist() and kept[-2:].tolist() == n.tolist()
    assert token[:-2].tolist() == np.floor(f32(u)[:-2].astype(float) * 2 ** 18).astype(int).tolist()


def test_sampled_steps_together(R):
    """Steps of a served model that samples: rotation, cells, attention over a shared prefix, draws, acceptance, the next lengths on the device."""
    rng = np.random.default_rng(12)
    n, heads, G, d, page, B, vocab, steps, shared = 6, 2, 4, 64, 16, 4, 900, 5, 50
    n_pages, width = 160, 20
    cap = n * B
    cache = R.kv4_cache(n_pages, page, heads, d)
    turns = R.rope_turns([1e4 ** (-2.0 * j / d) for j in range(d // 2)])
    weight = floats(1 + 0.2 * rng.standard_normal(d))
    status_word = status()
    # the prefix: pages 0 .. 3, filled as a prompt is
    prefix = torch.as_tensor(rng.standard_normal((shared, 2 * heads, d)), device="cuda").bfloat16()
    none = torch.empty((shared, 0, d), dtype=torch.bfloat16, device="cuda")
    _, pk = R.qk_norm_rope(none, prefix[:, :heads], ints(np.arange(shared)), turns, k_weight=weight, status=status_word)
    R.kv4_write(cache, pk, prefix[:, heads:], ints(np.arange(shared)), status=status_word)
    prefix_table, prefix_len, groups = ints(np.arange(4)[None]), ints([shared]), ints([0, n])
    held, table, ring, state = ints(np.zeros(n)), ints(np.full((n, width), -1)), ints(np.arange(4, n_pages).tolist() + [-1] * 4), ints([0, n_pages - 4])
    length, accepted, bonus, rows = ints(np.zeros(n)), ints(np.zeros(n)), ints(np.zeros(n)), ints(np.full(n, B))
    head = torch.as_tensor(rng.standard_normal((vocab, heads * G * d)), device="cuda").float()
    temperature = floats(np.full(cap, 0.7))
    drawn = 0
    for step in range(steps):
        qkv = torch.as_tensor(rng.standard_normal((cap, heads * G + 2 * heads, d)), device="cuda").bfloat16()
        before = length.cpu().numpy().copy()
        off, slots, pos = R.page_tables(length, rows, held, table, ring, state, page, cap, status=status_word)
        q, k = qkv[:, : heads * G], qkv[:, heads * G: heads * G + heads]
        q, k = R.qk_norm_rope(q, k, pos + shared, turns, q_weight=weight, k_weight=weight, q_out=q, k_out=k, status=status_word)
        R.kv4_write(cache, k, qkv[:, heads * G + heads:], slots, status=status_word)
        o = R.kv4_prefix_attention(cache, q, prefix_table, prefix_len, groups, table, length + rows, off, B, status=status_word)
        # the same through tables whose first positions are the prefix's cells, cell by cell
        K, W = R.kv4_read(cache, ints(np.arange(n_pages * page)))
        K, W = K.double().cpu().numpy(), W.double().cpu().numpy()
        tab = table.cpu().numpy()
        for s in range(n):
            at = np.arange(before[s] + B)
            cells = np.concatenate([np.arange(shared), tab[s, at // page] * page + at % page])
            for i in range(B):
                m = shared + before[s] + i + 1
                for h in range(heads * G):
                    x = K[cells[:m], h // G] @ q[s * B + i, h].double().cpu().numpy() / 8.0
                    p = np.exp(x - x.max())
                    v = W[cells[:m], h // G]
                    want, spread = p @ v / p.sum(), p @ np.abs(v) / p.sum()
                    tol = spread * (2.0 ** -10 + 2.0 ** -10 * (1 + np.abs(x).max())) + m * 2.0 ** -22 + 2.0 ** -8 * np.abs(want)
                    assert np.all(np.abs(o[s * B + i, h].double().cpu().numpy() - want) <= tol)
        logits_ = o.float().flatten(1) @ head.t()
        u = rng.random(cap)
        token, _, _ = check(R, logits_, u, temperature.cpu().numpy(), top_p=np.full(cap, 0.95))
        ids = R.sample_tokens(logits_, floats(u), temperature, top_p=floats(np.full(cap, 0.95)), status=status_word)[0]
        drafts = rng.integers(0, vocab, (n, B - 1)).astype(np.int32)
        drafts[:, 0] = ids.view(n, B)[:, 0].cpu().numpy()  # the first candidate is what is drawn
        R.accept(ints(drafts), ids.view(n, B).contiguous(), rows, accepted, bonus, anchor_pos=length)
        drawn += int(accepted.sum())
        assert np.array_equal(length.cpu().numpy(), before + accepted.cpu().numpy() + 1)
        assert np.array_equal(bonus.cpu().numpy(), token.reshape(n, B)[np.arange(n), accepted.cpu().numpy()])
    assert drawn >= n * steps and int(status_word) == 0
