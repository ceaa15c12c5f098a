"""Per-head norms with the position rotation on the GPU against the 64-bit form (sampling_ref.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import dflash_block_drafter_gb300 as D  # noqa: E402
import gpu_helpers as H  # noqa: E402
import sampling_ref as S  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


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


def floats(x):
    return None if x is None else torch.as_tensor(np.asarray(x, np.float32), device="cuda")


def bound(want, size, kind):
    """How far a result may be off: the rounding to the type (FP16: its smallest step too), and FP32 before it.  Its relative
    errors, in units of 2^-24: the sum of squares 13 (8 products in turn, 5 joins), halved by the root; rsqrt 4; the products
    with the weight, the cosine, the partner and 1 / rms 4; cosine and sine 6 (angle 2^-25 turns, function 2 units): under 32 in all."""
    half = S.STEP[kind]
    fp32 = 2.0 ** -19 * size
    return half * np.abs(want) + fp32 * (1 + half) + (2.0 ** -25 if kind == "fp16" else 1e-38)


def case(kind, rows, nq, nk, d, rot, n_axes=1, far=50000, seed=0, pad=8, gain=1.0):
    rng = np.random.default_rng(seed)
    width = (nq + 2 * nk) * d + pad
    x = S.to_type(gain * rng.standard_normal((rows, width)) * np.exp(rng.standard_normal((rows, 1))), kind)
    t = torch.as_tensor(x, device="cuda").to(TYPES[kind])
    freqs = [1e4 ** (-2.0 * j / rot) for j in range(rot // 2)] if rot else []
    turns = D.dflash_rope_turns(freqs)
    positions = rng.integers(0, far, (n_axes, rows))
    axes = rng.integers(0, n_axes, rot // 2) if n_axes > 1 else None
    weights = 1 + 0.3 * rng.standard_normal((2, d))
    weights = weights.astype(np.float32).astype(np.float64)
    return dict(x=x, t=t, q=t[:, : nq * d].unflatten(1, (nq, d)) if nq else None, k=t[:, nq * d: (nq + nk) * d].unflatten(1, (nk, d)) if nk else None,
                xq=x[:, : nq * d].reshape(rows, nq, d), xk=x[:, nq * d: (nq + nk) * d].reshape(rows, nk, d), freqs=freqs, turns=turns,
                positions=positions, axes=axes, weights=weights, kind=kind)


def call(R, c, norm=True, eps=1e-6, st=None, **kw):
    turns = R.rope_turns(c["freqs"]) if c["freqs"] else None
    pos = c["positions"] if c["axes"] is not None else c["positions"][0]
    axes = None if c["axes"] is None else torch.as_tensor(c["axes"].astype(np.uint8), device="cuda")
    return R.qk_norm_rope(c["q"], c["k"], ints(pos) if turns is not None else None, turns, q_weight=floats(c["weights"][0]) if norm else None,
                          k_weight=floats(c["weights"][1]) if norm and c["k"] is not None else None, eps=eps, axes=axes, status=st, **kw)


def check(c, got, norm=True, eps=1e-6, rows=slice(None)):
    angle = S.angles(c["positions"], c["turns"], c["axes"]) if c["freqs"] else None
    for x, w, g in ((c["xq"], c["weights"][0], got[0]), (c["xk"], c["weights"][1], got[1])):
        if g is None:
            continue
        want, size = S.norm_rope(x, w if norm else None, eps, angle)
        err = np.abs(g.double().cpu().numpy() - want)[rows]
        assert np.all(err <= bound(want, size, c["kind"])[rows]), err.max()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 0), (128, 128), (128, 48), (256, 256), (256, 64), (256, 16), (256, 0)])
@pytest.mark.parametrize("rows,nq,nk", [(1, 1, 1), (1, 24, 2), (9, 5, 3), (33, 16, 16), (700, 3, 1)])
def test_rows(R, kind, d, rot, rows, nq, nk):
    c = case(kind, rows, nq, nk, d, rot, seed=rows + d + rot)
    st = status()
    check(c, call(R, c, st=st))
    check(c, call(R, c, norm=False, st=st), norm=False)
    assert int(st) == 0


@pytest.mark.parametrize("n_axes", [2, 3, 4])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 96), (256, 128)])
def test_several_axes(R, n_axes, d, rot):
    c = case("bf16", 21, 6, 2, d, rot, n_axes=n_axes, seed=n_axes)
    check(c, call(R, c))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_in_place_leaves_the_rest(R, d):
    """On the fused projection's output itself: the values and the padding beside the queries and keys stay as they were."""
    c = case("bf16", 50, 7, 3, d, d, seed=d)
    apart = call(R, c)
    before = c["t"].clone()
    q, k = call(R, c, q_out=c["q"], k_out=c["k"])
    assert q.data_ptr() == c["q"].data_ptr() and torch.equal(q, apart[0]) and torch.equal(k, apart[1])
    assert torch.equal(c["t"][:, 10 * d:], before[:, 10 * d:])


def test_padded_rows_stay(R):
    c = case("fp16", 40, 4, 2, 128, 128, n_axes=2, seed=5)
    gone = np.arange(40) % 3 == 1
    c["positions"][0, gone] = -1
    c["positions"][1, 7] = -5  # any axis
    gone[7] = True
    c["t"][torch.as_tensor(gone, device="cuda")] = float("nan")  # not read, either
    q, k = torch.full_like(c["q"], 3), torch.full_like(c["k"], 3)
    st = status()
    call(R, c, q_out=q, k_out=k, st=st)
    assert int(st) == 0 and bool((q[torch.as_tensor(gone)] == 3).all()) and bool((k[torch.as_tensor(gone)] == 3).all())
    c["positions"][:, gone] = 0
    check(c, (q, k), rows=~gone)


def test_keys_or_queries_alone(R):
    c = case("bf16", 12, 4, 2, 128, 64)
    both = call(R, c)
    alone = {**c, "k": None}
    assert torch.equal(call(R, alone)[0], both[0]) and call(R, alone)[1] is None
    none = {**c, "q": c["t"][:, :0].unflatten(1, (0, 128))}
    assert torch.equal(call(R, none)[1], both[1])


def test_far_positions(R):
    """The angle of the largest positions is that of the table, however many turns they are."""
    c = case("fp16", 64, 2, 1, 128, 128, far=2 ** 31 - 1, seed=3)
    c["positions"][0, :2] = [2 ** 31 - 1, 0]
    check(c, call(R, c))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("gain,eps", [(1e30, 1e-6), (1e-30, 0.0), (1e-30, 1e-6), (3e18, 0.0), (1e-15, 1e-33)])
def test_values_beyond_the_squares_range(R, d, gain, eps):
    c = case("bf16", 9, 4, 2, d, d, gain=gain, seed=11)
    st = status()
    check(c, call(R, c, eps=eps, st=st), eps=eps)
    assert int(st) == 0


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rot", [0, 64])
@pytest.mark.parametrize("eps", [0.0, 1e-36, 3e38])
def test_heads_at_the_types_ends(R, d, rot, eps):
    """Heads of the largest values (whose products with a weight, and sums of pairs, pass FP32's range before the root divides them), of subnormal ones
    and of ordinary ones beside each other, and weights of any size: the results are ordinary."""
    c = case("bf16", 24, 9, 5, d, rot, seed=d + rot)
    rng = np.random.default_rng(d)
    for x, t in ((c["xq"], c["q"]), (c["xk"], c["k"])):
        size = np.asarray([3.3e38, 2.0 ** -133, 1.0, 1e19, 2.0 ** -126, 1e-17])[rng.integers(0, 6, x.shape[:2])][..., None]
        x[:] = S.to_type(np.sign(x) * rng.uniform(0.5, 1.0, x.shape) * size * np.where(size < 1e-39, 8, 1), "bf16")
        t.copy_(torch.as_tensor(x, device="cuda").float().bfloat16())
        assert np.array_equal(t.double().cpu().numpy(), x) and np.all(x.any(-1))
    for gain in (1.0, 2.5, 1e25, 1e-25):
        c["weights"] = (gain * (1 + 0.3 * rng.standard_normal((2, d)))).astype(np.float32).astype(np.float64)
        st = status()
        got = call(R, c, eps=eps, st=st)
        assert int(st) == 0 and all(bool(torch.isfinite(g).all()) for g in got)
        check(c, got, eps=eps)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("eps", [1e-30, 1e-20, 1e-6, 1e10])
def test_small_heads_beside_eps(R, d, eps):
    """Heads whose squares are far below eps, so that 1 / rms is eps's: the products with the weights lose nothing below FP32's range."""
    c = case("bf16", 24, 9, 5, d, 32, seed=d)
    rng = np.random.default_rng(d)
    for x, t in ((c["xq"], c["q"]), (c["xk"], c["k"])):
        size = np.exp2(rng.uniform(-130, -40, x.shape[:2]))[..., None]
        x[:] = S.to_type(np.sign(x) * rng.uniform(0.5, 1.0, x.shape) * size, "bf16")
        t.copy_(torch.as_tensor(x, device="cuda").float().bfloat16())
    for gain in (1.0, 1e-3, 1e-8, 1e-18, 1e9, 1e20):
        c["weights"] = (gain * (1 + 0.3 * rng.standard_normal((2, d)))).astype(np.float32).astype(np.float64)
        st = status()
        check(c, call(R, c, eps=eps, st=st), eps=eps)
        assert int(st) == 0


def test_heads_of_zeros(R):
    c = case("bf16", 3, 4, 2, 64, 64)
    c["t"][1] = 0
    c["xq"][1] = c["xk"][1] = 0
    st = status()
    q, k = call(R, c, eps=0.0, st=st)
    assert int(st) == 0 and not bool(q[1].any()) and not bool(k[1].any())
    check(c, (q, k), eps=0.0)


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("where", ["q", "k"])
def test_reports_values_that_are_not_finite(R, bad, norm, where):
    c = case("bf16", 20, 4, 2, 128, 128)
    c[where][13, 1, 77] = bad
    st = status()
    got = call(R, c, norm=norm, st=st)
    assert int(st) == D.DFLASH_DEV_NONFINITE
    check(c, got, norm=norm, rows=np.arange(20) != 13)


def test_reports_an_axis_that_does_not_exist(R):
    c = case("bf16", 4, 2, 1, 64, 64, n_axes=2)
    c["axes"][5] = 9
    st = status()
    got = call(R, c, st=st)
    assert int(st) == D.DFLASH_DEV_BAD_VALUE
    c["axes"][5] = 0
    check(c, got)


def test_no_rows(R):
    c = case("bf16", 2, 4, 2, 64, 64)
    q, k = R.qk_norm_rope(c["q"][:0], c["k"][:0], ints(np.zeros(0)), R.rope_turns(c["freqs"]))
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)


def test_graph_and_stream(R):
    """A captured call reads its rows and positions anew; a call on another stream belongs to it."""
    c = case("bf16", 24, 8, 2, 128, 128, seed=1)
    turns, pos, w = R.rope_turns(c["freqs"]), ints(c["positions"][0]), [floats(v) for v in c["weights"]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q, k = R.qk_norm_rope(c["q"], c["k"], pos, turns, *w, stream=side)
    side.synchronize()
    check(c, (q, k))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, k = R.qk_norm_rope(c["q"], c["k"], pos, turns, *w)
    d = case("bf16", 24, 8, 2, 128, 128, seed=2)
    c["t"].copy_(d["t"])
    pos.copy_(ints(d["positions"][0]))
    for to, v in zip(w, d["weights"]):  # the replayed call reads these, not the second case's
        to.copy_(floats(v))
    graph.replay()
    check(d, (q, k))


def test_more_than_32_bits_of_elements(R):
    """Rows whose elements lie beyond 2^31: the last ones are those of a small call."""
    n, d, heads = 1 << 15, 256, 320  # 2.7 G elements
    x = torch.zeros((n, heads, d), dtype=torch.bfloat16, device="cuda")
    c = case("bf16", 5, heads, 1, d, d, seed=4)
    x[-5:] = c["q"]
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")
    pos[-5:] = ints(c["positions"][0])
    w = floats(c["weights"][0])
    got, _ = R.qk_norm_rope(x, None, pos, R.rope_turns(c["freqs"]), q_weight=w, q_out=x)
    assert torch.equal(got[-5:], call(R, {**c, "k": None})[0]) and not bool(got[:-5].any())
