"""Attention cases whose arithmetic is exact in the kernels' types, so that a lost, repeated or exchanged cell shows, and bounds for
ordinary ones that follow from the roundings the kernels state.  NumPy only.

Exact cases: K is 0 or -1 and V -3 .. 3 (a -8 in every block of 32 channels makes the block's scale 1), q is 1 at one channel of
up to three blocks, the softmax scale is ln 2.  Scores are then 0 .. -3 in powers of two, weights powers of two, and the sums of
weights times V whole multiples of the smallest weight, below 2^24 of them: nothing is rounded but the score (an FP32 product by
the scale), the power of two, the sum of weights and the output."""
import numpy as np

import verify_ref as V


def cells(rng, n, heads, d):
    """K and V [n, heads, d], every cell its own."""
    k, v = rng.integers(-1, 1, (n, heads, d)), rng.integers(-3, 4, (n, heads, d))
    k[..., 31::32] = v[..., 31::32] = -8
    return k, v


def queries(rng, tokens, heads, d):
    q = np.zeros((tokens, heads, d))
    for t in range(tokens):
        for h in range(heads):
            for b in rng.permutation(d // 32)[:3]:
                q[t, h, 32 * b + rng.integers(0, 31)] = 1
    return q


def attend(k, v, q, causal, window=0, bias=None):
    """(o, spread) of a sequence's rows q [r, nq, d] over k, v [n, heads, d] in 64 bits, scores in log2 units; bias: [n] log2 weights
    (-inf: a cell left out, 1: taken twice)."""
    n, heads, d = k.shape
    r, nq = q.shape[:2]
    o, spread = np.zeros(q.shape), np.zeros(q.shape)
    k, v = k.astype(np.float64), v.astype(np.float64)
    for h in range(heads):
        rows = q[:, h * (nq // heads):(h + 1) * (nq // heads)]
        p = np.exp2(np.einsum("rgd,nd->rgn", rows, k[:, h]) + (0 if bias is None else bias))
        last = np.arange(n - r, n) if causal else np.full(r, n - 1)
        at = np.arange(n)
        sees = (at <= last[:, None]) & ((at > last[:, None] - window) | (window == 0))
        p = p * sees[:, None]
        total = np.maximum(p.sum(-1, keepdims=True), 1e-300)
        o[:, h * (nq // heads):(h + 1) * (nq // heads)] = p @ v[:, h] / total
        spread[:, h * (nq // heads):(h + 1) * (nq // heads)] = p @ np.abs(v[:, h]) / total
    return o, spread


def tolerance(o, spread, eps):
    """Of an exact case.  A weight is off by 2^-22 for the power of two and by 2^-22 for a score of 3 at most times an FP32 scale that is
    off by 2^-23; the sum of weights by 2^-24 an addition of tiles and cells, of which a warp's lanes make few hundred in turn, in
    random directions: 2^-19 of the output's terms in all.  The output is rounded once (eps: half a step)."""
    return spread * 2.0 ** -19 + np.abs(o) * eps + 1e-7


def rounded_attention(cache, q, table, kv_len, offsets, causal, scale, eps, k_fp16):
    """(o, tolerance) for ordinary values.  The reference takes V (and K where `k_fp16`) rounded to FP16 as the kernels do, so that
    what remains are P, the scores, sums and the output."""
    n_pages, heads, groups, size = cache.shape
    page, d = groups * 16, size // 18
    G = q.shape[1] // heads
    o, tol = np.zeros(q.shape), np.zeros(q.shape)
    for s in range(len(kv_len)):
        r0, r1, n = int(offsets[s]), int(offsets[s + 1]), int(kv_len[s])
        pos = np.arange(n)
        k, v = V.load(cache, table[s, pos // page].astype(np.int64) * page + pos % page)
        step = np.abs(k).reshape(n, heads, d // 32, 32).max(-1) / 7  # of a block at least its scale
        if k_fp16:
            k = k.astype(np.float16).astype(np.float64)
        v = v.astype(np.float16).astype(np.float64)
        for i in range(r1 - r0):
            m = n - (r1 - r0) + i + 1 if causal else n
            for h in range(q.shape[1]):
                x = q[r0 + i, h]
                score = scale * (k[:m, h // G] @ x)
                p = np.exp(score - score.max())
                total = p.sum()
                vv = v[:m, h // G]
                o[r0 + i, h] = p @ vv / total
                spread = p @ np.abs(vv) / total
                # a score: d / 16 products in turn and a few more steps, 2^-23 each of the sum of the terms, which in the warp-level
                # kernel are codes up to 15 and an offset of 8; there a block's sum of q is off by 2^-19 of the row's largest, times 8
                by_block = np.abs(x).reshape(-1, 32).sum(-1)
                terms = scale * (np.abs(k[:m, h // G]) @ np.abs(x)) if k_fp16 else 23 * scale * (step[:m, h // G] @ by_block)
                off = terms * (d / 16 + 4) * 2.0 ** -23 + np.abs(score).max() * 2.0 ** -22 + 2.0 ** -21
                if not k_fp16:
                    off = off + scale * step[:m, h // G].sum(-1) * np.abs(x).max() * 2.0 ** -16
                off = off.max()
                # P: 2^-11 of it or 2^-32 of the largest; O: 16 cells a step, 2^-23 each; a weight off by `off` moves o by that
                # part of what the cell adds to the sum and to the total
                tol[r0 + i, h] = spread * (2.0 ** -11 + off + m / 16 * 2.0 ** -23) + np.abs(o[r0 + i, h]) * (off + 2.0 ** -20 + eps) \
                    + m * 2.0 ** -32 * np.abs(vv).max() / total + 1e-7
    return o, tol
