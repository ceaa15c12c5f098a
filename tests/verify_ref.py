"""Plain 64-bit (and whole-number) forms of the verify-step operators, from the definitions in include/dflash.h, on the
CPU.  The tests hold the CUDA kernels to them."""
import numpy as np


# ------------------------------------------------------------- page tables
def page_tables(lengths, new_rows, held, table, ring, ring_state, page, row_cap):
    """(held, table, ring, ring_state, row_offsets, slots, positions, capacity flag)"""
    table, ring, held = table.copy(), ring.copy(), held.copy()
    n_pages, width = len(ring), table.shape[1]
    head, count = int(ring_state[0]), int(ring_state[1])
    before = count
    flag = False
    ask = taken = given = 0
    rows, offsets = [], [0]
    for s in range(len(lengths)):
        n, r = int(lengths[s]), int(new_rows[s])
        if n < 0 or r < 0:
            offsets.append(offsets[-1])
            continue
        need, ok = -(-(n + r) // page), True
        if need > width:
            flag, ok = True, False
        elif need > held[s]:
            take = need - int(held[s])
            if ask + take > before:
                flag, ok = True, False
            else:
                for i in range(take):
                    table[s, held[s] + i] = ring[(head + ask + i) % n_pages]
                held[s] = need
                taken += take
            ask += take
        elif need < held[s]:
            for i in range(need, held[s]):
                if before + given < n_pages:
                    ring[(head + before + given) % n_pages] = table[s, i]
                    given += 1
                else:
                    flag = True
            held[s] = need
        for j in range(r):
            p = n + j
            slot = -1
            if ok:
                pid = int(table[s, p // page])
                if 0 <= pid < n_pages:
                    slot = pid * page + p % page
                else:
                    flag = True
            rows.append((slot, p))
        offsets.append(offsets[-1] + r)
    slots = np.full(row_cap, -1, np.int32)
    positions = np.full(row_cap, -1, np.int32)
    for i, (slot, p) in enumerate(rows[:row_cap]):
        slots[i], positions[i] = slot, p
    flag |= len(rows) > row_cap
    state = np.array([(head + taken) % n_pages, before - taken + given], np.int32)
    return held, table, ring, state, np.array(offsets, np.int32), slots, positions, flag


# ----------------------------------------------------------------- the cache
def word_places(d):
    """Byte offsets in a 16-cell group: K codes, V codes [16, d / 2] and K, V scales [16, d / 32], in channel order."""
    kc, vc = np.zeros((16, d // 2), np.int64), np.zeros((16, d // 2), np.int64)
    ks, vs = np.zeros((16, d // 32), np.int64), np.zeros((16, d // 32), np.int64)
    for c in range(16):
        for w in range(d // 8):
            k = ((w % 4) * (d // 32) + w // 4) ^ (4 * ((c // 4) % 2) if d == 256 else 0)
            swap = 2 * (c % 4) if d == 256 else 4 * ((c // 2) % 2) if d == 128 else 0
            v = ((w % 8) ^ swap) * (d // 64) + w // 8
            for i in range(4):
                kc[c, 4 * w + i] = c * (d // 2) + 4 * k + i
                vc[c, 4 * w + i] = 9 * d + c * (d // 2) + 4 * v + i
        for b in range(d // 32):
            ks[c, b] = 8 * d + c * (d // 16) + 2 * b
            vs[c, b] = 17 * d + c * (d // 16) + 2 * ((b % 2) * (d // 64) + b // 2)
    return kc, vc, ks, vs


def quantise(x):
    """[..., d] -> codes [..., d] (0..15) and FP16 scales [..., d / 32]."""
    b = np.asarray(x, np.float64).reshape(x.shape[:-1] + (-1, 32))
    at = np.argmax(np.abs(b), -1)  # the first of equals
    m = np.take_along_axis(b, at[..., None], -1)
    d = (m / -8).astype(np.float16)
    df = d.astype(np.float64)
    q = np.rint(np.divide(b, df, out=np.zeros_like(b), where=df != 0))
    return (np.clip(q, -8, 7) + 8).astype(np.uint8).reshape(x.shape), d[..., 0]


def dequantise(codes, scales):
    return (codes.astype(np.float64) - 8) * np.repeat(scales.astype(np.float64), 32, -1)


def store(cache, slots, k, v):
    """Writes rows [n, heads, d] into the cache (numpy uint8 [pages, heads, groups, 18 d]) cell by cell."""
    n_pages, heads, groups, size = cache.shape
    d = size // 18
    kc, vc, ks, vs = word_places(d)
    for x, code_at, scale_at in ((k, kc, ks), (v, vc, vs)):
        codes, scales = quantise(x)
        for r, slot in enumerate(slots):
            if slot < 0 or slot >= n_pages * groups * 16:
                continue
            page, off = divmod(int(slot), groups * 16)
            g, c = divmod(off, 16)
            for h in range(heads):
                grp = cache[page, h, g]
                grp[code_at[c]] = codes[r, h, 0::2] | (codes[r, h, 1::2] << 4)
                sb = scales[r, h].view(np.uint8).reshape(-1, 2)
                grp[scale_at[c]] = sb[:, 0]
                grp[scale_at[c] + 1] = sb[:, 1]


def load(cache, slots):
    """(k, v) float64 [n, heads, d] of cells; zeros for slots outside."""
    n_pages, heads, groups, size = cache.shape
    d = size // 18
    kc, vc, ks, vs = word_places(d)
    out = []
    slots = np.asarray(slots)
    live = (slots >= 0) & (slots < n_pages * groups * 16)
    sl = np.where(live, slots, 0).astype(np.int64)
    page, off = np.divmod(sl, groups * 16)
    g, c = np.divmod(off, 16)
    grp = cache[page, :, g]  # [n, heads, size]
    for code_at, scale_at in ((kc, ks), (vc, vs)):
        by = np.take_along_axis(grp, np.broadcast_to(code_at[c][:, None], (len(sl), heads, d // 2)), -1)
        codes = np.stack([by & 15, by >> 4], -1).reshape(len(sl), heads, d)
        lo = np.take_along_axis(grp, np.broadcast_to(scale_at[c][:, None], (len(sl), heads, d // 32)), -1)
        hi = np.take_along_axis(grp, np.broadcast_to(scale_at[c][:, None] + 1, (len(sl), heads, d // 32)), -1)
        scales = (lo.astype(np.uint16) | (hi.astype(np.uint16) << 8)).view(np.float16)
        out.append(np.where(live[:, None, None], dequantise(codes, scales), 0.0))
    return out


# ----------------------------------------------------------------- attention
def attention(cache, q, table, kv_len, offsets, causal, window, scale):
    """(o [tokens, nq, d], spread [tokens, nq, d] = sum p |v| / sum p, top score in natural units, cells seen) in 64 bits.
    Rows of no sequence are NaN in o."""
    n_pages, heads, groups, size = cache.shape
    page, d = groups * 16, size // 18
    nq = q.shape[1]
    G = nq // heads
    o = np.full(q.shape, np.nan)
    spread = np.zeros(q.shape)
    top = np.zeros(q.shape[:2])
    seen = np.zeros(q.shape[:2])
    for s in range(len(kv_len)):
        r0, r1, n = int(offsets[s]), int(offsets[s + 1]), max(int(kv_len[s]), 0)
        pos = np.arange(n)
        k, v = load(cache, table[s, pos // page].astype(np.int64) * page + pos % page) if n else (None, None)
        for i in range(r1 - r0):
            last = n - (r1 - r0) + i if causal else n - 1
            lo = max(last - window + 1, 0) if window else 0
            for h in range(nq):
                if last < lo or last < 0:
                    o[r0 + i, h] = 0
                    continue
                x = scale * (k[lo:last + 1, h // G] @ q[r0 + i, h].astype(np.float64))
                p = np.exp(x - x.max())
                vv = v[lo:last + 1, h // G]
                o[r0 + i, h] = p @ vv / p.sum()
                spread[r0 + i, h] = p @ np.abs(vv) / p.sum()
                top[r0 + i, h] = np.abs(x).max()
                seen[r0 + i, h] = last + 1 - lo
    return o, spread, top, seen


# ------------------------------------------------------------------ logprobs
def logprobs(x, tokens, k):
    """(logp, entropy, ids, top logp, sum p |x - m|) of float64 logits."""
    n, vocab = x.shape
    m = x.max(-1)
    ok = m > -np.inf
    z = np.where(ok[:, None], x - np.where(ok, m, 0)[:, None], -np.inf)
    e = np.exp(z)
    s = e.sum(-1)
    ls = np.log(np.where(ok, s, 1))
    ez = np.where(e > 0, e * np.where(e > 0, z, 0), 0).sum(-1) / np.where(ok, s, 1)
    entropy = np.where(ok, ls - ez, 0)
    logp = np.zeros(n)
    for i, t in enumerate(tokens):
        if 0 <= t < vocab:
            logp[i] = z[i, t] - ls[i]
    order = np.argsort(-z, axis=-1, kind="stable")[:, :k]
    val = np.take_along_axis(z, order, -1)
    ids = np.where(val > -np.inf, order, -1)
    top = np.where(val > -np.inf, val - ls[:, None], -np.inf)
    if ids.shape[1] < k:
        pad = k - ids.shape[1]
        ids = np.pad(ids, ((0, 0), (0, pad)), constant_values=-1)
        top = np.pad(top, ((0, 0), (0, pad)), constant_values=-np.inf)
    return logp, entropy, ids, top, -ez
