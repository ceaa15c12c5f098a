"""Operators of a sampling serving step, measured: per-head norms with the position rotation, attention of requests that share a long
prefix over the 4-bit paged cache, and sampling from the verifier's logits.

Every operator has a plain form (elementary torch operations in 32 bits; angles, and the sums that a sampled id goes by, in 64)
and, with `own` set, the call that a user makes of the framework.  The sizes are those of the framework's own workloads (24 query
and 2 K/V heads of 256 channels, contexts of 8192 and 32768 positions, blocks of up to 8 rows, 16 sequences, a vocabulary of
151936) and generic ones.

The cache is a uint8 tensor [pages, kv heads, page size / 16, 18 * head_dim].  A group of 16 cells holds the K codes
(16 rows of head_dim / 2 bytes), the K scales (16 rows of head_dim / 32 FP16), the V codes and the V scales.  A code is
4 bits, the value of channel c is scale[c / 32] * (code - 8).  Channels 8w .. 8w + 7 make the 32-bit word w of a row, the even
channel of a byte in its low half; the words and the V scales of a row are stored in the order of `_orders`.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
GROUP = 16  # cells of a group
MOST_CELLS = 64 * 24 * 256 * 36000  # tokens x query heads x channels x cells of the largest attention case


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one verify block of 8 rows: launch latency
        dict(name="rope_block_8", op="rope", rows=8, nq=24, nkv=2, d=256, rot=256, axes=1, far=262144, norm=True, type="bf16", mix=1),
        # the blocks of 16 sequences, FP16, a quarter of the channels rotated
        dict(name="rope_step_128", op="rope", rows=128, nq=24, nkv=2, d=256, rot=64, axes=1, far=32768, norm=True, type="fp16", mix=2),
        # an image prompt: positions in time, height and width, queries and keys without a norm
        dict(name="rope_image_4097", op="rope", rows=4097, nq=16, nkv=16, d=64, rot=64, axes=3, far=4096, norm=False, type="bf16", mix=3),
        # a long prompt, 32 / 8 heads of 128
        dict(name="rope_prompt_30001", op="rope", rows=30001, nq=32, nkv=8, d=128, rot=128, axes=1, far=30001, norm=True, type="bf16", mix=4),
        # single tokens of eight requests with the same instructions of 8192 positions
        dict(name="prefix_token_8x8k", op="prefix", groups=1, n_seq=8, rows=1, nq=24, nkv=2, d=256, page=64, plo=8192, phi=8192, lo=1, hi=511, causal=True,
             type="bf16", mix=5),
        # a loaded server: 200 requests in five groups of other instructions, 32 / 8 heads of 128, odd lengths
        dict(name="prefix_token_200x5", op="prefix", groups=5, n_seq=200, rows=1, nq=32, nkv=8, d=128, page=16, plo=700, phi=6001, lo=1, hi=1023, causal=True,
             type="fp16", mix=6),
        # verify blocks of 2..8 rows of 16 sequences over one document of 32768 positions
        dict(name="prefix_block_16x32k", op="prefix", groups=1, n_seq=16, rows=8, nq=24, nkv=2, d=256, page=64, plo=32768, phi=32768, lo=8, hi=2048, causal=True,
             type="bf16", mix=7),
        # single tokens of 64 samples of one long prompt
        dict(name="prefix_token_64x32k", op="prefix", groups=1, n_seq=64, rows=1, nq=24, nkv=2, d=256, page=128, plo=32768, phi=32768, lo=1, hi=4096, causal=True,
             type="bf16", mix=8),
        # the rows of one verify block, nucleus sampling
        dict(name="sample_block_8", op="sample", rows=8, vocab=151936, mode="top_p", mask=0, type="bf16", mix=9),
        # the blocks of 16 sequences, each request with settings of its own, an odd vocabulary in FP32 with a grammar's mask
        dict(name="sample_step_128", op="sample", rows=128, vocab=100003, mode="mixed", mask=1, type="fp32", mix=10),
        # a token for each request of a large batch, the 50 best
        dict(name="sample_batch_256", op="sample", rows=256, vocab=151936, mode="top_k", mask=0, type="fp16", mix=11),
        # many continuations drawn from the whole distribution
        dict(name="sample_many_1000", op="sample", rows=1000, vocab=151936, mode="temperature", mask=0, type="bf16", mix=12),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "prefix", "prefix", "sample", "sample"])
    mix = rng.randrange(1 << 20)
    if op == "rope":
        d, nkv = rng.choice([64, 128, 256]), rng.randint(1, 8)
        nq = nkv * rng.randint(1, 12)
        rot = rng.choice([d, d, d // 2, d // 4])
        return dict(op=op, rows=_spread(rng, 1, min(40000, 30000 * 40 * 128 // ((nq + nkv) * d))), nq=nq, nkv=nkv, d=d, rot=rot, axes=rng.choice([1, 1, 3]),
                    far=_spread(rng, 1, 262144), norm=rng.random() < 0.7, type=rng.choice(["bf16", "fp16"]), mix=mix)
    if op == "prefix":
        d, nkv, rows = rng.choice([64, 128, 256]), rng.randint(1, 8), rng.randint(1, 8)
        group = rng.randint(1, 16 if d < 256 else 12)
        n = _spread(rng, 1, 200)
        groups = rng.randint(1, min(n, 6))
        cells = max(64, min(60000, MOST_CELLS // (n * rows * nkv * group * d), 262144 * 512 // (nkv * d * groups)))
        plo = _spread(rng, 1, cells)
        return dict(op=op, groups=groups, n_seq=n, rows=rows, nq=nkv * group, nkv=nkv, d=d, page=rng.choice([16, 32, 64, 128]), plo=plo,
                    phi=_spread(rng, plo, cells), lo=rng.randint(1, 8), hi=_spread(rng, 8, max(8, min(2048, cells // 8))), causal=rng.random() < 0.7,
                    type=rng.choice(["bf16", "fp16"]), mix=mix)
    vocab = _spread(rng, 1000, 200000)
    kind = rng.choice(["bf16", "fp16", "fp32"])
    return dict(op=op, rows=_spread(rng, 1, max(1, min(1000, 1000 * 151936 // (vocab * (2 if kind == "fp32" else 1))))), vocab=vocab,
                mode=rng.choice(["temperature", "top_p", "top_k", "mixed", "mixed"]), mask=rng.randint(0, 1), type=kind, mix=mix)


def _requests(case):
    """Prefix cells of each group, first sequence of each group, own cells and rows of each sequence: they go by the case alone."""
    rng = random.Random(case["mix"])
    n, groups = case["n_seq"], case["groups"]
    cuts = sorted(rng.sample(range(1, n), groups - 1)) if groups > 1 else []
    starts = [0] + cuts + [n]
    prefix = [rng.randint(case["plo"], case["phi"]) for _ in range(groups)]
    rows = [case["rows"] if n == 1 or case["rows"] == 1 else rng.randint(2, case["rows"]) for _ in range(n)]
    lens = [max(r, rng.randint(case["lo"], case["hi"])) for r in rows]
    return prefix, starts, lens, rows


def work(case):
    if case["op"] == "rope":
        n = case["rows"] * (case["nq"] + case["nkv"]) * case["d"]
        return {"bytes": 4 * n + 4 * case["axes"] * case["rows"], "flops": 8 * n}
    if case["op"] == "prefix":
        prefix, starts, lens, rows = _requests(case)
        size = {"bytes": 0, "flops": 0}
        for g, p in enumerate(prefix):
            size["bytes"] += p * case["nkv"] * case["d"] * 1.125 + 4 * -(-p // case["page"])
            for s in range(starts[g], starts[g + 1]):
                size["bytes"] += lens[s] * case["nkv"] * case["d"] * 1.125 + 2 * 2 * rows[s] * case["nq"] * case["d"] + 4 * -(-lens[s] // case["page"])
                size["flops"] += 4 * rows[s] * case["nq"] * case["d"] * (p + lens[s])
        return size
    n = case["rows"] * case["vocab"]
    return {"bytes": n * (4 if case["type"] == "fp32" else 2) + case["rows"] * 32, "flops": 4 * n}


# ------------------------------------------------------------------ inputs
def _orders(d):
    """The stored place of word w of the K row and of the V row of each of a group's 16 cells, as byte offsets [16, d / 2] in the
    group, and the place of the V scale of 32-channel block b in its row [d / 32]."""
    cell = torch.arange(GROUP)[:, None]
    w = torch.arange(d // 8)[None, :]
    k = (w % 4) * (d // 32) + w // 4
    if d == 256:  # 16-byte chunks of odd quads change places in pairs
        k = k ^ (((cell >> 2) & 1) << 2)
    v_chunk = w % 8
    if d == 256:
        v_chunk = v_chunk ^ ((cell & 3) << 1)
    elif d == 128:
        v_chunk = v_chunk ^ (((cell >> 1) & 1) << 2)
    v = v_chunk * (d // 64) + w // 8
    four = torch.arange(4)
    row = cell * (d // 2)
    k_bytes = (row + 4 * (k + 0 * cell))[:, :, None] + four
    v_bytes = (9 * d + row + 4 * (v + 0 * cell))[:, :, None] + four
    b = torch.arange(d // 32)
    return k_bytes.reshape(GROUP, -1), v_bytes.reshape(GROUP, -1), (b % 2) * (d // 64) + b // 2


def _layout(d, device):
    """Byte offsets in a group: codes [2, 16, d / 2] and scales [2, 16, d / 16] of K and V, in the order of the channels."""
    k, v, order = _orders(d)
    cell = torch.arange(GROUP)[:, None]
    two = torch.arange(2)
    ks = 8 * d + cell[:, :, None] * (d // 16) + (2 * torch.arange(d // 32)[None, :])[:, :, None] + two
    vs = 17 * d + cell[:, :, None] * (d // 16) + (2 * order[None, :])[:, :, None] + two
    return torch.stack([k, v]).to(device), torch.stack([ks.reshape(GROUP, -1), vs.reshape(GROUP, -1)]).to(device)


def _quantise(x):
    """[..., d] values -> codes as bytes [..., d / 2] and FP16 scales [..., d / 32]."""
    b = x.float().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    at = (b.abs() == top).to(torch.int8).argmax(-1, keepdim=True)
    d = (b.gather(-1, at) * -0.125).half()
    df = d.float()
    q = torch.where(df != 0, torch.round(b / torch.where(df != 0, df, torch.ones_like(df))), torch.zeros_like(b))
    codes = (q.clamp(-8, 7) + 8).to(torch.uint8).flatten(-2)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), d.squeeze(-1)


def _fill(cache, layout, gen):
    """Quantised normal rows in every cell, those of no request too; K's channels are of unequal size."""
    n_pages, heads, groups, size = cache.shape
    page, d = groups * GROUP, size // 18
    codes, scales = layout
    gain = torch.exp(0.3 * _normal((heads, d), gen))
    step = max(1, (1 << 24) // (heads * page * d))
    for at in range(0, n_pages, step):
        m = min(step, n_pages - at)
        part = cache[at:at + m].view(m, heads, groups, size)
        for side in (0, 1):
            x = _normal((m, heads, groups, GROUP, d), gen)
            q, s = _quantise(x * gain[:, None, None, :] if side == 0 else x)
            part[..., codes[side].reshape(-1)] = q.flatten(-2)
            part[..., scales[side].reshape(-1)] = s.contiguous().view(torch.uint8).flatten(-2)


def _values(codes, scales):
    """Packed codes [..., d / 2] and the bytes of scales [..., d / 16] -> FP32 values [..., d]."""
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float() - 8
    d = scales.contiguous().view(torch.float16).float()
    return (q.unflatten(-1, (-1, 32)) * d[..., None]).flatten(-2)


def _normal(shape, gen, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(counts, order, used):
    """A page table [requests, widest] of the next pages of `order` behind the first `used`; -1 behind a request's last page."""
    c = _ints(counts).long()
    col = torch.arange(max(1, max(counts)), device="cuda")
    at = used + (c.cumsum(0) - c)[:, None] + col
    return torch.where(col < c[:, None], order[at.clamp(max=order.numel() - 1)], torch.full((), -1, dtype=torch.int32, device="cuda")).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    if case["op"] == "rope":
        n, nq, nkv, d, rot = case["rows"], case["nq"], case["nkv"], case["d"], case["rot"]
        # rows of the fused projection's output: queries, keys and values of a row lie in one row of it
        x = _normal((n, (nq + 2 * nkv) * d), gen) * torch.exp(0.5 * _normal((1, (nq + 2 * nkv) * d), gen))
        x = x.to(TYPES[case["type"]])
        freqs = [1e7 ** (-2.0 * j / rot) for j in range(rot // 2)]
        # the table that a program keeps: the part of a turn per position, 64 binary places
        turns = [int(f / (2 * math.pi) * 2.0 ** 64) for f in freqs]
        turns = torch.tensor([t - (1 << 64) if t >= 1 << 63 else t for t in turns], dtype=torch.int64, device="cuda")
        axis = None
        if case["axes"] == 1:
            positions = (torch.arange(n, device="cuda") + max(0, case["far"] - n)).int()
            positions[: n // 3] = torch.randint(0, case["far"], (n // 3,), generator=gen, device="cuda", dtype=torch.int32)
        else:  # patches of images in a row of text: the axes take turns over the frequencies
            positions = torch.randint(0, case["far"], (case["axes"], n), generator=gen, device="cuda", dtype=torch.int32)
            axis = (torch.arange(rot // 2, device="cuda") % case["axes"]).to(torch.uint8)
        weights = [1.0 + 0.2 * _normal((d,), gen) if case["norm"] else None for _ in range(2)]
        return dict(op="rope", q=x[:, : nq * d].unflatten(-1, (nq, d)), k=x[:, nq * d:(nq + nkv) * d].unflatten(-1, (nkv, d)), positions=positions, axis=axis,
                    freqs=torch.tensor(freqs, dtype=torch.float64, device="cuda"), turns=turns, q_weight=weights[0], k_weight=weights[1], eps=1e-6)
    if case["op"] == "prefix":
        prefix, starts, lens, rows = _requests(case)
        page, d, nkv = case["page"], case["d"], case["nkv"]
        shared, owned = [-(-p // page) for p in prefix], [-(-n // page) for n in lens]
        n_pages = sum(shared) + sum(owned) + 3
        order = torch.randperm(n_pages, generator=gen, device="cuda").int()
        cache = torch.empty((n_pages, nkv, page // GROUP, 18 * d), dtype=torch.uint8, device="cuda")
        layout = _layout(d, "cuda")
        _fill(cache, layout, gen)
        offsets = [0]
        for r in rows:
            offsets.append(offsets[-1] + r)
        q = (2.0 * _normal((offsets[-1], case["nq"], d), gen)).to(TYPES[case["type"]])
        return dict(op="prefix", cache=cache, layout=layout, q=q, prefix_table=_table(shared, order, 0), prefix_len=_ints(prefix), group_offsets=_ints(starts),
                    table=_table(owned, order, sum(shared)), kv_len=_ints(lens), offsets=_ints(offsets), rows=case["rows"], causal=case["causal"],
                    in_group=max(offsets[b] - offsets[a] for a, b in zip(starts, starts[1:])))
    n, vocab = case["rows"], case["vocab"]
    x = torch.empty((n, vocab), dtype=TYPES[case["type"]], device="cuda")
    spread = 0.4 + 0.6 * torch.rand((n, 1), generator=gen, device="cuda")  # rows that are sure and rows that are not
    step = max(1, (1 << 27) // vocab)
    for at in range(0, n, step):  # logits with a heavy head: a few tokens carry most of the weight
        part = _normal((min(step, n - at), vocab), gen)
        x[at:at + step] = ((2.0 * part + 0.25 * part ** 3) * spread[at:at + step]).to(x.dtype)
    if case["mask"]:  # a grammar leaves about a third of the tokens, and for one row a single one
        x.masked_fill_(torch.rand((1, vocab), generator=gen, device="cuda") < 0.66, -math.inf)
        x[0].fill_(-math.inf)
        x[0, rng.randrange(vocab)] = 1.5
    uniform = torch.rand((n,), generator=gen, device="cuda")
    temperature = 0.6 + 0.6 * torch.rand((n,), generator=gen, device="cuda")
    top_k = top_p = min_p = None
    if case["mode"] == "top_k":
        top_k = torch.full((n,), 50, dtype=torch.int32, device="cuda")
    elif case["mode"] == "top_p":
        top_p = 0.9 + 0.08 * torch.rand((n,), generator=gen, device="cuda")
    elif case["mode"] == "mixed":  # one in eight greedy, and each filter off (0, 1, 0) for a part of the requests
        off = torch.rand((4, n), generator=gen, device="cuda")
        temperature = torch.where(off[0] < 0.125, torch.zeros_like(temperature), temperature)
        top_k = torch.where(off[1] < 0.5, 0, torch.randint(1, 200, (n,), generator=gen, device="cuda")).int()
        top_p = torch.where(off[2] < 0.3, 1.0, 0.8 + 0.19 * torch.rand((n,), generator=gen, device="cuda")).float()
        min_p = torch.where(off[3] < 0.5, 0.0, 0.1 * torch.rand((n,), generator=gen, device="cuda")).float()
    return dict(op="sample", x=x, uniform=uniform, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)


# ------------------------------------------------------------------ the plain forms
def _plain_rope(s):
    half = s["freqs"].numel()
    positions = s["positions"].double()
    if s["axis"] is None:
        angle = positions[:, None] * s["freqs"]
    else:
        angle = positions.transpose(0, 1)[:, s["axis"].long()] * s["freqs"]
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    out = []
    for name in ("q", "k"):
        x = s[name].float()
        if s[name + "_weight"] is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * s[name + "_weight"]
        a, b = x[..., :half], x[..., half:2 * half]
        out.append(torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., 2 * half:]], -1).to(s[name].dtype))
    return out


def _pages(cache, layout, table):
    """K and V of every request's cells, padded to the widest: [requests, kv heads, cells, d]."""
    codes, scales = layout
    d = cache.shape[-1] // 18
    cells = cache[table.clamp(min=0).long()]  # [requests, pages, kv heads, groups, size]
    return [_values(cells[..., codes[i]], cells[..., scales[i]]).permute(0, 2, 1, 3, 4, 5).reshape(table.shape[0], cache.shape[1], -1, d) for i in (0, 1)]


def _partial(rows, k, v, sees):
    """Maximum, sum and unnormalised output of rows [n, kv heads, rows, d] over the cells that each sees, `sees` [n, 1, rows, cells]."""
    scores = (rows @ k.transpose(-1, -2) * rows.shape[-1] ** -0.5).masked_fill(~sees, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    return top, p.sum(-1, keepdim=True), p @ v


def _plain_prefix(s):
    q, most, wide = s["q"], s["rows"], s["in_group"]
    total, nq, d = q.shape
    nkv = s["cache"].shape[1]
    per = nq // nkv
    offsets, starts, kv_len, prefix_len = (s[k].long() for k in ("offsets", "group_offsets", "kv_len", "prefix_len"))
    token = torch.arange(total, device=q.device)
    seq = torch.searchsorted(offsets, token, right=True) - 1
    group = torch.searchsorted(starts, seq, right=True) - 1
    heads = q.float().unflatten(1, (nkv, per))  # [tokens, kv heads, per, d]

    def pad(first, width):  # [n, kv heads, width * per, d] of the tokens from each of `first` on
        at = (first[:, None] + torch.arange(width, device=q.device)).clamp(max=total - 1)
        return heads[at].permute(0, 2, 1, 3, 4).reshape(first.numel(), nkv, width * per, d)

    def of_tokens(parts, n, i):  # back to [tokens, kv heads, per, ..]
        return [x.unflatten(2, (-1, per)).permute(0, 2, 1, 3, 4)[n, i] for x in parts]

    first = offsets[starts[:-1]]
    k, v = _pages(s["cache"], s["layout"], s["prefix_table"])
    sees = (torch.arange(k.shape[2], device=q.device) < prefix_len[:, None])[:, None, None, :]
    shared = of_tokens(_partial(pad(first, wide), k, v, sees), group, token - first[group])
    del k, v
    k, v = _pages(s["cache"], s["layout"], s["table"])
    i = torch.arange(most, device=q.device)
    count = offsets[1:] - offsets[:-1]
    last = kv_len[:, None] - count[:, None] + i if s["causal"] else (kv_len - 1)[:, None] + 0 * i
    sees = (torch.arange(k.shape[2], device=q.device) <= last[:, :, None]).repeat_interleave(per, 1)[:, None]
    mine = of_tokens(_partial(pad(offsets[:-1], most), k, v, sees), seq, token - offsets[seq])
    top = torch.maximum(shared[0], mine[0])
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    a, b = torch.exp(shared[0] - top), torch.exp(mine[0] - top)
    weight = a * shared[1] + b * mine[1]
    o = (a * shared[2] + b * mine[2]) / torch.where(weight > 0, weight, torch.ones_like(weight))
    return o.reshape(total, nq, d).to(q.dtype)


def _plain_sample(s):
    x = s["x"]
    n, vocab = x.shape
    greedy = s["temperature"] <= 0
    temperature = torch.where(greedy, torch.ones_like(s["temperature"]), s["temperature"]).double()[:, None]
    top = x.amax(-1, keepdim=True)
    least = torch.full((n, 1), -math.inf, dtype=torch.float64, device=x.device)
    if s["top_k"] is not None or s["top_p"] is not None:
        v = x.float().sort(-1, descending=True).values
        kept = torch.ones_like(v, dtype=torch.bool)
        if s["top_k"] is not None:
            k = torch.where((s["top_k"] <= 0) | (s["top_k"] > vocab), vocab, s["top_k"]).long()
            kept = v >= v.gather(-1, k[:, None] - 1)
        w = torch.exp((v.double() - top.double()) / temperature) * kept
        if s["top_p"] is not None:
            upto = w.cumsum(-1)
            p = s["top_p"].double()[:, None]
            kept &= (upto - w < p * upto[:, -1:]) | (p >= 1)
            del upto
        del w
        kept[:, 0] = True
        least = torch.where(kept, v, torch.full_like(v, math.inf)).amin(-1, keepdim=True).double()
        del v, kept
    w = torch.exp((x.double() - top.double()) / temperature)
    kept = (x >= least) & (x > -math.inf)
    if s["min_p"] is not None:
        kept &= w >= s["min_p"].double()[:, None]
    w *= kept
    count = kept.sum(-1)
    upto = w.cumsum(-1)
    whole = upto[:, -1:]
    token = (upto <= s["uniform"].double()[:, None] * whole).sum(-1)
    best = (x == top).to(torch.uint8).argmax(-1)  # the first of equals
    token = torch.where(greedy, best, token)
    logp = torch.log(w.gather(-1, token[:, None]) / whole).squeeze(-1)
    return dict(token=token.int(), logp=torch.where(greedy, torch.zeros_like(logp), logp).float(), kept=torch.where(greedy, torch.ones_like(count), count).int())


# ------------------------------------------------------------------ one pass
def run(state):
    s = state
    if own:
        from dflash_block_drafter_gb300 import runtime as R
        if s["op"] == "rope":
            return R.qk_norm_rope(s["q"], s["k"], s["positions"], s["turns"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"], axes=s["axis"])
        if s["op"] == "prefix":
            return R.kv4_prefix_attention(s["cache"], s["q"], s["prefix_table"], s["prefix_len"], s["group_offsets"], s["table"], s["kv_len"], s["offsets"],
                                          s["rows"], causal=s["causal"])
        token, logp, kept = R.sample_tokens(s["x"], s["uniform"], s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
        return dict(token=token, logp=logp, kept=kept)
    if s["op"] == "rope":
        return _plain_rope(s)
    if s["op"] == "prefix":
        return _plain_prefix(s)
    return _plain_sample(s)


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _cells_64(cache, slots, d):
    """[cells, heads, d] K and V of the cells, byte by byte from the format."""
    n_pages, heads, groups, size = cache.shape
    rows = cache.permute(0, 2, 1, 3).reshape(n_pages * groups, heads, size)
    group = rows[(slots // GROUP).long()]
    cell = (slots % GROUP).long()
    k_at, v_at, order = (t.to(cache.device) for t in _orders(d))
    take = lambda at: group.gather(-1, at[:, None, :].expand(-1, heads, -1))  # noqa: E731
    side = []
    for at, scale_at in ((k_at, 8 * d + 2 * torch.arange(d // 32, device=cache.device)), (v_at, 17 * d + 2 * order)):
        codes = take(at[cell]).to(torch.int16)
        at2 = (cell * (d // 16))[:, None] + scale_at
        low, high = take(at2).to(torch.int16), take(at2 + 1).to(torch.int16)
        scale = (low | (high << 8)).view(torch.float16).double()
        x = torch.empty(codes.shape[:-1] + (d,), dtype=torch.float64, device=cache.device)
        x[..., 0::2] = (codes % 16) - 8
        x[..., 1::2] = (codes // 16) - 8
        side.append(x * scale.repeat_interleave(32, -1))
    return side


def _slots(table, n, page):
    return (table[: -(-n // page)].long()[:, None] * page + torch.arange(page, device=table.device)).reshape(-1)[:n]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        out = []
        half = case["rot"] // 2
        for name in ("q", "k"):
            x = s[name].double()
            if case["norm"]:
                x = x * (x.pow(2).sum(-1, keepdim=True) / case["d"] + 1e-6).rsqrt() * s[name + "_weight"].double()
            z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous())
            where = s["positions"].double()[None] if case["axes"] == 1 else s["positions"].double()
            turn = torch.stack([where[j % case["axes"]] * s["freqs"][j] for j in range(half)], -1)
            z = z * torch.polar(torch.ones_like(turn), turn)[:, None, :]
            out.append(torch.cat([z.real, z.imag, x[..., 2 * half:]], -1))
        return out
    if case["op"] == "prefix":
        prefix, starts, lens, rows = _requests(case)
        d, nkv, page, per = case["d"], case["nkv"], case["page"], case["nq"] // case["nkv"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        r0 = 0
        for g, p in enumerate(prefix):
            both = _cells_64(s["cache"], _slots(s["prefix_table"][g], p, page), d)
            for i in range(starts[g], starts[g + 1]):
                n, r = lens[i], rows[i]
                mine = _cells_64(s["cache"], _slots(s["table"][i], n, page), d)
                at = torch.arange(n, device="cuda")
                last = torch.arange(n - r, n, device="cuda") if case["causal"] else torch.full((r,), n - 1, device="cuda")
                hidden = at[None, :] > last[:, None]
                for h in range(nkv):
                    q = s["q"][r0:r0 + r, h * per:(h + 1) * per].double().transpose(0, 1).reshape(per * r, d)
                    x = torch.cat([q @ both[0][:, h].T, (q @ mine[0][:, h].T).masked_fill_(hidden.repeat(per, 1), -math.inf)], -1) / math.sqrt(d)
                    w = torch.softmax(x, -1)
                    o = w[:, :p] @ both[1][:, h] + w[:, p:] @ mine[1][:, h]
                    out[r0:r0 + r, h * per:(h + 1) * per] = o.view(per, r, d).transpose(0, 1)
                r0 += r
        return out
    logp = []
    for i in range(case["rows"]):
        t = float(s["temperature"][i])
        if t <= 0:
            logp.append(torch.zeros((), dtype=torch.float64, device="cuda"))
            continue
        x = s["x"][i].double()
        live = x > -math.inf
        if s["top_k"] is not None and 0 < int(s["top_k"][i]) < case["vocab"]:
            live &= x >= x.kthvalue(case["vocab"] + 1 - int(s["top_k"][i])).values
        p = torch.softmax(torch.where(live, x / t, torch.full_like(x, -math.inf)), -1)
        if s["top_p"] is not None and float(s["top_p"][i]) < 1:
            level, which = torch.unique(x[live], return_inverse=True)  # ascending
            mass = torch.zeros_like(level).index_add_(0, which, p[live])
            above = mass.flip(0).cumsum(0).flip(0) - mass
            live &= x >= level[above < float(s["top_p"][i])].min()
        if s["min_p"] is not None:
            live &= x - x.max() >= t * math.log(max(float(s["min_p"][i]), 1e-300))
        ids = live.nonzero().squeeze(-1)
        q = torch.softmax(x[ids] / t, 0)
        at = torch.searchsorted(q.cumsum(0), s["uniform"][i].double(), right=True).clamp(max=ids.numel() - 1)
        logp.append(torch.log_softmax(x[ids] / t, 0)[at])
    return dict(token=None, logp=torch.stack(logp), kept=None)
