"""The verify-step operators, measured: page bookkeeping, the 4-bit paged K/V cache (write and read back), attention over
it, and token log probabilities.

Every operator has a plain form (elementary torch operations in 32 bits) and, with `own` set, the call that a user makes of
the framework.  The sizes are those of the framework's own workloads (24 query and 2 K/V heads of 256 channels, contexts of
8192, 2048..32768 and 262144 positions, blocks of up to 8 rows, 16 sequences, a vocabulary of 151936) and generic ones.

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


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one serving step of 16 sequences with blocks of 8 rows: every call is launch latency
        dict(name="pages_step_16", op="pages", n_seq=16, page=64, lo=2048, hi=32768, rows=8, prefill=0, mix=1),
        # a loaded server: 2000 requests, most decode, some just arrived with long prompts, some finished
        dict(name="pages_server_2000", op="pages", n_seq=2000, page=16, lo=1, hi=8191, rows=4, prefill=40, mix=2),
        # the cells of one step of 16 sequences, FP16 as the drafter's own cells
        dict(name="write_step_128", op="write", rows=128, heads=2, d=256, page=64, pages=512, type="fp16", pad=5, mix=3),
        # the cells of a long prompt, BF16, 8 heads of 128
        dict(name="write_prompt_30001", op="write", rows=30001, heads=8, d=128, page=32, pages=1100, type="bf16", pad=0, mix=4),
        # one token after an 8192-position context: the smallest attention call
        dict(name="attn_token_8k", op="attention", n_seq=1, rows=1, nq=24, nkv=2, d=256, page=64, lo=8192, hi=8192, window=0,
             causal=True, type="bf16", mix=5),
        # single tokens of the batched serving mix
        dict(name="attn_token_mix16", op="attention", n_seq=16, rows=1, nq=24, nkv=2, d=256, page=64, lo=2048, hi=32768, window=0,
             causal=True, type="fp16", mix=6),
        # single tokens of many short requests, 32 / 8 heads of 128, odd lengths
        dict(name="attn_token_200x1k", op="attention", n_seq=200, rows=1, nq=32, nkv=8, d=128, page=16, lo=1, hi=2047, window=0,
             causal=True, type="bf16", mix=7),
        # verify blocks of 8 rows of the batched serving mix
        dict(name="attn_block_mix16", op="attention", n_seq=16, rows=8, nq=24, nkv=2, d=256, page=64, lo=2048, hi=32768, window=0,
             causal=True, type="bf16", mix=8),
        # one block over the long context
        dict(name="attn_block_262144", op="attention", n_seq=1, rows=8, nq=24, nkv=2, d=256, page=128, lo=262144, hi=262144, window=0,
             causal=False, type="bf16", mix=9),
        # one verified block of 8 rows over the framework's vocabulary
        dict(name="logprobs_block_8", op="logprobs", rows=8, vocab=151936, top=8, type="bf16", mask=0, mix=10),
        # the blocks of 16 sequences in FP32, an odd vocabulary with a grammar's mask
        dict(name="logprobs_step_128", op="logprobs", rows=128, vocab=100003, top=20, type="fp32", mask=1, mix=11),
        # scoring a prompt
        dict(name="logprobs_prompt_2000", op="logprobs", rows=2000, vocab=151936, top=5, type="bf16", mask=0, mix=12),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pages", "write", "attention", "attention", "logprobs"])
    mix = rng.randrange(1 << 20)
    if op == "pages":
        n = _spread(rng, 1, 2000)
        lo = _spread(rng, 1, 4096)
        return dict(op=op, n_seq=n, page=rng.choice([16, 32, 64, 128]), lo=lo, hi=_spread(rng, lo, 8192), rows=rng.randint(1, 8),
                    prefill=rng.randint(0, min(n, 40)), mix=mix)
    if op == "write":
        heads, d = rng.randint(1, 8), rng.choice([64, 128, 256])
        rows = _spread(rng, 1, 30000 * 1024 // (heads * d))
        rows = min(rows, 60000)
        page = rng.choice([16, 32, 64, 128])
        return dict(op=op, rows=rows, heads=heads, d=d, page=page, pages=rows // page + rng.randint(1, 100), type=rng.choice(["bf16", "fp16"]),
                    pad=rng.randint(0, 9), mix=mix)
    if op == "attention":
        d, nkv, rows = rng.choice([64, 128, 256]), rng.randint(1, 8), rng.randint(1, 8)
        group = rng.randint(1, 16 if d < 256 else 12)
        cells = 262144 * 512 // (nkv * d)  # as many as the largest listed case holds
        lo = _spread(rng, 1, min(cells, 100000))
        hi = _spread(rng, lo, min(cells, 200000))
        n = _spread(rng, 1, max(1, min(256, cells // hi)))
        return dict(op=op, n_seq=n, rows=rows, nq=nkv * group, nkv=nkv, d=d, page=rng.choice([16, 32, 64, 128]), lo=lo, hi=hi,
                    window=rng.choice([0, 0, _spread(rng, 16, 8192)]), causal=rng.random() < 0.7, type=rng.choice(["bf16", "fp16"]), mix=mix)
    vocab = _spread(rng, 1000, 200000)
    rows = _spread(rng, 1, max(1, min(4000, 300000000 // vocab)))
    kind = rng.choice(["bf16", "fp16", "fp32"])
    if kind == "fp32":
        rows = max(1, rows // 2)
    return dict(op=op, rows=rows, vocab=vocab, top=rng.choice([0, 1, 5, 20, 32]), type=kind, mask=rng.randint(0, 1), mix=mix)


def _lengths(case):
    """Cells of each sequence after the step, and rows of each in it: they go by the case alone."""
    rng = random.Random(case["mix"])
    lens = [rng.randint(case["lo"], case["hi"]) for _ in range(case["n_seq"])]
    rows = [case["rows"]] * case["n_seq"]
    if case["n_seq"] > 1 and case["rows"] > 1:
        rows = [rng.randint(2, case["rows"]) for _ in lens]
    return [max(n, r) if case["op"] == "attention" else n for n, r in zip(lens, rows)], rows


def _requests(case):
    """Tokens held, rows appended and pages held of each request: some finished (they give their pages back) and some new."""
    rng = random.Random(case["mix"])
    lens, rows = _lengths(case)
    held = []
    for s in range(case["n_seq"]):
        if s < case["prefill"]:
            lens[s], rows[s] = 0, rng.randint(1, case["hi"])
            held.append(0)
            continue
        pages = -(-lens[s] // case["page"])
        if case["n_seq"] > 8 and rng.random() < 0.05:
            lens[s] = rows[s] = 0
        held.append(pages)
    return lens, rows, held


def work(case):
    if case["op"] == "pages":
        lens, rows, held = _requests(case)
        need = [-(-(n + r) // case["page"]) for n, r in zip(lens, rows)]
        moved = sum(abs(n - h) for n, h in zip(need, held))
        total = sum(rows)
        return {"bytes": 20 * case["n_seq"] + 8 * moved + 8 * total, "flops": 4 * total}
    if case["op"] == "write":
        n = case["rows"] * case["heads"] * case["d"]
        # 16-bit K and V in, the cells out, the cells in, FP32 K and V out
        return {"bytes": n * (2 * 2 + 2 * 1.125 + 2 * 4) + 8 * case["rows"], "flops": 12 * n}
    if case["op"] == "attention":
        lens, rows = _lengths(case)
        size = {"bytes": 0, "flops": 0}
        for n, r in zip(lens, rows):
            seen = n if not case["window"] else min(n, case["window"] + (r - 1 if case["causal"] else 0))
            size["bytes"] += seen * case["nkv"] * case["d"] * 1.125 + 2 * 2 * r * case["nq"] * case["d"] + 4 * -(-seen // case["page"])
            size["flops"] += 4 * r * case["nq"] * case["d"] * min(seen, case["window"] or seen)
        return size
    n = case["rows"] * case["vocab"]
    return {"bytes": n * (4 if case["type"] == "fp32" else 2) + case["rows"] * (12 + 8 * case["top"]), "flops": 6 * n}


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
    at = (b.abs() == top).to(torch.int8).argmax(-1, keepdim=True)  # the first of equals
    d = (b.gather(-1, at) * -0.125).half()
    df = d.float()
    q = torch.where(df != 0, torch.round(b / torch.where(df != 0, df, torch.ones_like(df))), torch.zeros_like(b))
    codes = (q.clamp(-8, 7) + 8).to(torch.uint8).flatten(-2)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), d.squeeze(-1)


def _store(cache, layout, slots, k, v):
    """Writes the rows' cells into the cache, rows of slot -1 left out."""
    n_pages, heads, groups, size = cache.shape
    page = groups * GROUP
    codes, scales = layout
    flat = cache.view(-1)
    keep = (slots >= 0).nonzero().squeeze(-1)
    slot = slots[keep].long()
    cell = slot % GROUP
    base = ((slot // page)[:, None] * heads + torch.arange(heads, device=cache.device)) * (groups * size) + ((slot % page // GROUP) * size)[:, None]
    for side, x in enumerate((k, v)):
        q, d = _quantise(x[keep])
        flat[(base[:, :, None] + codes[side][cell][:, None, :]).reshape(-1)] = q.reshape(-1)
        flat[(base[:, :, None] + scales[side][cell][:, None, :]).reshape(-1)] = d.contiguous().view(torch.uint8).reshape(-1)


def _values(codes, scales):
    """Packed codes [..., d / 2] and the bytes of scales [..., d / 16] -> FP32 values [..., d]."""
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float() - 8
    d = scales.contiguous().view(torch.float16).float()
    return (q.unflatten(-1, (-1, 32)) * d[..., None]).flatten(-2)


def _load(cache, layout, slots):
    """Values [rows, heads, d] of the cells of K and V; rows of slot -1 are zero."""
    n_pages, heads, groups, size = cache.shape
    page = groups * GROUP
    codes, scales = layout
    flat = cache.view(-1)
    slot = slots.clamp(min=0).long()
    cell = slot % GROUP
    base = ((slot // page)[:, None] * heads + torch.arange(heads, device=cache.device)) * (groups * size) + ((slot % page // GROUP) * size)[:, None]
    live = (slots >= 0)[:, None, None]
    out = []
    for side in (0, 1):
        x = _values(flat[base[:, :, None] + codes[side][cell][:, None, :]], flat[base[:, :, None] + scales[side][cell][:, None, :]])
        out.append(torch.where(live, x, torch.zeros_like(x)))
    return out


def _normal(shape, gen, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    if case["op"] == "pages":
        lens, rows, held = _requests(case)
        need = [-(-(n + r) // case["page"]) for n, r in zip(lens, rows)]
        width = max(max(need), max(held)) + 1
        used, spare = sum(held), sum(max(0, n - h) for n, h in zip(need, held)) + 7
        n_pages = used + spare
        order = torch.randperm(n_pages, generator=gen, device="cuda").int()
        h = _ints(held).long()
        start = h.cumsum(0) - h
        col = torch.arange(width, device="cuda")
        table = torch.where(col < h[:, None], order[(start[:, None] + col).clamp(max=n_pages - 1)], torch.full((), -1, dtype=torch.int32, device="cuda"))
        head = rng.randrange(n_pages)
        ring = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
        ring[(head + torch.arange(spare, device="cuda")) % n_pages] = order[used:]
        return dict(op="pages", page=case["page"], n_pages=n_pages, row_cap=sum(rows) + 64, lengths=_ints(lens), rows=_ints(rows), held=_ints(held),
                    table=table.contiguous(), ring=ring, ring_state=_ints([head, spare]), held_out=_ints(held), ring_out=_ints([head, spare]))
    if case["op"] == "write":
        n, heads, d = case["rows"], case["heads"], case["d"]
        cache = torch.zeros((case["pages"], heads, case["page"] // GROUP, 18 * d), dtype=torch.uint8, device="cuda")
        # rows of the fused projection's output: K and V of a row lie in one row of it
        both = _normal((n + case["pad"], 2 * heads * d), gen)
        both *= torch.exp(0.5 * _normal((1, 2 * heads * d), gen))  # channels of unequal size
        both = both.to(TYPES[case["type"]])
        slots = torch.randperm(case["pages"] * case["page"], generator=gen, device="cuda")[: n + case["pad"]].int()
        slots[n:] = -1  # rows of the padded batch
        k = both[:, : heads * d].unflatten(-1, (heads, d))
        v = both[:, heads * d:].unflatten(-1, (heads, d))
        return dict(op="write", cache=cache, k=k, v=v, slots=slots, layout=_layout(d, "cuda"))
    if case["op"] == "attention":
        lens, rows = _lengths(case)
        page, d, nkv = case["page"], case["d"], case["nkv"]
        counts = [-(-n // page) for n in lens]
        width, n_pages = max(counts), sum(counts) + 3
        order = torch.randperm(n_pages, generator=gen, device="cuda").int()
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        cache = torch.empty((n_pages, nkv, page // GROUP, 18 * d), dtype=torch.uint8, device="cuda")
        layout = _layout(d, "cuda")
        c = _ints(counts).long()
        col = torch.arange(width, device="cuda")
        start = c.cumsum(0) - c
        table = torch.where(col < c[:, None], order[(start[:, None] + col).clamp(max=n_pages - 1)], torch.full((), -1, dtype=torch.int32, device="cuda"))
        gain = torch.exp(0.3 * _normal((nkv, d), gen))
        step = max(1, (1 << 24) // (nkv * page * d))
        for at in range(0, n_pages, step):  # every cell holds a quantised row, those of no sequence too
            m = min(step, n_pages - at)
            slots = torch.arange(at * page, (at + m) * page, device="cuda")
            _store(cache, layout, slots, _normal((m * page, nkv, d), gen) * gain, _normal((m * page, nkv, d), gen))
        total = sum(rows)
        q = (2.0 * _normal((total, case["nq"], d), gen)).to(TYPES[case["type"]])
        offsets = [0]
        for r in rows:
            offsets.append(offsets[-1] + r)
        return dict(op="attention", cache=cache, layout=layout, q=q, table=table.contiguous(), kv_len=_ints(lens), offsets=_ints(offsets), rows=case["rows"],
                    causal=case["causal"], window=case["window"], longest=max(lens))
    n, vocab = case["rows"], case["vocab"]
    x = torch.empty((n, vocab), dtype=TYPES[case["type"]], device="cuda")
    step = max(1, (1 << 27) // vocab)
    for at in range(0, n, step):  # logits with a heavy head: a few tokens carry most of the weight
        part = _normal((min(step, n - at), vocab), gen)
        x[at:at + step] = (2.0 * part + 0.25 * part ** 3).to(x.dtype)
    if case["mask"]:  # a grammar leaves about a third of the tokens
        x.masked_fill_(torch.rand((1, vocab), generator=gen, device="cuda") < 0.66, -math.inf)
        x[0].fill_(-math.inf)
        x[0, rng.randrange(vocab)] = 1.5
    tokens = torch.randint(0, vocab, (n,), generator=gen, device="cuda", dtype=torch.int64)
    best = torch.rand((n,), generator=gen, device="cuda") < 0.7
    tokens = torch.where(best | (case["mask"] == 1), x.float().argmax(-1), tokens).int()
    return dict(op="logprobs", x=x, tokens=tokens, top=case["top"])


# ------------------------------------------------------------------ the plain forms
def _plain_pages(s):
    n_pages, page, cap = s["n_pages"], s["page"], s["row_cap"]
    length, new, held = s["lengths"].long(), s["rows"].long(), s["held"].long()
    head, count = s["ring_state"].long().unbind()
    width = s["table"].shape[1]
    zero = torch.zeros_like(length)
    valid = (length >= 0) & (new >= 0)
    need = (length + new + page - 1).div(page, rounding_mode="floor")
    fits = valid & (need <= width)
    take = torch.where(fits, (need - held).clamp(min=0), zero)
    give = torch.where(fits, (held - need).clamp(min=0), zero)
    upto = take.cumsum(0)
    got = fits & ((take == 0) | (upto <= count))
    taken = torch.where(got, take, zero)
    first = upto - take
    gave = give.cumsum(0)
    held_out = torch.where(got, need, held)
    col = torch.arange(width, device=held.device)
    fresh = (col >= held[:, None]) & (col < (held + taken)[:, None])
    page_at = s["ring"][(head + first[:, None] + col - held[:, None]) % n_pages]
    table = torch.where(fresh, page_at, s["table"])
    # the pages given back, at the ring's tail
    place = (torch.arange(n_pages, device=held.device) - head - count) % n_pages
    who = torch.searchsorted(gave, place, right=True).clamp(max=held.numel() - 1)
    back = s["table"][who, (need[who] + place - (gave - give)[who]).clamp(0, width - 1)]
    ring = torch.where(place < gave[-1], back, s["ring"])
    many = torch.where(valid, new, zero)
    ends = many.cumsum(0)
    row = torch.arange(cap, device=held.device)
    of = torch.searchsorted(ends, row, right=True).clamp(max=held.numel() - 1)
    at = length[of] + row - (ends - many)[of]
    live = row < ends[-1]
    slot = table[of, at.div(page, rounding_mode="floor").clamp(0, width - 1)].long() * page + at % page
    none = torch.full_like(slot, -1)
    slots = torch.where(live & got[of], slot, none).int()
    positions = torch.where(live, at, none).int()
    s["table"].copy_(table)
    s["ring"].copy_(ring)
    offsets = torch.cat([zero[:1], ends]).int()
    moved = taken.sum()
    state = torch.stack([(head + moved) % n_pages, count - moved + gave[-1]]).int()
    return dict(held=held_out.int(), table=s["table"], ring=s["ring"], ring_state=state, offsets=offsets, slots=slots, positions=positions)


def _plain_write(s):
    _store(s["cache"], s["layout"], s["slots"], s["k"], s["v"])
    k, v = _load(s["cache"], s["layout"], s["slots"])
    return dict(k=k, v=v)


def _plain_attention(s):
    cache, q = s["cache"], s["q"]
    n_pages, nkv, groups, size = cache.shape
    page, d = groups * GROUP, size // 18
    n_seq, nq = s["kv_len"].numel(), q.shape[1]
    codes, scales = s["layout"]
    kv_len, offsets, most = s["kv_len"].long(), s["offsets"].long(), s["rows"]
    # every sequence's cells, padded to the longest: [n_seq, nkv, cells, d]
    cells = cache[s["table"].clamp(min=0).long()]  # [n_seq, pages, nkv, groups, size]
    k, v = (_values(cells[..., codes[i]], cells[..., scales[i]]).permute(0, 2, 1, 3, 4, 5).reshape(n_seq, nkv, -1, d) for i in (0, 1))
    # the rows, padded to `most` of each sequence: [n_seq, nkv, group * most, d]
    i = torch.arange(most, device=q.device)
    count = offsets[1:] - offsets[:-1]
    pick = (offsets[:-1, None] + i).clamp(max=q.shape[0] - 1)
    rows = q[pick].float().unflatten(2, (nkv, nq // nkv)).permute(0, 2, 3, 1, 4).reshape(n_seq, nkv, -1, d)
    scores = rows @ k.transpose(-1, -2) * d ** -0.5
    at = torch.arange(scores.shape[-1], device=q.device)
    last = kv_len[:, None] - count[:, None] + i if s["causal"] else (kv_len - 1)[:, None] + 0 * i
    sees = at <= last[:, :, None]
    if s["window"]:
        sees = sees & (at > (last - s["window"])[:, :, None])
    scores = scores.view(n_seq, nkv, nq // nkv, most, -1).masked_fill(~sees[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).view(n_seq, nkv, nq // nkv, most, d) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.permute(0, 3, 1, 2, 4).reshape(n_seq, most, nq, d)
    return o[i < count[:, None]].to(q.dtype)


def _plain_logprobs(s):
    x, top = s["x"].float(), s["top"]
    m = x.amax(-1, keepdim=True)
    y = x - m
    e = torch.exp(y)
    total = e.sum(-1)
    lse = torch.log(total)
    entropy = lse - torch.where(e > 0, e * y, torch.zeros_like(y)).sum(-1) / total
    logp = y.gather(-1, s["tokens"].long()[:, None]).squeeze(-1) - lse
    out = dict(logp=logp, entropy=entropy)
    if top:
        del e, y
        # one whole number for a value and its place, so that ties go to the lowest id
        bits = (x + 0.0).view(torch.int32).long()
        key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits) * (1 << 32) + (0xFFFFFFFF - torch.arange(x.shape[-1], device=x.device))
        best = 0xFFFFFFFF - (torch.topk(key, top, -1).values & 0xFFFFFFFF)
        value = x.gather(-1, best)
        out["top_ids"] = torch.where(value > -math.inf, best, torch.full_like(best, -1)).int()
        out["top_logp"] = value - m - lse[:, None]
    return out


# ------------------------------------------------------------------ one pass
def run(state):
    s = state
    if own:
        from dflash_block_drafter_gb300 import runtime as R
        if s["op"] == "pages":
            offsets, slots, positions = R.page_tables(s["lengths"], s["rows"], s["held"], s["table"], s["ring"], s["ring_state"], s["page"], s["row_cap"],
                                                      held_out=s["held_out"], ring_state_out=s["ring_out"])
            return dict(held=s["held_out"], table=s["table"], ring=s["ring"], ring_state=s["ring_out"], offsets=offsets, slots=slots, positions=positions)
        if s["op"] == "write":
            R.kv4_write(s["cache"], s["k"], s["v"], s["slots"])
            k, v = R.kv4_read(s["cache"], s["slots"])
            return dict(k=k, v=v)
        if s["op"] == "attention":
            return R.kv4_attention(s["cache"], s["q"], s["table"], s["kv_len"], s["offsets"], s["rows"], causal=s["causal"], window=s["window"])
        logp, entropy, ids, top = R.token_logprobs(s["x"], s["tokens"], top_k=s["top"])
        return dict(logp=logp, entropy=entropy, top_ids=ids, top_logp=top) if s["top"] else dict(logp=logp, entropy=entropy)
    if s["op"] == "pages":
        return _plain_pages(s)
    if s["op"] == "write":
        return _plain_write(s)
    if s["op"] == "attention":
        return _plain_attention(s)
    return _plain_logprobs(s)


# ------------------------------------------------------------------ from the definitions, in 64 bits
def _cells_64(cache, slots, d):
    """[rows, heads, d] K and V of the cells, byte by byte from the format."""
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


def exact(case, seed):
    if case["op"] == "pages":
        return None  # whole numbers: they are equal or wrong
    s = prepare(case, seed)
    if case["op"] == "write":
        out = {}
        for name in ("k", "v"):
            x = s[name].double().unflatten(-1, (-1, 32))
            size = x.abs()
            first = (size >= size.max(-1, keepdim=True).values).double()
            first = first * (first.cumsum(-1) == 1)
            d = ((x * first).sum(-1, keepdim=True) / -8).half().double()
            ratio = x / d
            q = torch.floor(ratio + 0.5)
            q = q - ((q - ratio == 0.5) & (q % 2 != 0)).double()  # halves go to the even neighbour
            x = torch.nan_to_num(q.clamp(-8, 7) * d).flatten(-2)
            out[name] = x * (s["slots"] >= 0)[:, None, None]
        return out
    if case["op"] == "attention":
        lens, rows = _lengths(case)
        d, nkv, page = case["d"], case["nkv"], case["page"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        r0 = 0
        for i, (n, r) in enumerate(zip(lens, rows)):
            slots = (s["table"][i, : -(-n // page)].long()[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:n]
            # a group of cells lies behind one page's group of another head: the places of (page, group) in order
            k, v = _cells_64(s["cache"], slots, d)
            for h in range(nkv):
                group = case["nq"] // nkv
                q = s["q"][r0:r0 + r, h * group:(h + 1) * group].double().transpose(0, 1)  # [group, r, d]
                x = torch.einsum("grd,nd->grn", q, k[:, h]) / math.sqrt(d)
                at = torch.arange(n, device="cuda")
                last = torch.arange(n - r, n, device="cuda") if case["causal"] else torch.full((r,), n - 1, device="cuda")
                hidden = at[None, :] > last[:, None]
                if case["window"]:
                    hidden |= at[None, :] <= last[:, None] - case["window"]
                x[:, hidden] = -math.inf
                w = torch.exp(x - x.max(-1, keepdim=True).values)
                out[r0:r0 + r, h * group:(h + 1) * group] = torch.einsum("grn,nd->rgd", w / w.sum(-1, keepdim=True), v[:, h])
            r0 += r
        return out
    out = dict(logp=[], entropy=[], top_ids=None, top_logp=[])
    step = max(1, (1 << 26) // case["vocab"])
    for at in range(0, case["rows"], step):
        x = s["x"][at:at + step].double()
        lse = torch.logsumexp(x, -1)
        p = torch.exp(x - lse[:, None])
        out["logp"].append(x[torch.arange(x.shape[0], device="cuda"), s["tokens"][at:at + step].long()] - lse)
        out["entropy"].append(-(p * torch.nan_to_num(torch.log(p), neginf=0.0)).sum(-1))
        if case["top"]:
            out["top_logp"].append(x.sort(-1, descending=True).values[:, : case["top"]] - lse[:, None])
    done = dict(logp=torch.cat(out["logp"]), entropy=torch.cat(out["entropy"]))
    if case["top"]:
        done.update(top_ids=None, top_logp=torch.cat(out["top_logp"]))
    return done
