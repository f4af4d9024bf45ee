"""The packed key/value cache's operators as they are measured: 4-bit writing and reading back, and attention over the packed pages.

A cache keeps, for every token and key/value head, D key and D value numbers as 4-bit codes in groups of 32 with an fp16
scale s and an fp16 base b each: x = b + s (c - 8).  Tokens lie in pages of P tokens; a page holds, per head, P / 16 chunks of
16 tokens, and a chunk is [key codes 8 D bytes][key (s, b) pairs 2 D][value codes 8 D][value pairs 2 D].  Inside a row of D / 8
code words (word w = numbers 8 w .. 8 w + 7, the lowest in the lowest nibble) and of D / 32 pairs the order is the one the
kernels read in:
  keys:   row t = token t, word 4 g + c at place c D / 32 + g, pairs in the order of their groups;
  values: row t / 2 + 8 (t % 2) = token t, word r + 8 j at place r D / 64 + j, pair g at place (g % 2) D / 64 + g / 2.

A step (`cu_new`, `start`, `page_table`) names, for each sequence, the new tokens' rows and their first position; new token
i of a sequence stands at position start + i, and its query sees the positions up to its own (the last `window` of them).
"""
import math
import random

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
CLAMP = 65000.0  # a stored number's largest size: the largest dequantised number stays inside fp16


# --------------------------------------------------------------------- cases -----
def listed():
    base = {"op": "attention", "type": "bf16", "seqs": 1, "ctx": 1024, "ragged": False, "new": 1, "heads": 8, "group": 4,
            "dim": 128, "page": 64, "window": 0, "far": False}

    def case(name, **more):
        return {**base, **more, "name": name}

    return [
        # the smallest call of a generating loop: one sequence's new token enters the cache
        case("write_1", op="write", type="fp16", ctx=1000),
        # a served batch's new tokens, each sequence at its own length
        case("write_64", op="write", seqs=64, ctx=8000, ragged=True),
        # prompts of several requests enter the cache at once
        case("write_prompts", op="write", seqs=3, ctx=500, new=5000, ragged=True),
        # one short context read back, small heads, small pages
        case("read_777", op="read", type="fp16", ctx=0, new=777, heads=2, dim=64, page=16),
        # contexts read back whole, as before a move to another place or another precision
        case("read_contexts", op="read", seqs=16, ctx=0, new=16000, ragged=True),
        # one conversation, one token: latency
        case("attend_777", type="fp16", ctx=776),
        # one long document, one token: the split over the context
        case("attend_32k", ctx=32767),
        # a served batch, one token each, lengths as they come
        case("attend_batch", seqs=64, ctx=8191, ragged=True),
        # a few very long contexts in a pool beyond 4 GiB
        case("attend_far", type="fp16", seqs=4, ctx=131071, far=True),
        # one query head per key head, small heads and pages
        case("attend_mha", type="fp16", seqs=16, ctx=2047, heads=32, group=1, dim=64, page=16, ragged=True),
        # four drafted tokens a sequence are verified under a sliding window
        case("attend_draft", seqs=8, ctx=20000, new=4, heads=4, group=8, window=4096, page=32, ragged=True),
        # a prompt's next pieces attend to what is cached and to themselves
        case("attend_chunk", seqs=2, ctx=4096, new=512, ragged=True),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    c = {"op": rng.choice(["write", "read", "attention", "attention", "attention"]), "type": rng.choice(["fp16", "bf16"]),
         "ragged": rng.random() < 0.7, "dim": rng.choice([64, 128, 128, 256]), "page": rng.choice([16, 32, 64, 128]),
         "heads": rng.choice([1, 2, 4, 8, 8, 16]), "group": rng.choice([1, 2, 3, 4, 5, 8, 12]), "window": 0, "far": False}
    c["seqs"] = _spread(rng, 1, 100)
    if c["op"] == "attention":
        c["new"] = rng.choice([1, 1, 1, 2, 4, _spread(rng, 3, 600)])
        c["ctx"] = _spread(rng, 1, 100000)
        c["window"] = rng.choice([0, 0, 0, _spread(rng, 1, 8192)])
    else:
        c["new"] = _spread(rng, 1, 20000) if c["op"] == "read" else rng.choice([1, _spread(rng, 1, 6000)])
        c["ctx"] = 0 if c["op"] == "read" else rng.randint(0, 4000)
    # no more than the largest listed case of the kind: packed bytes, dense numbers, scores
    for _ in range(64):
        tokens = c["seqs"] * (c["ctx"] + c["new"])
        scores = c["seqs"] * c["new"] * c["heads"] * c["group"] * (c["ctx"] + c["new"])
        if tokens * c["heads"] * c["dim"] <= 4e8 and c["seqs"] * c["new"] * c["heads"] * c["group"] * c["dim"] <= 5e7 and (
                c["op"] != "attention" or scores <= 1.4e8):
            break
        c["seqs"] = max(1, c["seqs"] // 2)
        if c["seqs"] == 1:
            c["ctx"], c["new"] = c["ctx"] // 2, max(1, c["new"] // 2)
    return c


def _lengths(case):
    """(positions before the step, new tokens) of every sequence: fixed by the case alone."""
    r = random.Random("%(seqs)d %(ctx)d %(new)d %(heads)d" % case)
    spans = []
    for _ in range(case["seqs"]):
        start, new = case["ctx"], case["new"]
        if case["ragged"]:
            start, new = r.randint(start // 4, start), r.randint((new + 1) // 2, new)
        spans.append((start, new))
    return spans


def work(case):
    spans, d, hk = _lengths(case), case["dim"], case["heads"]
    packed = hk * d * 2 * 5 // 8  # 4-bit codes and 32 bits a group of 32, keys and values of a token
    new = sum(n for _, n in spans)
    if case["op"] == "write":
        return {"bytes": new * (hk * d * 2 * 2 + packed) + new * (packed + hk * d * 2 * 2), "flops": new * hk * d * 2 * 8}
    if case["op"] == "read":
        return {"bytes": new * (packed + hk * d * 2 * 2), "flops": new * hk * d * 2 * 2}
    hq, w = hk * case["group"], case["window"]
    seen = sum(min(s + n, n - 1 + w) if w else s + n for s, n in spans)  # tokens that some query of the sequence sees
    pairs = sum(min(s + i + 1, w) if w else s + i + 1 for s, n in spans for i in range(n))
    return {"bytes": seen * packed + new * hq * (2 * d * 2 + 4), "flops": 4 * pairs * hq * d}


# -------------------------------------------------------------------- inputs -----
def prepare(case, seed):
    dev, dt = "cuda", TYPES[case["type"]]
    g = torch.Generator(dev).manual_seed(seed)
    hk, d, p, spans = case["heads"], case["dim"], case["page"], _lengths(case)
    need = [-(-(s + n) // p) for s, n in spans]
    page_bytes = hk * (p // 16) * 20 * d
    n_pages = sum(need) + 1
    if case["far"]:
        n_pages = max(n_pages, (9 << 29) // page_bytes)  # 4.5 GiB
    # page 0 is nobody's; the others are scattered over the pool
    order = 1 + torch.randperm(n_pages - 1, device=dev, generator=g)[:sum(need)]
    table = torch.zeros(len(spans), max(need), dtype=torch.int32, device=dev)
    rows = torch.repeat_interleave(torch.arange(len(spans), device=dev), torch.tensor(need, device=dev))
    first = torch.tensor([0] + need, device=dev).cumsum(0)[:-1]
    table[rows, torch.arange(sum(need), device=dev) - first[rows]] = order.to(torch.int32)
    meta = -(-n_pages * page_bytes // 256) * 256
    store = torch.zeros(meta + 256, dtype=torch.uint8, device=dev)
    pool = store[:n_pages * page_bytes].view(n_pages, hk, p // 16, 20 * d)
    for at in range(0, len(order), 2048):  # random codes, scales and bases of numbers near N(0, 1)
        part = order[at:at + 2048]
        x = torch.randint(0, 256, (len(part), hk, p // 16, 20 * d), dtype=torch.uint8, device=dev, generator=g)
        shape = (len(part), hk, p // 16, d)
        for lo in (8 * d, 18 * d):
            pair = torch.empty(shape, dtype=torch.float16, device=dev)
            pair[..., 0::2] = torch.rand((*shape[:3], d // 2), device=dev, generator=g) * 0.2 + 0.18
            pair[..., 1::2] = torch.randn((*shape[:3], d // 2), device=dev, generator=g) * 0.2
            x[..., lo:lo + 2 * d] = pair.view(torch.uint8)
        pool[part] = x
    total = sum(n for _, n in spans)
    state = {
        "case": case, "store": store, "pool": pool, "table": table, "spans": spans, "total": total,
        "start": torch.tensor([s for s, _ in spans], dtype=torch.int32, device=dev),
        "cu": torch.tensor([0] + [n for _, n in spans], device=dev).cumsum(0).to(torch.int32),
        "scale": d ** -0.5,
    }
    # the three projections of a step's tokens lie side by side in one row, as a joined product leaves them
    hq = hk * case["group"]
    if case["op"] == "attention":
        state["q"] = torch.randn(total, (hq + 2 * hk) * d, device=dev, generator=g).mul_(1.5).to(dt)[:, :hq * d].view(total, hq, d)
    elif case["op"] == "write":
        kv = torch.randn(total, 2 * hk * d, device=dev, generator=g)
        kv[:, 5::97] *= 8.0  # a few channels are large, as in trained models
        kv = kv.to(dt)
        state["k"], state["v"] = kv[:, :hk * d].view(total, hk, d), kv[:, hk * d:].view(total, hk, d)
    if own:
        import residual_block_decomp_b200 as bs

        state["cache"] = bs.bs_cache_create(hk, d, p, n_pages, store)
        state["step"] = bs.CacheStep(state["start"], table, total, max(n for _, n in spans), state["cu"])
        if case["op"] == "attention":
            need = bs.bs_cache_attention_workspace_bytes(state["cache"], state["step"], hq)
            state["ws"] = torch.zeros(need, dtype=torch.uint8, device=dev)
    return state


# ---------------------------------------------------------------- plain forms -----
def _places(d, dev):
    """Where the words and pairs of a row lie: (key words, value words, value pairs), by natural number."""
    w, g = torch.arange(d // 8, device=dev), torch.arange(d // 32, device=dev)
    return w % 4 * (d // 32) + w // 4, w % 8 * (d // 64) + w // 8, g % 2 * (d // 64) + g // 2


def _rows(dev):
    t = torch.arange(16, device=dev)
    return t // 2 + 8 * (t % 2)  # a token's row among a chunk's values


def _numbers(words, pairs):
    """Codes (..., D / 8 words) and (s, b) pairs (..., D / 32, 2) as float32 numbers (..., D)."""
    codes = (words.unsqueeze(-1) >> torch.arange(0, 32, 4, device=words.device, dtype=torch.int32)) & 15
    x = codes.flatten(-2).unflatten(-1, (-1, 32)).float() - 8.0
    return (x * pairs[..., :1].float() + pairs[..., 1:].float()).flatten(-2)


def _unpack(chunks, d):
    """Chunks (..., 20 D bytes) as keys and values (..., 16, D) in float32."""
    kw, vw, vp = _places(d, chunks.device)
    rows = _rows(chunks.device)
    part = [x.contiguous() for x in chunks.split([8 * d, 2 * d, 8 * d, 2 * d], -1)]
    k = _numbers(part[0].view(torch.int32).unflatten(-1, (16, -1))[..., kw],
                 part[1].view(torch.float16).unflatten(-1, (16, -1, 2)))
    v = _numbers(part[2].view(torch.int32).unflatten(-1, (16, -1))[..., rows, :][..., vw],
                 part[3].view(torch.float16).unflatten(-1, (16, -1, 2))[..., rows, :, :][..., vp, :])
    return k, v


def _quantise(x):
    """Numbers (..., D) as words (..., D / 8) and pairs (..., D / 32, 2)."""
    x = x.float().nan_to_num(0.0, CLAMP, -CLAMP).clamp(-CLAMP, CLAMP).unflatten(-1, (-1, 32))
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s = (high - low) / 15.0
    b = (low + 8.0 * s).half()
    s = s.half()
    c = torch.where(s > 0, ((x - b.float()) / s.float() + 8.0).round().clamp(0, 15), 8.0)
    shift = torch.arange(0, 32, 4, device=x.device)
    words = (c.long().flatten(-2).unflatten(-1, (-1, 8)) << shift).sum(-1).to(torch.int32)
    return words, torch.cat([s, b], -1)


def _rows_of(state):
    """(sequence, position, page) of every new token."""
    dev = state["start"].device
    cu = state["cu"].long()
    row = torch.arange(state["total"], device=dev)
    seq = torch.searchsorted(cu, row, right=True) - 1
    pos = state["start"].long()[seq] + row - cu[seq]
    return seq, pos, state["table"].long()[seq, pos // state["case"]["page"]]


def _write(state):
    d, p, pool = state["case"]["dim"], state["case"]["page"], state["pool"]
    _, pos, page = _rows_of(state)
    kw, vw, vp = _places(d, pool.device)
    at = pos % 16
    head = torch.arange(pool.shape[1], device=pool.device)
    for x, lo, wi, pi, row in ((state["k"], 0, kw, None, at), (state["v"], 10 * d, vw, vp, at // 2 + 8 * (at % 2))):
        words, pairs = _quantise(x)
        placed, both = torch.empty_like(words), torch.empty_like(pairs)
        placed[..., wi] = words
        both[..., slice(None) if pi is None else pi, :] = pairs
        for data, start, size in ((placed.view(torch.uint8), lo, d // 2), (both.flatten(-2).view(torch.uint8), lo + 8 * d, d // 8)):
            byte = start + row[:, None] * size + torch.arange(size, device=pool.device)
            pool[page[:, None, None], head[None, :, None], (pos % p // 16)[:, None, None], byte[:, None, :]] = data


def _read(state):
    case, pool = state["case"], state["pool"]
    _, pos, page = _rows_of(state)
    kw, vw, vp = _places(case["dim"], pool.device)
    d, at = case["dim"], pos % 16
    chunk = pos % case["page"] // 16
    head = torch.arange(pool.shape[1], device=pool.device)

    def bytes_of(lo, row, size):
        byte = lo + row[:, None] * size + torch.arange(size, device=pool.device)
        return pool[page[:, None, None], head[None, :, None], chunk[:, None, None], byte[:, None, :]]

    rv = at // 2 + 8 * (at % 2)
    k = _numbers(bytes_of(0, at, d // 2).view(torch.int32)[..., kw], bytes_of(8 * d, at, d // 8).view(torch.float16).unflatten(-1, (-1, 2)))
    v = _numbers(bytes_of(10 * d, rv, d // 2).view(torch.int32)[..., vw],
                 bytes_of(18 * d, rv, d // 8).view(torch.float16).unflatten(-1, (-1, 2))[..., vp, :])
    return k.to(TYPES[case["type"]]), v.to(TYPES[case["type"]])


def _attend(state):
    case, pool = state["case"], state["pool"]
    hk, gr, d, p, w = case["heads"], case["group"], case["dim"], case["page"], case["window"]
    dev = pool.device
    seqs, new = len(state["spans"]), max(n for _, n in state["spans"])
    # the step's queries, one padded block a sequence
    seq, pos, _ = _rows_of(state)
    col = torch.arange(state["total"], device=dev) - state["cu"].long()[seq]
    q = torch.zeros(seqs, new, hk, gr, d, device=dev)
    q[seq, col] = state["q"].float().view(-1, hk, gr, d)
    at = torch.full((seqs, new), -1, device=dev)
    at[seq, col] = pos
    k, v = _unpack(pool[state["table"].long()], d)  # seqs, pages, heads, chunks, 16, d
    k, v = (x.permute(0, 2, 1, 3, 4, 5).reshape(seqs, hk, -1, d) for x in (k, v))
    token = torch.arange(k.shape[2], device=dev)
    see = token <= at[..., None]
    if w:
        see = see & (token > at[..., None] - w)
    see = see[:, None, :, None, :]  # seqs, 1, new, 1, tokens
    s = (q.permute(0, 2, 1, 3, 4).reshape(seqs, hk, new * gr, d) @ k.transpose(-1, -2)).view(seqs, hk, new, gr, -1) * state["scale"]
    s = s.masked_fill(~see, -math.inf)
    top = s.amax(-1, keepdim=True).clamp_min(-3e38)
    e = torch.exp(s - top)
    z = e.sum(-1, keepdim=True)
    v = v.masked_fill(~see.any(2).any(2)[..., None], 0.0)
    o = (e.view(seqs, hk, new * gr, -1) @ v).view(seqs, hk, new, gr, d) / z
    lse = (top + torch.log(z)).squeeze(-1)
    o, lse = (x.transpose(1, 2)[seq, col].flatten(1, 2) for x in (o, lse))
    return o.to(TYPES[case["type"]]), lse


def run(state):
    op = state["case"]["op"]
    if not own:
        if op == "attention":
            return _attend(state)
        if op == "write":
            _write(state)
        return _read(state)
    import residual_block_decomp_b200 as bs

    if op == "attention":
        q = state["q"]
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
        bs.bs_cache_attention(state["cache"], state["step"], q, out, state["ws"], scale=state["scale"],
                              window=state["case"]["window"], lse=lse)
        return out, lse
    if op == "write":
        bs.bs_cache_append(state["cache"], state["step"], state["k"], state["v"])
    shape = (state["total"], state["case"]["heads"], state["case"]["dim"])
    k = torch.empty(shape, dtype=TYPES[state["case"]["type"]], device=state["store"].device)
    v = torch.empty_like(k)
    bs.bs_cache_read(state["cache"], state["step"], k, v)
    return k, v


# --------------------------------------------------------------- in 64 bits -----
def exact(case, seed):
    """From the definition, one sequence and head at a time: the number of (token, dim) by its address in the pool."""
    state = prepare(case, seed)
    store, table, hk, d, p = state["store"], state["table"].long(), case["heads"], case["dim"], case["page"]
    dev, f8 = store.device, torch.float64
    dim = torch.arange(d, device=dev)

    def dense(b, h, first, last, value):
        pos = torch.arange(first, last, device=dev)
        base = ((table[b, pos // p] * hk + h) * (p // 16) + pos % p // 16) * (20 * d) + (10 * d if value else 0)
        t, w, g = pos % 16, dim // 8, dim // 32
        row = t // 2 + t % 2 * 8 if value else t
        word = w % 8 * (d // 64) + w // 8 if value else w % 4 * (d // 32) + w // 4
        pair = g % 2 * (d // 64) + g // 2 if value else g
        code = store[(base + row * (d // 2))[:, None] + word * 4 + dim % 8 // 2].long() >> (dim % 2 * 4) & 15
        both = (base + 8 * d + row * (d // 8))[:, None] + pair * 4

        def half(at):
            return (store[at].to(torch.int16) | store[at + 1].to(torch.int16) << 8).view(torch.float16).to(f8)

        return half(both + 2) + half(both) * (code - 8).to(f8)

    if case["op"] == "write":
        outs = []
        for x in (state["k"], state["v"]):
            x = x.to(f8).nan_to_num(0.0, CLAMP, -CLAMP).clamp(-CLAMP, CLAMP).reshape(-1, 32)
            low, high = x.min(1, keepdim=True).values, x.max(1, keepdim=True).values
            s = (high - low) / 15
            b, s = (low + 8 * s).to(torch.float16).to(f8), s.to(torch.float16).to(f8)
            c = torch.where(s > 0, torch.round((x - b) / s + 8).clamp(0, 15), torch.full_like(x, 8.0))
            outs.append((b + s * (c - 8)).view(-1, hk, d))
        return tuple(outs)
    if case["op"] == "read":
        if state["total"] * hk * d > 4e8:
            return None
        outs = [torch.empty(state["total"], hk, d, dtype=f8, device=dev) for _ in range(2)]
        for i, out in enumerate(outs):
            at = 0
            for b, (s, n) in enumerate(state["spans"]):
                for h in range(hk):
                    out[at:at + n, h] = dense(b, h, s, s + n, i == 1)
                at += n
        return tuple(outs)
    gr, q = case["group"], state["q"].to(f8)
    out = torch.empty(q.shape, dtype=f8, device=dev)
    lse = torch.empty(q.shape[:2], dtype=f8, device=dev)
    at = 0
    for b, (s, n) in enumerate(state["spans"]):
        first = max(0, s + 1 - case["window"]) if case["window"] else 0
        token = torch.arange(first, s + n, device=dev)
        place = torch.arange(s, s + n, device=dev)[:, None]
        hidden = token > place
        if case["window"]:
            hidden |= token <= place - case["window"]
        for h in range(hk):
            k, v = (dense(b, h, first, s + n, i == 1) for i in range(2))
            x = torch.einsum("ngd,td->gnt", q[at:at + n, h * gr:(h + 1) * gr], k) / math.sqrt(d)
            x = x.masked_fill(hidden, -math.inf)
            lse[at:at + n, h * gr:(h + 1) * gr] = torch.logsumexp(x, -1).T
            out[at:at + n, h * gr:(h + 1) * gr] = torch.einsum("gnt,td->ngd", torch.softmax(x, -1), v)
        at += n
    return out, lse
