"""Cases for the operators of a chunked-prefill step: the step's plan, cache append with query and key norms, and
attention of the new tokens over the paged cache, with or without a sliding window.

Each operator has a plain form in elementary torch operations (``own`` False) and the call a user makes of the package
(``own`` True).  Sizes follow the package's own decode workloads: 16-token pages, head dimension 128, 1 to 8 query
heads per KV head, batches up to a few hundred requests, contexts up to 32768 tokens.
"""
import math

import numpy as np
import torch

own = False

PAGE, DIM = 16, 128
DEV = "cuda"


# ------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------
def _chunk(name, fmt, decodes, chunks, new, ctx, hq, hkv, window=0, sinks=0, out="bf16"):
    """`decodes` sequences with one new token each and `chunks` with up to `new`, behind up to `ctx` earlier ones."""
    return {"op": "chunk", "name": name, "format": fmt, "decodes": decodes, "chunks": chunks, "new": new, "ctx": ctx,
            "hq": hq, "hkv": hkv, "window": window, "sinks": sinks, "out": out}


def _append(name, tokens, hq, hkv, rot=128, interleaved=False, max_pos=8192, pad=0.0, per_head=False, base=1000000.0):
    return {"op": "append", "name": name, "tokens": tokens, "hq": hq, "hkv": hkv, "rot": rot,
            "interleaved": interleaved, "max_pos": max_pos, "pad": pad, "per_head": per_head, "base": base}


def _plan(name, requests, new, ctx, slots, width, pad=0):
    return {"op": "plan", "name": name, "requests": requests, "new": new, "ctx": ctx, "slots": slots, "width": width,
            "pad": pad}


def listed():
    return [
        # one prompt from its first token on: causal, nothing cached before it
        _chunk("chunk-prompt", "raw", 0, 1, 4096, 0, 32, 8),
        # the last chunk of a long prompt: bound by the matrix products
        _chunk("chunk-long", "raw", 0, 1, 2039, 30710, 32, 8),
        # a serving step that mixes decoding sequences and ragged prompt chunks, 5 query heads per KV head
        _chunk("chunk-mixed", "raw", 31, 3, 700, 7490, 40, 8),
        # a chunk behind a document in 12-bit pages, 8 query heads per KV head
        _chunk("chunk-12bit", "12bit", 0, 1, 1024, 15360, 64, 8),
        # five draft tokens a sequence checked at once, 12-bit pages, float32 outputs
        _chunk("verify-12bit", "12bit", 0, 16, 5, 8186, 32, 8, out="float32"),
        # a prompt through a sliding-window layer whose first tokens stay visible
        _chunk("window-prompt", "raw", 0, 1, 8191, 0, 32, 8, window=1024, sinks=4),
        # decoding through a sliding-window layer: pages between first tokens and window have been given back
        _chunk("window-decode", "raw", 64, 0, 1, 32767, 64, 8, window=4096, sinks=64),
        # the same over 12-bit pages, few sequences: latency counts
        _chunk("window-decode-12bit", "12bit", 4, 0, 1, 12000, 16, 4, window=2048, sinks=16),
        # a decode batch of 64 sequences with normed queries and keys
        _append("norm-decode", 64, 32, 8, max_pos=131072),
        # ragged prompts packed into one batch, some padding tokens, norm weights for each head
        _append("norm-prefill", 16381, 32, 8, max_pos=32768, pad=0.03, per_head=True),
        # a decode step of 256 requests, one new token each
        _plan("plan-decode", 256, 1, 8000, 300, 512),
        # a step of ragged prompts, the batch padded to a fixed size
        _plan("plan-prompts", 61, 1021, 3000, 128, 2048, pad=500),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    hkv = rng.choice((1, 2, 4, 8))
    hq = hkv * rng.randint(1, 8)
    kind = rng.random()
    if kind < 0.2:
        c = _append("", _log(rng, 1, 12000), hq, hkv, rot=rng.choice((16, 32, 64, 96, 128, 128)),
                    interleaved=rng.random() < 0.4, max_pos=_log(rng, 64, 1 << 20), pad=rng.choice((0.0, 0.05)),
                    per_head=rng.random() < 0.3, base=rng.choice((10000.0, 1000000.0)))
    elif kind < 0.35:
        n = _log(rng, 1, 400)
        c = _plan("", n, _log(rng, 1, 16000 // n), _log(rng, 1, 8000), n + rng.randint(0, 40), rng.choice((600, 1031, 2048)),
                  pad=rng.randint(0, 300))
    else:
        chunks = rng.choice((0, 1, 1, 2, 5))
        c = _chunk("", rng.choice(("raw", "12bit")), rng.choice((0, 3, 17)) if chunks else _log(rng, 1, 64), chunks,
                   _log(rng, 1, 2000 // max(chunks, 1)), _log(rng, 1, 12000), hq, hkv,
                   window=rng.choice((0, 0, _log(rng, 1, 5000))), out=rng.choice(("bf16", "bf16", "float32")))
        c["sinks"] = rng.choice((0, 4, 100)) if c["window"] else 0
    del c["name"]
    return c


# ------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _dev(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _spread(n, lo, hi, salt):
    """n whole numbers over [lo, hi], the first one hi (the same for every seed)."""
    b = np.arange(n, dtype=np.int64)
    x = (b * 2654435761 + 40503 * salt) % 4294967296 % (hi - lo + 1) + lo
    x[:1] = hi
    return x


def _lens(c):
    """(new tokens, tokens with them) of each sequence of a chunk case: the decoding ones first."""
    d, k = c["decodes"], c["chunks"]
    new = np.concatenate([np.ones(d, np.int64), _spread(k, max(1, c["new"] // 8), c["new"], 1)])
    # a lone sequence's context is the case's, others' are half of it to all of it
    before = np.concatenate([_spread(d, c["ctx"] // 2, c["ctx"], 2), _spread(k, c["ctx"] // 2, c["ctx"], 3)])
    return new, before + new


def _channel_scales(g, hkv):
    """Per-channel K and V scales: spread channels, four outlier channels a head, logits of deviation 2."""
    ks = torch.exp2(torch.rand((hkv, DIM), generator=g, device=DEV) * 3 - 2)
    top = torch.rand((hkv, DIM), generator=g, device=DEV).argsort(1)[:, :4]
    ks.scatter_(1, top, ks.gather(1, top) * 8)
    ks *= 2 / ks.square().mean(1, keepdim=True).sqrt()
    vs = torch.exp2(torch.rand((hkv, DIM), generator=g, device=DEV) * 4 - 3)
    return torch.stack([ks, vs], 1)  # [hkv][2][128]


def _storage_order():
    """Flat (token, dim) index, within a 16 x 32 block, of each element in a 12-bit block's storage order: K, V."""
    e = np.arange(512)
    lane, f, i = e // 16, e // 8 % 2, e % 8
    r = lane // 4 + 8 * (i // 2 % 2)
    col = 2 * (lane % 4) + i % 2 + 8 * (i // 4)
    return np.stack([r * 32 + 16 * f + col, col * 32 + 16 * f + r])


def _encode_12bit(pages):
    """BF16 pages [P][hkv][2][16][128] -> arena bytes and metadata [P][hkv][2] of the 12-bit block format."""
    P, hkv = pages.shape[:2]
    order = torch.from_numpy(_storage_order()).to(DEV)
    words = pages.view(torch.int16).unflatten(-1, (4, 32)).transpose(3, 4).reshape(P, hkv, 2, 4, 512)
    words = words.gather(-1, order[None, None, :, None].expand(P, hkv, 2, 4, 512)).to(torch.int32) & 0xFFFF
    exp = words >> 7 & 0xFF
    base = exp.amin(-1) & ~1
    raw = exp.amax(-1) > base + 15
    d = (exp - base[..., None]) >> 1
    sign = words >> 15
    d8, s8 = d.unflatten(-1, (64, 2, 4)), sign.unflatten(-1, (64, 2, 4))
    code = s8[..., 0, :] << 7 | d8[..., 1, :] << 4 | s8[..., 1, :] << 3 | d8[..., 0, :]
    low = words & 0xFF
    small = torch.cat([low, code.flatten(-2), torch.zeros_like(low)[..., :256]], -1).to(torch.uint8)
    big = torch.stack([low, words >> 8], -1).flatten(-2).to(torch.uint8)
    blocks = torch.where(raw[..., None], big, small).view(-1, 4, 256)
    keep = torch.ones(blocks.shape[:2], dtype=torch.bool, device=DEV)
    keep[:, 3] = raw.flatten()
    arena = blocks[keep].flatten()
    size = (3 + raw.to(torch.int64)).sum(-1).flatten()
    offset = (size.cumsum(0) - size).view(P, hkv, 2)
    tag = torch.where(raw, 255, base >> 1).to(torch.int64)
    tags = tag[..., 0] | tag[..., 1] << 8 | tag[..., 2] << 16 | tag[..., 3] << 24
    return arena, offset | tags << 32


def _prepare_chunk(c, seed):
    g = _gen(seed)
    hq, hkv = c["hq"], c["hkv"]
    new, lens = _lens(c)
    order = np.random.RandomState(seed % (1 << 31)).permutation(c["decodes"])  # which decoding sequence has which length
    lens[: c["decodes"]] = lens[: c["decodes"]][order]
    B, width = len(new), -(-int(lens.max()) // PAGE)
    # pages that a token of this step sees; the others are not there any more
    col = np.arange(width)
    used = col[None] * PAGE < lens[:, None]
    if c["window"]:
        first = np.maximum(lens - new - c["window"] + 1, 0) // PAGE
        used &= (col[None] >= first[:, None]) | (col[None] * PAGE < c["sinks"])
    n = int(used.sum())
    pool = (_randn(g, n, hkv, 2, PAGE, DIM) * _channel_scales(g, hkv)[None, :, :, None]).to(torch.bfloat16)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    table[torch.from_numpy(used).to(DEV)] = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
    start = np.concatenate([[0], np.cumsum(new)])
    T = int(start[-1])
    s = {"case": c, "new": new.tolist(), "lens": lens.tolist(), "q": _randn(g, T, hq, DIM).to(torch.bfloat16),
         "q_start": _dev(start), "seq_lens": _dev(lens),
         "out": torch.empty((T, hq, DIM), dtype=torch.float32 if c["out"] == "float32" else torch.bfloat16, device=DEV),
         "status": torch.zeros(1, dtype=torch.int32, device=DEV)}
    if c["format"] == "raw":
        return {**s, "pool": pool, "page_ids": table}
    # whole pages are coded; the tokens behind them stay in one raw page a sequence
    arena, meta = _encode_12bit(pool)
    last = table.long().gather(1, torch.from_numpy(np.minimum(lens // PAGE, width - 1)).to(DEV)[:, None])[:, 0]
    tail = torch.where(s["seq_lens"] % PAGE > 0, torch.arange(B, device=DEV, dtype=torch.int32), -1).to(torch.int32)
    return {**s, "pool": pool[last], "meta": meta, "arena": arena, "tail_page": tail,
            "page_ids": table[:, : int(lens.max()) // PAGE].contiguous()}


def _prepare_append(c, seed):
    g = _gen(seed)
    T, hq, hkv = c["tokens"], c["hq"], c["hkv"]
    # the fused projection's output of these tokens
    qkv = _randn(g, T, (hq + 2 * hkv) * DIM)
    q, k, v = (x.unflatten(1, (-1, DIM)) for x in (qkv * 3).to(torch.bfloat16).split((hq * DIM, hkv * DIM, hkv * DIM), 1))
    pages = (T + 3 if T <= 256 else (T + PAGE - 1) // PAGE + 3)
    pool = _randn(g, pages, hkv, 2, PAGE, DIM).to(torch.bfloat16)
    if T <= 256:  # decode: a page for each token
        slots = torch.randperm(pages, generator=g, device=DEV)[:T] * PAGE + torch.randint(0, PAGE, (T,), generator=g, device=DEV)
        pos = torch.randint(0, c["max_pos"], (T,), generator=g, device=DEV)
    else:  # prefill: consecutive tokens fill consecutive rows of shuffled pages
        i = torch.arange(T, device=DEV)
        slots = torch.randperm(pages, generator=g, device=DEV)[i // PAGE] * PAGE + i % PAGE
        pos = (i + torch.randint(0, c["max_pos"], (1,), generator=g, device=DEV)) % c["max_pos"]
    if c["pad"]:
        slots = torch.where(torch.rand(T, generator=g, device=DEV) < c["pad"], -1, slots)
    n = c["rot"] // 2
    weight = lambda h: (1 + 0.3 * _randn(g, *((h, DIM) if c["per_head"] else (DIM,)))).to(torch.bfloat16)  # noqa: E731
    return {"case": c, "q": q, "k": k, "v": v, "pool": pool, "slots": slots.to(torch.int32),
            "positions": pos.to(torch.int32), "q_norm": weight(hq), "k_norm": weight(hkv),
            "inv_freq": c["base"] ** (-torch.arange(n, device=DEV, dtype=torch.float64) / n),
            "q_out": torch.empty((T, hq, DIM), dtype=torch.bfloat16, device=DEV),
            "status": torch.zeros(1, dtype=torch.int32, device=DEV)}


def _prepare_plan(c, seed):
    g = _gen(seed)
    B, S, width = c["requests"], c["slots"], c["width"]
    rng = np.random.RandomState(seed % (1 << 31))
    new = _spread(B, max(1, c["new"] // 8), c["new"], 1)
    lens = np.zeros(S, np.int64)
    rows = rng.permutation(S)[:B]
    lens[rows] = _spread(B, 0, c["ctx"], 2)[rng.permutation(B)]
    have, want = -(-lens[rows] // PAGE), -(-(lens[rows] + new) // PAGE)
    total = int(have.sum())
    spare = int((want - have).sum()) + 37
    ids = torch.randperm(total + spare, generator=g, device=DEV).to(torch.int32)
    table = torch.full((S, width), -1, dtype=torch.int32, device=DEV)
    held = torch.zeros((S, width), dtype=torch.bool, device=DEV)
    held[torch.from_numpy(rows).to(DEV)] = torch.arange(width, device=DEV) < torch.from_numpy(have).to(DEV)[:, None]
    table[held] = ids[:total]
    T = int(new.sum()) + c["pad"]
    empty = lambda *shape: torch.empty(shape, dtype=torch.int32, device=DEV)  # noqa: E731
    return {"case": c, "rows": _dev(rows), "new": _dev(new), "lens": _dev(lens), "tables": table,
            "free_pages": ids[total:].contiguous(), "free_count": _dev([spare]), "tokens": T,
            "lens_out": empty(S), "free_out": empty(1), "status": torch.zeros(1, dtype=torch.int32, device=DEV)}


def prepare(case, seed):
    return {"chunk": _prepare_chunk, "append": _prepare_append, "plan": _prepare_plan}[case["op"]](case, seed)


# ------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------
def _decode_12bit(meta, arena):
    """Groups of the 12-bit format, metadata [N][hkv][2], as BF16 pages [N][hkv][2][16][128]."""
    tags = torch.stack([meta >> (32 + 8 * j) & 0xFF for j in range(4)], -1)
    size = torch.where(tags == 255, 4, 3)
    first = (meta & 0xFFFFFFFF)[..., None] + size.cumsum(-1) - size
    granules = torch.nn.functional.pad(arena, (0, 256)).view(-1, 256)
    data = granules[first[..., None] + torch.arange(4, device=DEV)].flatten(-2).to(torch.int32)
    big = data[..., 0::2] | data[..., 1::2] << 8
    low = data[..., :512].unflatten(-1, (64, 2, 4))
    code = data[..., 512:768].unflatten(-1, (64, 4))
    high = torch.stack([code & 0x87, code >> 4 & 7 | (code & 8) << 4], -2) + tags[..., None, None, None].to(torch.int32)
    words = torch.where(tags[..., None] == 255, big, (low | high << 8).flatten(-3))
    order = torch.from_numpy(np.argsort(_storage_order(), 1)).to(DEV)
    words = words.gather(-1, order[:, None].expand(*words.shape[:-3], 2, 4, 512))
    words = words.unflatten(-1, (PAGE, 32)).transpose(-3, -2).flatten(-2)
    return torch.where(words >= 32768, words - 65536, words).to(torch.int16).view(torch.bfloat16)


def _plain_batch(s, lo, hi):
    """Attention of the sequences [lo, hi), padded to the longest of them; their output rows, one after another."""
    c = s["case"]
    hq, hkv, W = c["hq"], c["hkv"], c["window"]
    new, lens = s["new"][lo:hi], s["lens"][lo:hi]
    n, longest = max(new), max(lens)
    # the pages that are looked at: the window's, and those of the first tokens before it
    first = [max(a - b - W + 1, 0) // PAGE if W else 0 for a, b in zip(lens, new)]
    cols = torch.arange(max(-(-a // PAGE) - f for a, f in zip(lens, first)), device=DEV) + _dev(first)[:, None]
    ahead = torch.arange(min(-(-c["sinks"] // PAGE), max(first)), device=DEV).expand(hi - lo, -1)
    cols = torch.cat([ahead, cols], 1)  # [sequences][columns]
    twice = torch.arange(cols.shape[1], device=DEV) < ahead.shape[1]
    twice = twice & (cols >= _dev(first)[:, None])  # a page of first tokens that the window has too
    ids = s["page_ids"][lo:hi].long()
    ids = ids.gather(1, cols.clamp(max=ids.shape[1] - 1)).clamp(min=0) if ids.shape[1] else torch.zeros_like(cols)
    if c["format"] == "raw":
        pages = s["pool"][ids]
    else:
        pages = _decode_12bit(s["meta"][ids], s["arena"])
        last = cols == (s["seq_lens"][lo:hi].long() // PAGE)[:, None]
        tail = s["pool"][s["tail_page"][lo:hi].long().clamp(min=0)]
        pages = torch.where(last[:, :, None, None, None, None], tail[:, None], pages)
    at = (cols[:, :, None] * PAGE + torch.arange(PAGE, device=DEV)).flatten(1)  # the columns' token positions
    L = s["seq_lens"][lo:hi, None]
    live = (at < L) & ~twice.repeat_interleave(PAGE, 1)
    kv = pages.permute(0, 2, 3, 1, 4, 5).flatten(3, 4).float()  # [sequences][hkv][2][tokens][128]
    kv = torch.where(live[:, None, None, :, None], kv, 0.0)
    i = torch.arange(n, device=DEV)
    own_rows = i < _dev(new)[:, None]  # [sequences][n]
    token = (s["q_start"][lo:hi].long()[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][token].float().unflatten(2, (hkv, -1)) / math.sqrt(DIM)  # [sequences][n][hkv][G][128]
    score = q.permute(0, 2, 3, 1, 4).flatten(2, 3) @ kv[:, :, 0].transpose(-1, -2)  # [sequences][hkv][G n][tokens]
    p = (L - _dev(new)[:, None] + i)[:, :, None]  # positions of the new tokens
    seen = live[:, None] & (at[:, None] <= p)
    if W:
        seen &= (at[:, None] > p - W) | (at[:, None] < c["sinks"])
    score = score.unflatten(2, (-1, n))
    score = torch.where(seen[:, None, None], score, -math.inf)
    score = torch.exp(score - score.amax(-1, keepdim=True))
    out = (score.flatten(2, 3) @ kv[:, :, 1]).unflatten(2, (-1, n)) / score.sum(-1, keepdim=True)
    return out.permute(0, 3, 1, 2, 4).flatten(2, 3)[own_rows]  # [rows][hq][128]


def _plain_chunk(s):
    d, B = s["case"]["decodes"], len(s["new"])
    parts = ([_plain_batch(s, 0, d)] if d else []) + ([_plain_batch(s, d, B)] if B > d else [])
    s["out"].copy_(torch.cat(parts))
    return s["out"]


def _normed(x, weight):
    """x [T][H][128] in 32 bits over its root mean square, times the weights."""
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()


def _rotate(x, cos, sin, rot, interleaved):
    """x [T][H][128] in 32 bits, cos and sin [T][1][rot/2]."""
    h = x[..., :rot]
    a, b = (h[..., 0::2], h[..., 1::2]) if interleaved else (h[..., : rot // 2], h[..., rot // 2:])
    ra, rb = a * cos - b * sin, a * sin + b * cos
    r = torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _plain_append(s):
    c = s["case"]
    # angles in 64 bits: a far position times a frequency loses its turns in 32
    angle = s["positions"][:, None].double() * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    turn = lambda x, w: _rotate(_normed(x.float(), w), cos, sin, c["rot"], c["interleaved"]).to(torch.bfloat16)  # noqa: E731
    s["q_out"].copy_(turn(s["q"], s["q_norm"]))
    slots = s["slots"].long()
    keep = slots >= 0
    slots, k, v = slots[keep], turn(s["k"], s["k_norm"])[keep], s["v"][keep]
    s["pool"][slots // PAGE, :, 0, slots % PAGE] = k
    s["pool"][slots // PAGE, :, 1, slots % PAGE] = v
    return {"q": s["q_out"], "pool": s["pool"]}


def _plain_plan(s):
    rows, new, T = s["rows"].long(), s["new"].long(), s["tokens"]
    before = s["lens"][rows].long()
    after = before + new
    have, want = (before + PAGE - 1) // PAGE, (after + PAGE - 1) // PAGE
    taken = (want - have).cumsum(0)
    # pages from the end of the free list, requests in order
    col = torch.arange(s["tables"].shape[1], device=DEV)
    nth = (taken - (want - have))[:, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < want[:, None])
    got = s["free_pages"][(s["free_count"].long() - 1 - nth).clamp(min=0, max=s["free_pages"].numel() - 1)]
    table = torch.where(fresh, got, s["tables"][rows])
    s["tables"][rows] = table
    start = torch.cat([torch.zeros_like(taken[:1]), new.cumsum(0)])
    i = torch.arange(T, device=DEV)
    of = torch.searchsorted(start[1:], i, right=True)
    live = of < rows.numel()
    of = of.clamp(max=rows.numel() - 1)
    pos = torch.where(live, before[of] + i - start[of], 0)
    page = table[of, (pos // PAGE).clamp(max=col.numel() - 1)]
    s["lens_out"].copy_(s["lens"])
    s["lens_out"][rows] = after.to(torch.int32)
    s["free_out"].copy_(s["free_count"] - taken[-1])
    return {"q_start": start.to(torch.int32), "seq_lens": after.to(torch.int32),
            "page_ids": torch.where(col < want[:, None], table, -1), "positions": pos.to(torch.int32),
            "slots": torch.where(live, page * PAGE + pos % PAGE, -1).to(torch.int32), "tables": s["tables"],
            "lens": s["lens_out"], "free": s["free_out"]}


# ------------------------------------------------------------------------------------
# the package's calls
# ------------------------------------------------------------------------------------
def _own_chunk(s):
    import decode_attention_value_gb300 as kvz

    c = s["case"]
    coded = c["format"] != "raw"
    if "workspace" not in s:
        size = kvz.chunk_attention_workspace_size(c["hkv"], s["q"].shape[0], c["hq"], len(s["new"]),
                                                  s["page_ids"].shape[1], coded=coded)
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    if coded:
        kvz.chunk_attention(s["q"], s["q_start"], s["page_ids"], s["seq_lens"], s["tail_page"], s["meta"], s["arena"],
                            s["pool"], s["out"], s["status"], window=c["window"], sinks=c["sinks"],
                            workspace=s["workspace"])
    else:
        kvz.chunk_attention_raw(s["q"], s["q_start"], s["page_ids"], s["seq_lens"], s["pool"], s["out"], s["status"],
                                window=c["window"], sinks=c["sinks"], workspace=s["workspace"])
    return s["out"]


def _own_append(s):
    import decode_attention_value_gb300 as kvz

    if "rope" not in s:  # a model constant
        s["rope"] = kvz.rope_table(s["inv_freq"])
    c = s["case"]
    kvz.append_tokens(s["k"], s["v"], s["slots"], s["pool"], s["status"], q=s["q"], q_out=s["q_out"], rope=s["rope"],
                      positions=s["positions"], interleaved=c["interleaved"], q_norm=s["q_norm"], k_norm=s["k_norm"],
                      norm_eps=1e-6)
    return {"q": s["q_out"], "pool": s["pool"]}


def _own_plan(s):
    import decode_attention_value_gb300 as kvz

    if "plan" not in s:  # the step's buffers, kept by the loop
        s["plan"] = kvz.new_step_plan(s["case"]["requests"], s["tokens"], s["case"]["width"])
    p = kvz.plan_step(s["rows"], s["new"], s["lens"], s["tables"], s["free_pages"], s["free_count"], s["plan"],
                      s["status"], lens_out=s["lens_out"], free_out=s["free_out"])
    return {"q_start": p.q_start, "seq_lens": p.seq_lens, "page_ids": p.page_ids, "positions": p.positions,
            "slots": p.slots, "tables": s["tables"], "lens": s["lens_out"], "free": s["free_out"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"chunk": _own_chunk, "append": _own_append, "plan": _own_plan}[op](state)
    return {"chunk": _plain_chunk, "append": _plain_append, "plan": _plain_plan}[op](state)


# ------------------------------------------------------------------------------------
# least work, exact values
# ------------------------------------------------------------------------------------
def _pairs(c, new, lens):
    """(query, key) pairs of one query head, and keys that any of a sequence's new tokens sees, over the sequences."""
    pairs = keys = 0
    for n, L in zip(new.tolist(), lens.tolist()):
        p = np.arange(L - n, L)
        if not c["window"]:
            pairs += int((p + 1).sum())
            keys += L
            continue
        first = np.maximum(p - c["window"] + 1, 0)
        pairs += int((p + 1 - first + np.minimum(first, c["sinks"])).sum())
        keys += L - int(first[0]) + min(int(first[0]), c["sinks"])
    return pairs, keys


def work(case):
    c = case
    if c["op"] == "append":
        T, live = c["tokens"], 1 - c["pad"]
        heads = c["hq"] + 2 * c["hkv"] * live  # padding tokens have no K and V to move
        return {"bytes": T * (heads * DIM * 2 * 2 + 4 + 4) + (c["hq"] + c["hkv"] if c["per_head"] else 2) * DIM * 2,
                "flops": T * (c["hq"] + c["hkv"] * live) * (c["rot"] * 3 + 4 * DIM)}
    if c["op"] == "plan":
        s = _spread(c["requests"], max(1, c["new"] // 8), c["new"], 1)
        T, lens = int(s.sum()) + c["pad"], _spread(c["requests"], 0, c["ctx"], 2)
        held = int((-(-(lens + s) // PAGE)).sum())
        # lengths, the requests' pages read and the step's table written, two numbers a token
        return {"bytes": 4 * (6 * c["requests"] + 2 * c["slots"] + held + c["requests"] * c["width"] + 2 * T), "flops": 0}
    new, lens = _lens(c)
    pairs, keys = _pairs(c, new, lens)
    size = 512 if c["format"] == "raw" else 385  # bytes a token and KV head: 12-bit pages and their metadata
    out = 4 if c["out"] == "float32" else 2
    return {"bytes": keys * c["hkv"] * size + int(new.sum()) * c["hq"] * DIM * (2 + out), "flops": pairs * c["hq"] * 4 * DIM}


def _exact_chunk(c, seed):
    # the same numbers before they were coded: a raw case of the same seed
    s = _prepare_chunk({**c, "format": "raw"}, seed)
    hkv, G = c["hkv"], c["hq"] // c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for b, (n, L) in enumerate(zip(s["new"], s["lens"])):
        ids = s["page_ids"][b].long()
        for r0 in range(0, n, 256):  # 256 tokens at a time
            r1 = min(n, r0 + 256)
            pos = torch.arange(L - n + r0, L - n + r1, device=DEV)
            j = torch.arange(L - n + r1, device=DEV)  # keys up to the last one's own
            if c["window"]:
                j = j[(j > int(pos[0]) - c["window"]) | (j < c["sinks"])]
            kv = s["pool"][ids[j // PAGE], :, :, j % PAGE].double()  # [keys][hkv][2][128]
            hide = j[None] > pos[:, None]
            if c["window"]:
                hide |= (j[None] <= pos[:, None] - c["window"]) & (j[None] >= c["sinks"])
            for h in range(hkv):
                q = s["q"][at + r0: at + r1, h * G: (h + 1) * G].double()
                score = torch.einsum("tgd,kd->gtk", q, kv[:, h, 0]) / DIM ** 0.5
                w = torch.softmax(score.masked_fill(hide, -math.inf), -1)
                out[at + r0: at + r1, h * G: (h + 1) * G] = torch.einsum("gtk,kd->tgd", w, kv[:, h, 1])
        at += n
    return out


def _exact_append(c, seed):
    s = _prepare_append(c, seed)
    n = c["rot"] // 2
    unit = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       torch.outer(s["positions"].double(), s["inv_freq"]))[:, None]

    def turned(x, weight):
        x = x.double()
        y = x / torch.linalg.vector_norm(torch.cat([x / DIM ** 0.5, torch.full_like(x[..., :1], 1e-3)], -1), dim=-1)[..., None]
        y = y * weight.double()
        pairs = y[..., : 2 * n].reshape(*y.shape[:2], n, 2) if c["interleaved"] else \
            torch.stack(y[..., : 2 * n].chunk(2, -1), -1)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit)
        y[..., : 2 * n] = z.flatten(-2) if c["interleaved"] else torch.cat(z.unbind(-1), -1)
        return y

    pool = s["pool"].double().permute(0, 3, 1, 2, 4).flatten(0, 1)  # [slots][hkv][2][128]
    live = torch.nonzero(s["slots"] >= 0)[:, 0]
    pool[s["slots"][live].long()] = torch.stack([turned(s["k"], s["k_norm"]), s["v"].double()], 2)[live]
    return {"q": turned(s["q"], s["q_norm"]), "pool": pool.unflatten(0, (-1, PAGE)).permute(0, 2, 3, 1, 4).contiguous()}


def exact(case, seed):
    if case["op"] == "plan":  # whole numbers
        return None
    return (_exact_append if case["op"] == "append" else _exact_chunk)(case, seed)
