"""Cases for the cache-append and shared-prefix attention operators.

Each operator has a plain form in elementary torch operations (``own`` False) and the call a user makes of the package
(``own`` True).  Sizes follow the package's own decode workloads: 16-token pages, head dimension 128, 1 to 8 query
heads per KV head, contexts from one token to 131072.
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
def _append(name, tokens, hq, hkv, rot=128, interleaved=False, axes=1, max_pos=8192, pad=0.0, base=500000.0):
    return {"op": "append", "name": name, "tokens": tokens, "hq": hq, "hkv": hkv, "rot": rot,
            "interleaved": interleaved, "axes": axes, "max_pos": max_pos, "pad": pad, "base": base}


def _prefix(name, fmt, groups, per_group, hq, hkv, prefix, own_max, out="bf16"):
    return {"op": "prefix", "name": name, "format": fmt, "groups": groups, "per_group": per_group, "hq": hq,
            "hkv": hkv, "prefix": prefix, "own_max": own_max, "out": out}


def listed():
    return [
        # one sequence decoding far into its context: the latency of a layer's append
        _append("append-decode-1", 1, 32, 8, max_pos=131072),
        # a decode batch of 64 sequences, 8 query heads per KV head
        _append("append-decode-64", 64, 64, 8, max_pos=131072),
        # ragged prompts packed into one prefill batch, some padding tokens at the end of each
        _append("append-prefill", 16381, 32, 8, max_pos=32768, pad=0.03),
        # neighbouring-pair rotation of half of the dimensions
        _append("append-interleaved", 2047, 40, 8, rot=64, interleaved=True, base=10000.0),
        # one image in a prompt: time, height and width positions
        _append("axes-image", 1021, 32, 8, axes=3, max_pos=4096, base=1000000.0),
        # a clip of video frames
        _append("axes-video", 12289, 32, 8, axes=3, max_pos=16384, base=1000000.0),
        # four samples of one short prompt
        _prefix("prefix-raw-short", "raw", 1, 4, 8, 2, 263, 40),
        # a decode batch behind one system prompt
        _prefix("prefix-raw-chat", "raw", 1, 32, 32, 8, 2055, 255),
        # four prompts, sixteen samples of each, 5 query heads per KV head
        _prefix("prefix-raw-groups", "raw", 4, 16, 40, 8, 8191, 120),
        # many sequences behind one document: bound by the matrix products
        _prefix("prefix-raw-wide", "raw", 1, 128, 64, 8, 16384, 200),
        # the 12-bit pages at an 8K prefix
        _prefix("prefix-12bit-8k", "12bit", 1, 16, 32, 8, 8192, 255, out="float32"),
        # a 128K document in 12-bit pages, a few raw tokens behind its last whole page
        _prefix("prefix-12bit-long", "12bit", 1, 16, 32, 8, 131079, 300),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    hkv = rng.choice((1, 2, 4, 8))
    hq = hkv * rng.randint(1, 8)
    if rng.random() < 0.4:
        axes = rng.choice((1, 1, 2, 3, 4))
        c = _append("", _log(rng, 1, 12000), hq, hkv, rot=rng.choice((16, 32, 64, 96, 128, 128)),
                    interleaved=rng.random() < 0.4, axes=axes, max_pos=_log(rng, 64, 1 << 20),
                    pad=rng.choice((0.0, 0.05)), base=rng.choice((10000.0, 500000.0)))
    else:
        fmt = rng.choice(("raw", "12bit"))
        groups = rng.choice((1, 1, 2, 5))
        rows = _log(rng, 1, 400 // groups)  # query rows of a group and KV head
        c = _prefix("", fmt, groups, max(1, rows // (hq // hkv)), hq, hkv, _log(rng, 1, 40000 // groups),
                    _log(rng, 1, 300), out=rng.choice(("bf16", "bf16", "float32")))
    del c["name"]
    return c


# ------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 11)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _own_lens(c):
    """Own tokens of each sequence, 0 to own_max (the multiset is the same for every seed)."""
    b = np.arange(c["groups"] * c["per_group"], dtype=np.int64)
    return (b * 2654435761 + 40503) % 4294967296 % (c["own_max"] + 1)


def _prefix_lens(c):
    """Prefix tokens of each group: the first as the case says, the others shorter."""
    return [max(1, c["prefix"] - i * (c["prefix"] // 7)) for i in range(c["groups"])]


def _channel_scales(g, hkv):
    """Per-channel K and V scales: spread channels, four outlier channels a head, logits of deviation 2."""
    ks = torch.exp2(torch.rand((hkv, DIM), generator=g, device=DEV) * 3 - 2)
    top = torch.rand((hkv, DIM), generator=g, device=DEV).argsort(1)[:, :4]
    ks.scatter_(1, top, ks.gather(1, top) * 8)
    ks *= 2 / ks.square().mean(1, keepdim=True).sqrt()
    vs = torch.exp2(torch.rand((hkv, DIM), generator=g, device=DEV) * 4 - 3)
    return torch.stack([ks, vs], 1)  # [hkv][2][128]


def _prepare_append(c, seed):
    g = _gen(seed)
    T, hq, hkv = c["tokens"], c["hq"], c["hkv"]
    # the fused projection's output of these tokens
    qkv = _randn(g, T, (hq + 2 * hkv) * DIM).to(torch.bfloat16)
    q, k, v = (x.unflatten(1, (-1, DIM)) for x in qkv.split((hq * DIM, hkv * DIM, hkv * DIM), 1))
    pages = (T + PAGE - 1) // PAGE + 3
    pool = _randn(g, pages, hkv, 2, PAGE, DIM).to(torch.bfloat16)
    table = torch.randperm(pages, generator=g, device=DEV)
    if T <= 256:  # decode: a page for each token
        pool = _randn(g, T + 3, hkv, 2, PAGE, DIM).to(torch.bfloat16)
        row = torch.randint(0, PAGE, (T,), generator=g, device=DEV)
        slots = torch.randperm(T + 3, generator=g, device=DEV)[:T] * PAGE + row
        first = torch.randint(0, c["max_pos"], (T,), generator=g, device=DEV)
    else:  # prefill: consecutive tokens fill consecutive rows of shuffled pages
        i = torch.arange(T, device=DEV)
        slots = table[i // PAGE] * PAGE + i % PAGE
        first = (i + torch.randint(0, c["max_pos"], (1,), generator=g, device=DEV)) % c["max_pos"]
    if c["pad"]:
        slots = torch.where(torch.rand(T, generator=g, device=DEV) < c["pad"], -1, slots)
    pos = [first]
    for _ in range(c["axes"] - 1):  # heights and widths start at the text position before the image
        pos.append(first // 2 + torch.randint(0, 64, (T,), generator=g, device=DEV))
    n = c["rot"] // 2
    inv_freq = c["base"] ** (-torch.arange(n, device=DEV, dtype=torch.float64) / n)
    axis = torch.arange(n, device=DEV) * c["axes"] // n  # contiguous sections of the pairs
    return {"case": c, "q": q, "k": k, "v": v, "pool": pool, "slots": slots.to(torch.int32),
            "positions": torch.stack(pos).to(torch.int32), "inv_freq": inv_freq, "axis": axis,
            "q_out": torch.empty((T, hq, DIM), dtype=torch.bfloat16, device=DEV),
            "status": torch.zeros(1, dtype=torch.int32, device=DEV)}


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


def _prepare_prefix(c, seed):
    g = _gen(seed)
    hq, hkv = c["hq"], c["hkv"]
    B = c["groups"] * c["per_group"]
    plens = _prefix_lens(c)
    lens = _own_lens(c)[np.random.RandomState(seed % (1 << 31)).permutation(B)]
    width, own_width = (max(plens) + PAGE - 1) // PAGE, (c["own_max"] + PAGE - 1) // PAGE
    n = c["groups"] * width + B * own_width
    pool = (_randn(g, n, hkv, 2, PAGE, DIM) * _channel_scales(g, hkv)[None, :, :, None]).to(torch.bfloat16)
    ids = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
    ptable = ids[: c["groups"] * width].view(c["groups"], width)
    table = ids[c["groups"] * width:].view(B, own_width)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    s = {"case": c, "q": _randn(g, B, hq, DIM).to(torch.bfloat16), "prefix_lens": dev(plens), "seq_lens": dev(lens),
         "group_start": dev(np.arange(c["groups"] + 1) * c["per_group"]),
         "out": torch.empty((B, hq, DIM), dtype=torch.float32 if c["out"] == "float32" else torch.bfloat16, device=DEV),
         "status": torch.zeros(1, dtype=torch.int32, device=DEV)}
    if c["format"] == "raw":
        return {**s, "pool": pool, "prefix_ids": ptable.contiguous(), "page_ids": table.contiguous()}
    # whole pages are coded; the tokens behind them stay in one raw page a group and a sequence
    arena, meta = _encode_12bit(pool)
    pt = ptable.long().gather(1, (s["prefix_lens"].long() // PAGE).clamp(max=width - 1)[:, None])[:, 0]
    st = table.long().gather(1, (s["seq_lens"].long() // PAGE).clamp(max=own_width - 1)[:, None])[:, 0]
    tails = pool[torch.cat([pt, st])]
    which = torch.arange(c["groups"] + B, device=DEV, dtype=torch.int32)
    rest = torch.cat([s["prefix_lens"], s["seq_lens"]]) % PAGE
    which = torch.where(rest > 0, which, -1).to(torch.int32)
    return {**s, "pool": tails, "meta": meta, "arena": arena,
            "prefix_ids": ptable[:, : max(plens) // PAGE].contiguous(), "prefix_tail": which[: c["groups"]].contiguous(),
            "page_ids": table[:, : c["own_max"] // PAGE].contiguous(), "tail_page": which[c["groups"]:].contiguous()}


def prepare(case, seed):
    return (_prepare_append if case["op"] == "append" else _prepare_prefix)(case, seed)


# ------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------
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
    angle = s["positions"][s["axis"]].T.double() * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    rot = lambda x: _rotate(x.float(), cos, sin, c["rot"], c["interleaved"]).to(torch.bfloat16)  # noqa: E731
    s["q_out"].copy_(rot(s["q"]))
    slots = s["slots"].long()
    keep = slots >= 0
    slots, k, v = slots[keep], rot(s["k"])[keep], s["v"][keep]
    s["pool"][slots // PAGE, :, 0, slots % PAGE] = k
    s["pool"][slots // PAGE, :, 1, slots % PAGE] = v
    return {"q": s["q_out"], "pool": s["pool"]}


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


def _plain_prefix(s):
    c = s["case"]
    hq, hkv, groups, per = c["hq"], c["hkv"], c["groups"], c["per_group"]
    G = hq // hkv

    def rows(ids, lens, tail):  # [n][hkv][2][tokens][128] in 32 bits
        pages = s["pool"][ids.long()] if "meta" not in s else _whole_pages(s, ids, lens, tail)
        x = pages.permute(0, 2, 3, 1, 4, 5).flatten(3, 4).float()
        live = torch.arange(x.shape[3], device=DEV) < lens[:, None]
        return torch.where(live[:, None, None, :, None], x, 0.0), live

    pre, plive = rows(s["prefix_ids"], s["prefix_lens"], s.get("prefix_tail"))
    mine, live = rows(s["page_ids"], s["seq_lens"], s.get("tail_page"))
    q = s["q"].float().view(groups, per, hkv, G, DIM) / math.sqrt(DIM)
    a = q.permute(0, 2, 1, 3, 4).flatten(2, 3) @ pre[:, :, 0].transpose(-1, -2)  # [groups][hkv][per G][tokens]
    a = torch.where(plive[:, None, None], a, -math.inf)
    b = q.flatten(0, 1) @ mine[:, :, 0].transpose(-1, -2)  # [B][hkv][G][own tokens]
    b = torch.where(live[:, None, None], b, -math.inf)
    a_top = a.amax(-1).unflatten(2, (per, G)).transpose(1, 2).flatten(0, 1)  # [B][hkv][G]
    top = torch.maximum(a_top, b.amax(-1)) if b.shape[-1] else a_top
    a = torch.exp(a - top.unflatten(0, (groups, per)).transpose(1, 2).flatten(2, 3)[..., None])
    b = torch.exp(b - top[..., None])
    num = (a @ pre[:, :, 1]).unflatten(2, (per, G)).transpose(1, 2).flatten(0, 1) + b @ mine[:, :, 1]
    den = a.sum(-1).unflatten(2, (per, G)).transpose(1, 2).flatten(0, 1) + b.sum(-1)
    s["out"].copy_((num / den[..., None]).flatten(1, 2))
    return s["out"]


def _whole_pages(s, ids, lens, tail):
    """The rows' pages with the raw tail page in its place behind the decoded ones."""
    pages = _decode_12bit(s["meta"][ids.long()], s["arena"])
    pages = torch.cat([pages, torch.zeros_like(s["pool"][: ids.shape[0], None])], 1)
    n = torch.arange(ids.shape[0], device=DEV)
    at = lens.long() // PAGE
    last = torch.where((tail >= 0)[:, None, None, None, None], s["pool"][tail.long().clamp(min=0)], pages[n, at])
    pages[n, at] = last
    return pages


# ------------------------------------------------------------------------------------
# the package's calls
# ------------------------------------------------------------------------------------
def _own_append(s):
    import decode_attention_value_gb300 as kvz

    if "rope" not in s:  # a model constant
        s["rope"] = kvz.rope_table(s["inv_freq"], s["axis"])
    c = s["case"]
    kvz.append_tokens(s["k"], s["v"], s["slots"], s["pool"], s["status"], q=s["q"], q_out=s["q_out"], rope=s["rope"],
                      positions=s["positions"], interleaved=c["interleaved"])
    return {"q": s["q_out"], "pool": s["pool"]}


def _own_prefix(s):
    import decode_attention_value_gb300 as kvz

    c = s["case"]
    if "workspace" not in s:
        size = kvz.prefix_attention_workspace_size(c["hkv"], s["q"].shape[0], c["hq"], c["groups"],
                                                   s["prefix_ids"].shape[1], s["page_ids"].shape[1])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    if c["format"] == "raw":
        kvz.prefix_attention_raw(s["q"], s["group_start"], s["prefix_ids"], s["prefix_lens"], s["page_ids"],
                                 s["seq_lens"], s["pool"], s["out"], s["status"], workspace=s["workspace"])
    else:
        kvz.prefix_attention(s["q"], s["group_start"], s["prefix_ids"], s["prefix_lens"], s["prefix_tail"],
                             s["page_ids"], s["seq_lens"], s["tail_page"], s["meta"], s["arena"], s["pool"], s["out"],
                             s["status"], workspace=s["workspace"])
    return s["out"]


def run(state):
    if state["case"]["op"] == "append":
        return _own_append(state) if own else _plain_append(state)
    return _own_prefix(state) if own else _plain_prefix(state)


# ------------------------------------------------------------------------------------
# least work, exact values
# ------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "append":
        T, live = c["tokens"], 1 - c["pad"]
        heads = c["hq"] + 2 * c["hkv"] * live  # padding tokens have no K and V to move
        return {"bytes": T * (heads * DIM * 2 * 2 + 4 + 4 * c["axes"]),
                "flops": T * (c["hq"] + c["hkv"] * live) * c["rot"] * 3}
    B, plens, lens = c["groups"] * c["per_group"], _prefix_lens(c), _own_lens(c)
    tokens = sum(plens) + int(lens.sum())
    size = 512 if c["format"] == "raw" else 385  # bytes a token and KV head: 12-bit pages and their metadata
    out = 4 if c["out"] == "float32" else 2
    rows = sum(p * c["per_group"] for p in plens) + int(lens.sum())
    return {"bytes": tokens * c["hkv"] * size + B * c["hq"] * DIM * (2 + out), "flops": rows * c["hq"] * 4 * DIM}


def _exact_append(c, seed):
    s = _prepare_append(c, seed)
    n = c["rot"] // 2
    turn = torch.stack([s["positions"][int(a)].double() * f for a, f in zip(s["axis"].tolist(), s["inv_freq"])], 1)
    unit = torch.polar(torch.ones_like(turn), turn)[:, None]

    def rotated(x):
        x = x.double()
        pairs = x[..., : 2 * n].reshape(*x.shape[:2], n, 2) if c["interleaved"] else \
            torch.stack(x[..., : 2 * n].chunk(2, -1), -1)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * unit)
        y = x.clone()
        y[..., : 2 * n] = z.flatten(-2) if c["interleaved"] else torch.cat(z.unbind(-1), -1)
        return y

    pool = s["pool"].double().permute(0, 3, 1, 2, 4).flatten(0, 1)  # [slots][hkv][2][128]
    live = torch.nonzero(s["slots"] >= 0)[:, 0]
    pool[s["slots"][live].long()] = torch.stack([rotated(s["k"]), s["v"].double()], 2)[live]
    return {"q": rotated(s["q"]), "pool": pool.unflatten(0, (-1, PAGE)).permute(0, 2, 3, 1, 4).contiguous()}


def _exact_prefix(c, seed):
    # the same numbers before they were coded: a raw case of the same seed
    s = _prepare_prefix({**c, "format": "raw"}, seed)
    hkv, G = c["hkv"], c["hq"] // c["hkv"]
    out = torch.empty((s["q"].shape[0], c["hq"], DIM), dtype=torch.float64, device=DEV)
    lens = s["seq_lens"].tolist()
    for i, n in enumerate(s["prefix_lens"].tolist()):
        pre = s["pool"][s["prefix_ids"][i].long()].double().permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :n]
        for b in range(i * c["per_group"], (i + 1) * c["per_group"]):
            mine = s["pool"][s["page_ids"][b].long()].double().permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, : lens[b]]
            q = s["q"][b].double().view(hkv, G, DIM)
            score = torch.cat([q @ pre[:, 0].mT, q @ mine[:, 0].mT], -1) / DIM ** 0.5
            p = torch.softmax(score, -1)
            out[b] = (p[..., :n] @ pre[:, 1] + p[..., n:] @ mine[:, 1]).flatten(0, 1)
    return out


def exact(case, seed):
    return (_exact_append if case["op"] == "append" else _exact_prefix)(case, seed)
