"""kvz_append_tokens on the GPU against the rotation in 64 bits: rotary pairings, partial and
several-axis rotation, strides, padding, bad slots, far positions, streams and graphs."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

PAGE, D = 16, 128


def _table(kvz, rot, base=500000.0, axes=1):
    n = rot // 2
    inv = base ** (-torch.arange(n, dtype=torch.float64) / max(n, 1))
    axis = torch.arange(n) * axes // max(n, 1)
    return kvz.rope_table(inv, axis).cuda()


def _angles(table, positions):
    """Angles of the table's definition: position * turns, modulo one turn in integers."""
    t, ax = table[:, 0].cpu(), table[:, 1].cpu()
    pos = positions.cpu().to(torch.int64).reshape(-1, positions.shape[-1])
    wrapped = pos[ax].T * t  # int64 multiplication wraps modulo 2^64, that is one turn
    return wrapped.double() * (2 * math.pi / 2.0 ** 64)


def _rotated(x, ang, rot, interleaved, scale=1.0):
    """64-bit rotation of x [T][H][128] and, per value, |a| + |b| of its pair."""
    x = x.cpu().double()
    if rot == 0:
        return x, torch.zeros_like(x)
    c, s = (scale * ang.cos())[:, None], (scale * ang.sin())[:, None]
    h = x[..., :rot]
    a, b = (h[..., 0::2], h[..., 1::2]) if interleaved else h.chunk(2, -1)
    ra, rb, m = a * c - b * s, a * s + b * c, scale * (a.abs() + b.abs())
    out, mag = x.clone(), torch.zeros_like(x)
    join = (lambda p, q: torch.stack([p, q], -1).flatten(-2)) if interleaved else (lambda p, q: torch.cat([p, q], -1))
    out[..., :rot], mag[..., :rot] = join(ra, rb), join(m, m)
    return out, mag


def _close(got, want, mag, what):
    # one rounding to bf16 (half a step, 2^-8 of the value) of an fp32 value that is off by at
    # most 2^-21 (|a| + |b|): sine and cosine 1.5 * 2^-24, their argument 2^-23, two products
    # and a sum 2^-24 each
    err = (got.cpu().double() - want).abs()
    tol = 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * 2.0 ** -21 * mag
    assert (err <= tol).all(), f"{what}: {(err - tol).max().item():.3e} over"
    plain = mag == 0
    assert torch.equal(got.cpu().double()[plain], want[plain]), f"{what}: unrotated values changed"


def _inputs(T, hq, hkv, pages, seed=0, fused=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn((T, (hq + 2 * hkv) * D), generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split((hq * D, hkv * D, hkv * D), 1))
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pool = torch.randn((pages, hkv, 2, PAGE, D), generator=g, device="cuda").to(torch.bfloat16)
    slots = torch.randperm(pages * PAGE, generator=g, device="cuda")[:T].to(torch.int32)
    return q, k, v, pool, slots


def _check(kvz, q, k, v, pool, slots, table, positions, rot, interleaved, scale=1.0, q_out=None, bad=0):
    before, status = pool.clone(), kvz.new_status()
    out = kvz.append_tokens(k, v, slots, pool, status, q=q, q_out=q_out, rope=table, positions=positions,
                            interleaved=interleaved, rope_scale=scale)
    torch.cuda.synchronize()
    assert int(status.item()) == bad
    ang = _angles(table, positions) if rot else None
    if q is not None:
        _close(out, *_rotated(q, ang, rot, interleaved, scale), "q")
    live = ((slots >= 0) & (slots < pool.shape[0] * PAGE)).cpu()
    at = slots.cpu().long()[live]
    got = pool.permute(0, 3, 1, 2, 4).flatten(0, 1)  # [slots][hkv][2][128]
    want_k, mag = _rotated(k, ang, rot, interleaved, scale)
    _close(got[at.cuda(), :, 0], want_k[live], mag[live], "k")
    assert torch.equal(got[at.cuda(), :, 1], v[live.cuda()])
    rest = torch.ones(pool.shape[0] * PAGE, dtype=torch.bool)
    rest[at] = False
    old = before.permute(0, 3, 1, 2, 4).flatten(0, 1)
    assert torch.equal(got[rest.cuda()].view(torch.int16), old[rest.cuda()].view(torch.int16)), "other rows changed"
    return out


@pytest.mark.parametrize("T,hq,hkv", [(1, 32, 8), (1, 1, 1), (2, 3, 1), (7, 8, 2), (64, 64, 8), (129, 40, 8),
                                      (1021, 5, 5), (4099, 32, 8)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_matches_64_bits(T, hq, hkv, interleaved):
    import decode_attention_value_gb300 as kvz

    q, k, v, pool, slots = _inputs(T, hq, hkv, T // PAGE + 4, seed=T)
    pos = torch.randint(0, 131072, (T,), device="cuda", dtype=torch.int32)
    _check(kvz, q, k, v, pool, slots, _table(kvz, 128), pos, 128, interleaved)


@pytest.mark.parametrize("rot", [0, 16, 32, 48, 96, 112])
@pytest.mark.parametrize("interleaved", [False, True])
def test_partial_rotation(rot, interleaved):
    import decode_attention_value_gb300 as kvz

    q, k, v, pool, slots = _inputs(37, 6, 2, 5, seed=rot, fused=False)
    pos = torch.randint(0, 5000, (37,), device="cuda", dtype=torch.int32)
    table = _table(kvz, rot) if rot else None
    _check(kvz, q, k, v, pool, slots, table, pos if rot else None, rot, interleaved)


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("T", [1, 65, 700])
def test_several_axes(axes, T):
    import decode_attention_value_gb300 as kvz

    q, k, v, pool, slots = _inputs(T, 8, 4, T // PAGE + 2, seed=axes)
    pos = torch.randint(0, 40000, (axes, T), device="cuda", dtype=torch.int32)
    # contiguous sections and a round robin over the axes
    _check(kvz, q, k, v, pool, slots, _table(kvz, 128, axes=axes), pos, 128, False)
    table = _table(kvz, 128)
    table[:, 1] = torch.arange(64) % axes
    _check(kvz, q, k, v, pool, slots, table, pos, 128, True)


def test_equal_axes_are_one_axis():
    import decode_attention_value_gb300 as kvz

    q, k, v, pool, slots = _inputs(33, 8, 2, 4)
    pos = torch.randint(0, 9000, (33,), device="cuda", dtype=torch.int32)
    st, other = kvz.new_status(), pool.clone()
    a = kvz.append_tokens(k, v, slots, pool, st, q=q, rope=_table(kvz, 128), positions=pos)
    b = kvz.append_tokens(k, v, slots, other, st, q=q, rope=_table(kvz, 128, axes=3), positions=pos.expand(3, 33).contiguous())
    assert torch.equal(a, b) and torch.equal(pool, other) and int(st.item()) == 0


def test_far_and_negative_positions_wrap_exactly():
    import decode_attention_value_gb300 as kvz

    pos = torch.tensor([0, 1, -1, 2 ** 20 + 1, 2 ** 31 - 1, -2 ** 31, 123456789], device="cuda", dtype=torch.int32)
    q, k, v, pool, slots = _inputs(pos.numel(), 4, 2, 2, seed=3)
    _check(kvz, q, k, v, pool, slots, _table(kvz, 128, base=10000.0), pos, 128, False, scale=1.25)


def test_padding_and_bad_slots():
    import decode_attention_value_gb300 as kvz

    T = 50
    q, k, v, pool, slots = _inputs(T, 8, 2, 6, seed=5)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    slots[::3] = -1
    _check(kvz, q, k, v, pool, slots, _table(kvz, 128), pos, 128, False)
    slots[4], slots[5], slots[7] = 6 * PAGE, -2, 2 ** 31 - 1
    _check(kvz, q, k, v, pool, slots, _table(kvz, 128), pos, 128, False, bad=kvz.STATUS_BAD_INDEX)
    slots.fill_(-1)
    _check(kvz, q, k, v, pool, slots, _table(kvz, 128), pos, 128, False)


def test_bad_axis_is_flagged_and_not_turned():
    import decode_attention_value_gb300 as kvz

    q, k, v, pool, slots = _inputs(3, 2, 1, 2)
    pos = torch.tensor([5, 6, 7], device="cuda", dtype=torch.int32)
    table = _table(kvz, 128)
    table[9, 1], table[10, 1] = 1, -1
    st = kvz.new_status()
    out = kvz.append_tokens(k, v, slots, pool, st, q=q, rope=table, positions=pos)
    assert int(st.item()) == kvz.STATUS_BAD_INDEX
    for d in (9, 10, 73, 74):
        assert torch.equal(out[..., d], q[..., d])


def test_queries_alone_keys_alone_and_in_place():
    import decode_attention_value_gb300 as kvz

    q, k, v, pool, slots = _inputs(70, 16, 4, 6, seed=8, fused=False)
    pos = torch.randint(0, 3000, (70,), device="cuda", dtype=torch.int32)
    table, st = _table(kvz, 128), kvz.new_status()
    want = _check(kvz, q, k, v, pool, slots, table, pos, 128, False)
    filled = pool.clone()
    alone = kvz.append_tokens(None, None, None, None, st, q=q, rope=table, positions=pos)
    assert torch.equal(alone, want)
    pool.zero_()
    assert kvz.append_tokens(k, v, slots, pool, st, rope=table, positions=pos) is None
    at = slots.long()
    assert torch.equal(pool[at // PAGE, :, :, at % PAGE], filled[at // PAGE, :, :, at % PAGE])
    inplace = q.clone()
    assert kvz.append_tokens(None, None, None, None, st, q=inplace, q_out=inplace, rope=table, positions=pos) is inplace
    assert torch.equal(inplace, want) and int(st.item()) == 0


def test_head_strides_zero_strides_and_no_tokens():
    import decode_attention_value_gb300 as kvz

    q, k, v, pool, slots = _inputs(21, 4, 4, 3, seed=9)
    pos = torch.arange(21, device="cuda", dtype=torch.int32)
    kv = torch.stack([k, v], 2)  # [T][hkv][2][128]: the cache's order, head stride 256
    kt = k.transpose(0, 1).contiguous().transpose(0, 1)  # head-major
    one = v[:, :1].expand(21, 4, D)  # one value head shared by all
    _check(kvz, q, kv[:, :, 0], kv[:, :, 1], pool, slots, _table(kvz, 128), pos, 128, False)
    _check(kvz, q, kt, one, pool, slots, _table(kvz, 128), pos, 128, True)
    st = kvz.new_status()
    out = kvz.append_tokens(k[:0], v[:0], slots[:0], pool, st, q=q[:0], rope=_table(kvz, 128), positions=pos[:0])
    assert out.shape == (0, 4, D) and int(st.item()) == 0


def test_special_values_are_copied():
    import decode_attention_value_gb300 as kvz

    q, k, v, pool, slots = _inputs(5, 2, 2, 1, seed=10, fused=False)
    v[0, 0, :4] = torch.tensor([float("inf"), float("-inf"), float("nan"), -0.0])
    st = kvz.new_status()
    kvz.append_tokens(k, v, slots, pool, st)  # no rotation: bit for bit
    at = slots.long()
    assert torch.equal(pool[at // PAGE, :, 0, at % PAGE].view(torch.int16), k.view(torch.int16))
    assert torch.equal(pool[at // PAGE, :, 1, at % PAGE].view(torch.int16), v.view(torch.int16))


def test_one_slot_twice_touches_nothing_else():
    import decode_attention_value_gb300 as kvz

    q, k, v, pool, slots = _inputs(6, 2, 2, 2, seed=11)
    before, st = pool.clone(), kvz.new_status()
    slots[:] = 19
    kvz.append_tokens(k, v, slots, pool, st)
    pool[1, :, :, 3] = before[1, :, :, 3]
    assert torch.equal(pool, before) and int(st.item()) == 0


def test_graph_replay_and_other_streams():
    import decode_attention_value_gb300 as kvz

    q, k, v, pool, slots = _inputs(40, 8, 2, 5, seed=12, fused=False)
    pos = torch.arange(40, device="cuda", dtype=torch.int32)
    table, st, out = _table(kvz, 128), kvz.new_status(), torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = kvz.append_tokens(k, v, slots, pool, st, q=q, rope=table, positions=pos)
    with torch.cuda.stream(side):
        kvz.append_tokens(k, v, slots, pool.clone(), st, q=q, q_out=out, rope=table, positions=pos)
    other = kvz.append_tokens(None, None, None, None, st, q=q, rope=table, positions=pos, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(other, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvz.append_tokens(k, v, slots, pool, st, q=q, q_out=out, rope=table, positions=pos)
    for step in range(3):
        pos += 11 * step
        q.copy_(q.flip(0))
        g.replay()
        assert torch.equal(out, kvz.append_tokens(None, None, None, None, st, q=q, rope=table, positions=pos))
    assert int(st.item()) == 0


def test_binding_refusals():
    import decode_attention_value_gb300 as kvz

    q, k, v, pool, slots = _inputs(4, 4, 2, 2, seed=13, fused=False)
    pos, table, st = torch.arange(4, device="cuda", dtype=torch.int32), _table(kvz, 128), kvz.new_status()
    ok = dict(k=k, v=v, slots=slots, raw_pool=pool, status=st, q=q, rope=table, positions=pos)
    for name, bad in (("k", k.float()), ("k", k[:3]), ("k", k.transpose(1, 2)), ("v", v[:, :1]), ("q", q.half()),
                      ("q", q.cpu()), ("slots", slots.long()), ("slots", slots[:3]), ("raw_pool", pool[:, :1]),
                      ("raw_pool", pool.float()), ("raw_pool", pool.transpose(0, 1)), ("positions", pos.long()),
                      ("positions", pos[:3]), ("positions", None), ("rope", table[:, :1]), ("rope", table.int()),
                      ("slots", None), ("status", st.cpu()), ("q_out", torch.empty_like(q)[:2])):
        with pytest.raises(ValueError):
            kvz.append_tokens(**{**ok, name: bad})
    with pytest.raises(kvz.KvzError):
        kvz.append_tokens(**{**ok, "rope": table[:7]})  # 14 rotated dimensions
    with pytest.raises(kvz.KvzError):
        kvz.append_tokens(**{**ok, "positions": pos.expand(5, 4).contiguous()})
    assert int(st.item()) == 0


@pytest.mark.parametrize("compressed", [True, False])
def test_cache_append_rotates(compressed):
    """The cache classes' append with a rotary table: what one call per layer writes and returns."""
    import decode_attention_value_gb300 as kvz
    from decode_attention_value_gb300.cache import CompressedKVCache, RawKVCache

    L, hkv, hq, n = 3, 2, 8, 4
    cache = CompressedKVCache(L, hkv, n, 4, arena_bytes=64 * 256 * 256, chunk_granules=1024) if compressed else \
        RawKVCache(L, hkv, n, 4, num_slots=3 * n)
    table = _table(kvz, 128)
    slots = [2, 0, 3]
    st = kvz.new_status()
    for step in range(18):  # past one page
        kv = torch.randn((L, 3, hkv, 2, D), device="cuda").to(torch.bfloat16)
        q = torch.randn((L, 3, hq, D), device="cuda").to(torch.bfloat16)
        got = cache.append(slots, kv, q=q, rope=table)
        pos = torch.full((3,), step, device="cuda", dtype=torch.int32)
        for layer in range(L):
            page = torch.zeros((3, hkv, 2, PAGE, D), device="cuda", dtype=torch.bfloat16)
            rows = torch.arange(3, device="cuda", dtype=torch.int32) * PAGE
            want = kvz.append_tokens(kv[layer, :, :, 0], kv[layer, :, :, 1], rows, page, st, q=q[layer], rope=table,
                                     positions=pos)
            assert torch.equal(got[layer], want)
            if step % PAGE != PAGE - 1 or not compressed:
                pages = cache.tails[layer, slots] if compressed else \
                    cache.pool[layer, [cache.pages[s][step // PAGE] for s in slots]]
                assert torch.equal(pages[:, :, :, step % PAGE], page[:, :, :, 0]), step
    assert cache.lens[slots].tolist() == [18] * 3 and int(cache.status.item()) == 0
    with pytest.raises(ValueError):
        cache.append([1, 1], kv[:, :2])


def test_large_calls_are_written_past_the_cache():
    """More than 64 MB of results: 6001 tokens of 56 heads, ragged, with padding and a partial rotation."""
    import decode_attention_value_gb300 as kvz

    T, hq, hkv = 6001, 40, 8
    q, k, v, pool, slots = _inputs(T, hq, hkv, T // PAGE + 4, seed=61)
    slots[5::97] = -1
    pos = torch.randint(0, 131072, (T,), device="cuda", dtype=torch.int32)
    _check(kvz, q, k, v, pool, slots, _table(kvz, 96), pos, 96, False)
