"""The workspace of chunk attention over 12-bit pages: as large as what the step's tokens see, not as the table is wide;
pages beyond its room are left out and flagged; nothing behind it is written."""
import random

import pytest
import torch

from chunk_case import PAGE, ChunkCase

pytestmark = pytest.mark.gpu

PAGE_BYTES = 2 * PAGE * 128 * 2  # of a KV head


def _seen(c):
    """Pages that new tokens see, by sequence: keys from the first new token's window on, and the first tokens."""
    out = []
    for n, L in c.seqs:
        first = max(max(L - n, 0) - c.window + 1, 0) // PAGE if c.window else 0
        out.append([p for p in range(-(-L // PAGE)) if n and (p >= first or (c.window and p * PAGE < c.sinks))])
    return out


def _size(c, **kw):
    return c.kvz.chunk_attention_workspace_size(c.hkv, c.T, c.hq, len(c.seqs), c.whole.shape[1], coded=True, **kw)


def test_sizes():
    import decode_attention_value_gb300 as kvz

    size = lambda *a, **kw: kvz.chunk_attention_workspace_size(*a, coded=True, **kw)  # noqa: E731
    fixed = lambda h, t, q, b, p: size(h, t, q, b, p, seen_pages=0)  # noqa: E731
    for h, t, q, b, p in ((8, 64, 64, 64, 2047), (8, 256, 64, 256, 2047), (1, 5000, 8, 3, 100), (4, 1, 4, 1024, 9), (2, 1, 2, 1, 0)):
        assert size(h, t, q, b, p) - fixed(h, t, q, b, p) == b * (p + 1) * h * PAGE_BYTES
        assert size(h, t, q, b, p, seen_pages=7) - fixed(h, t, q, b, p) == min(7, b * (p + 1)) * h * PAGE_BYTES
        assert size(h, t, q, b, p, seen_pages=10 ** 15) == size(h, t, q, b, p)
        assert size(h, t, q, b, p, window=10 ** 12, sinks=10 ** 12) == size(h, t, q, b, p)
        # the table's entries, 4 bytes a page and KV head, and partial results of the device's SMs
        assert fixed(h, t, q, b, p) < (64 << 20) + 4 * b * (p + 1) * h + 4096
    # 64 single tokens behind windows of 4096 in tables of 2047 pages: 257 or 258 pages each, and those of 64 first tokens
    assert size(8, 64, 64, 64, 2047, window=4096, sinks=64) - fixed(8, 64, 64, 64, 2047) <= 64 * (258 + 4 + 1) * 8 * PAGE_BYTES


def _fuzz(rng):
    B = rng.choice((1, 3, 40, 129, 300))
    seqs = [(rng.choice((0, 1, 1, rng.randint(1, 90))), rng.randint(0, rng.choice((40, 700, 2500)))) for _ in range(B)]
    window = rng.choice((0, 1, 15, 16, 17, rng.randint(1, 600)))
    hkv = rng.choice((1, 2))
    return seqs, hkv * rng.choice((1, 4)), hkv, window, rng.choice((0, 1, 16, 33, 900)) if window else 0


@pytest.mark.parametrize("seed", range(12))
def test_room_for_what_is_seen_is_enough_and_never_left(seed):
    rng = random.Random(seed)
    seqs, hq, hkv, window, sinks = _fuzz(rng)
    if not any(n for n, _ in seqs):
        seqs[0] = (1, seqs[0][1])
    c = ChunkCase(seqs, hq, hkv, window=window, sinks=sinks, seed=seed, wide=rng.choice((0, 3, 500)))
    c.encode()
    want, n = c.run_coded(workspace=torch.empty(_size(c), dtype=torch.uint8, device="cuda")), sum(map(len, _seen(c)))
    c.check(want)
    assert _size(c, window=window, sinks=sinks) >= _size(c, seen_pages=n)
    for size in (_size(c, window=window, sinks=sinks), _size(c, window=window, sinks=sinks, seen_pages=n)):
        for off in (0, 16, 240):
            buf = torch.full((size + off + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
            out = c.run_coded(workspace=buf[off: off + size])
            torch.cuda.synchronize()
            assert int(c.status.item()) == 0
            assert torch.equal(out, want)
            assert (buf[:off] == 0xA5).all() and (buf[off + size:] == 0xA5).all()
    assert torch.equal(c.run_coded(), want)  # a workspace of the call's own


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 40)])
def test_pages_beyond_the_room_are_left_out_and_flagged(window, sinks):
    import decode_attention_value_gb300 as kvz

    c = ChunkCase([(20, 300), (0, 90), (1, 217), (3, 400)], 8, 2, window=window, sinks=sinks, seed=3, wide=40)
    c.encode()
    seen = _seen(c)
    order = [(b, p) for b, pages in enumerate(seen) for p in pages]
    for room in (0, 1, len(seen[0]), len(order) - 5, len(order) - 1, len(order)):
        ref = c.reference(order[room:])
        for dtype in (torch.float32, torch.bfloat16):
            c.status.zero_()
            buf = torch.full((_size(c, seen_pages=room) + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
            out = c.run_coded(dtype=dtype, workspace=buf[:-4096])
            torch.cuda.synchronize()
            assert int(c.status.item()) == (0 if room == len(order) else kvz.STATUS_ARENA_FULL), room
            c.check(out, ref, f"room for {room}")
            assert (buf[-4096:] == 0xA5).all()
    with pytest.raises(kvz.KvzError):  # not even the parts that hold no page
        c.run_coded(workspace=torch.empty(_size(c, seen_pages=0) - 512, dtype=torch.uint8, device="cuda"))


def test_a_wide_table_costs_what_is_seen():
    """64 sequences in tables of 2047 pages with 8 KV heads: the call's own workspace was 8.6 GB."""
    c = ChunkCase([(1, 2000 + i) for i in range(64)], 64, 8, window=512, sinks=16, seed=5)
    c.encode()
    want = c.run_coded()
    narrow = c.whole
    c.whole = torch.full((64, 2047), -1, dtype=torch.int32, device="cuda")
    c.whole[:, : narrow.shape[1]] = narrow
    torch.cuda.empty_cache()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    out = c.run_coded()
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() - before < 400 << 20
    assert torch.equal(out, want) and int(c.status.item()) == 0


def test_window_and_sinks_that_are_no_numbers_are_refused():
    c = ChunkCase([(1, 50)], 2, 1)
    c.encode()
    for bad in (1.5, None, "9"):
        for run in (c.run_raw, c.run_coded):
            c.window = bad
            with pytest.raises(ValueError):
                run()
            c.window = -1
            with pytest.raises(ValueError):
                run()
            c.window = 0
