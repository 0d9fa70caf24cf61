"""Chunk attention where a CTA takes many blocks of one unit: outputs that are folded into partials in memory every few
blocks, a running maximum that rises late, streams that share their rows and those that do not, units finished in
place, cut in two and cut across several CTAs, rows that fill no warp."""
import pytest
import torch

from chunk_case import PAGE, ChunkCase

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
BLOCK, ROWS = 128, 256


def _segments(c):
    """(streams share the rows, blocks, unit finished in place) of every range of a unit that a CTA takes: the units'
    blocks are one line, cut evenly over min(SMs, half of them) CTAs."""
    tile, units = ROWS // c.G, []
    for n, L in c.seqs:
        tiles = []
        for t0 in range(0, n, tile):
            tokens, p0 = min(tile, n - t0), L - n + t0
            hi, lo = max(0, p0 + tokens), max(0, max(p0, 0) - c.window + 1) if c.window else 0
            wb, s = lo // BLOCK, min(c.sinks, hi) if c.window else 0
            tiles.append((tokens * c.G <= 128, max(1, min(wb, -(-s // BLOCK)) + -(-hi // BLOCK) - wb)))
        units += tiles * c.hkv
    W = sum(n for _, n in units)
    C = min(torch.cuda.get_device_properties(0).multi_processor_count, (W + 1) // 2)
    cuts, out, at = [-(-k * W // C) for k in range(C + 1)], [], 0
    for both, n in units:
        inside = [x for x in cuts if at < x < at + n]
        ends = [at, *inside, at + n]
        out += [(both, b - a, not inside) for a, b in zip(ends, ends[1:])]
        at += n
    return out


def _rising(c, last):
    """Keys that grow along each sequence, up to `last` times as large: maxima rise late."""
    scale = torch.ones(c.pool.shape[0], device="cuda")
    for b, (_, L) in enumerate(c.seqs):
        n = -(-L // PAGE)
        if n:
            scale[c.full_ids[b, :n].long()] = torch.linspace(0.05, last, n, device="cuda")
    for pool in (c.pool, c.clean):
        pool[:, :, 0] = (pool[:, :, 0].float() * scale[:, None, None, None]).to(BF16)


def _check(c, names=("raw", "coded")):
    ref = c.reference()
    for dtype in (F32, BF16):
        for name in names:
            out = getattr(c, f"run_{name}")(dtype=dtype)
            torch.cuda.synchronize()
            assert int(c.status.item()) == 0, name
            c.check(out, ref, f"{name} {dtype}")
            assert torch.equal(getattr(c, f"run_{name}")(dtype=dtype), out)


@pytest.mark.parametrize("last", [0.0, 3.0])
@pytest.mark.parametrize("hq,hkv,B", [(16, 4, 96), (4, 4, 110), (40, 8, 60), (8, 1, 160)])
def test_single_tokens_over_many_blocks(hq, hkv, B, last):
    c = ChunkCase([(1, 3001 + 997 * i % 3000) for i in range(B)], hq, hkv, seed=B)
    if last:
        _rising(c, last)
    seg = _segments(c)
    # streams of more than two folds (four blocks each) in units finished in place and in cut ones
    assert all(both for both, _, _ in seg)
    for whole in (True, False):
        assert max(n for _, n, w in seg if w == whole) // 2 > 8
    _check(c)


@pytest.mark.parametrize("last", [0.0, 3.0])
@pytest.mark.parametrize("hq,hkv,seqs", [(16, 4, [(300, 7900), (701, 5000), (1, 6001), (130, 4097)]),
                                         (8, 8, [(300, 4011), (513, 3500), (200, 6000), (256, 2900), (129, 8000)]),
                                         (10, 2, [(500, 8190), (411, 6000), (5, 8000), (300, 3900)]),
                                         (16, 2, [(299, 8190), (411, 6000), (17, 8000), (300, 7001)])])
def test_chunks_over_many_blocks(hq, hkv, seqs, last):
    c = ChunkCase(seqs, hq, hkv, seed=hq + hkv, lead=2, trail=3)
    if last:
        _rising(c, last)
    seg = _segments(c)
    assert max(n for both, n, _ in seg if not both) > 8 and max(n for both, n, _ in seg if both) // 2 > 4
    assert any(n > 8 and not whole and not both for both, n, whole in seg)
    _check(c)


@pytest.mark.parametrize("sinks", [0, 300])
def test_windows_over_many_blocks(sinks):
    c = ChunkCase([(1, 5000 + 61 * i) for i in range(80)] + [(600, 6000)], 16, 4, window=3000, sinks=sinks, seed=sinks)
    _rising(c, 2.0)
    seg = _segments(c)
    assert max(n for both, n, _ in seg if both) // 2 > 8 and max(n for both, n, _ in seg if not both) > 8
    _check(c)


@pytest.mark.parametrize("n,hq", [(1, 8), (40, 64)])
def test_bf16_outputs_folded_after_256_blocks(n, hq):
    """Tables that name the same 64 pages again and again; V is positive, so an output is not small beside the sum of what
    it is made of, and a lost part of it is seen."""
    L, hkv, B = 600 * BLOCK, 8, 20 if n == 1 else 10
    c = ChunkCase([(n, 64 * PAGE)], hq, hkv, seed=n)
    c.seqs, c.width, c.T = [(n, L)] * B, L // PAGE, n * B
    g = torch.Generator(device="cuda").manual_seed(n)
    c.start = [n * b for b in range(B + 1)]
    c.q_start = torch.tensor(c.start, dtype=torch.int32, device="cuda")
    c.seq_lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    c.full_ids = c.page_ids = torch.randint(0, 64, (B, c.width), generator=g, device="cuda", dtype=torch.int32)
    c.q = torch.randn((c.T, hq, 128), generator=g, device="cuda").to(BF16)
    c.clean[:, :, 1] = c.clean[:, :, 1].abs()
    c.pool = c.clean
    seg = _segments(c)
    assert max(m // 2 if both else m for both, m, _ in seg) > 256
    if n > 1:
        assert max(m for both, m, _ in seg if not both) > 256
    _check(c, ("raw",))
