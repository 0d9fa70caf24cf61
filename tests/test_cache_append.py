"""What a refused append leaves of a cache: everything as it was."""
import pytest
import torch

L, HKV, HQ = 2, 2, 4


@pytest.fixture(scope="module")
def kvz():
    from decode_attention_value_gb300 import _build

    _build.build()
    import decode_attention_value_gb300 as m

    return m


def _state(c):
    rows = c.pool if hasattr(c, "pool") else c.tails
    return (list(getattr(c, "free", [])), [list(p) for p in getattr(c, "pages", [])], c.lens.tolist(), rows.clone())


def _refused(c, slots, bad, then):
    """Each of `bad`, several times over, is refused and changes nothing; `then` works afterwards."""
    for kw in bad:
        for _ in range(3):
            before = _state(c)
            with pytest.raises((ValueError, RuntimeError)):
                c.append(slots, **kw)
            after = _state(c)
            assert before[:3] == after[:3], list(kw)
            assert torch.equal(before[3].view(torch.int16), after[3].view(torch.int16)), list(kw)
    lens = c.lens.copy()
    c.append(slots, **then)
    assert (c.lens[slots] == lens[slots] + 1).all()
    args = c.batch_args(slots)
    assert args[1].tolist() == c.lens[slots].tolist()


def _kv(n, dev):
    return torch.randn((L, n, HKV, 2, 128), device=dev).to(torch.bfloat16)


def test_refused_appends_take_no_pages(kvz):
    from decode_attention_value_gb300.cache import OutOfSpace, RawKVCache

    c = RawKVCache(L, HKV, 3, 4, num_slots=9, device="cpu")
    c.admit(1, torch.zeros((L, 1, HKV, 2, 16, 128), dtype=torch.bfloat16), 16)  # slots 0, 1 and 2 start a page
    good = dict(kv=_kv(3, "cpu"))
    bad = [dict(kv=_kv(3, "cpu"), rope=kvz.rope_table(torch.ones(64))), dict(kv=_kv(2, "cpu"))]
    _refused(c, [2, 0, 1], bad, good)
    assert c.free_pages() == 5 and [len(p) for p in c.pages] == [1, 2, 1]
    for i, slot in enumerate([2, 0, 1]):
        n = int(c.lens[slot]) - 1
        assert torch.equal(c.pool[:, c.pages[slot][n // 16], :, :, n % 16], good["kv"][:, i])
    assert len({p for own in c.pages for p in own} | set(c.free)) == 9  # no page lost, none held twice
    c.free = c.free[:1]
    c.lens[:] = [16, 32, 16]  # every slot starts a page
    before = _state(c)
    with pytest.raises(OutOfSpace):
        c.append([0, 1], _kv(2, "cpu"))
    assert _state(c)[:3] == before[:3]


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["raw", "compressed"])
def test_refused_appends_on_the_gpu(kvz, name):
    from decode_attention_value_gb300.cache import CompressedKVCache, RawKVCache

    c = RawKVCache(L, HKV, 3, 4, num_slots=9) if name == "raw" else CompressedKVCache(L, HKV, 3, 4, arena_bytes=1 << 24)
    rope = kvz.rope_table(torch.ones(64, dtype=torch.float64)).cuda()
    q = torch.randn((L, 3, HQ, 128), device="cuda").to(torch.bfloat16)
    kv = _kv(3, "cuda")
    bad = [dict(kv=kv, q=q, rope=rope, positions=[1, 2]), dict(kv=kv, q=q.float(), rope=rope),
           dict(kv=kv, q=q[..., :64], rope=rope), dict(kv=kv, rope=rope.int()), dict(kv=_kv(2, "cuda"))]
    _refused(c, [2, 0, 1], bad, dict(kv=kv, q=q, rope=rope))
    assert int(c.status.item()) == 0


def test_slots_counted_from_the_end(kvz):
    from decode_attention_value_gb300.cache import RawKVCache

    c = RawKVCache(L, HKV, 3, 4, num_slots=9, device="cpu")
    kv = _kv(2, "cpu")
    before = _state(c)
    with pytest.raises(ValueError):  # the same slot by both names
        c.append([2, -1], kv)
    with pytest.raises(IndexError):
        c.append([0, 3], kv)
    assert _state(c)[:3] == before[:3]
    c.append([0, -1], kv)
    assert c.lens.tolist() == [1, 0, 1] and torch.equal(c.pool[:, c.pages[2][0], :, :, 0], kv[:, 1])


@pytest.mark.gpu
def test_slots_counted_from_the_end_on_the_gpu(kvz):
    """Also where a page fills: each layer's rows go to the layer's own last tail page."""
    from decode_attention_value_gb300.cache import CompressedKVCache

    a, b = (CompressedKVCache(L, HKV, 3, 4, arena_bytes=1 << 24) for _ in range(2))
    for step in range(17):
        kv = _kv(2, "cuda")
        a.append([1, 2], kv)
        b.append([1, -1], kv)
        assert a.lens.tolist() == b.lens.tolist() == [0, step + 1, step + 1]
        assert torch.equal(a.tails, b.tails), step
    assert torch.equal(a.meta, b.meta) and torch.equal(a.arena, b.arena)
    assert int(a.status.item()) == 0 and int(b.status.item()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["raw", "compressed"])
def test_an_append_copies_to_the_device_once(kvz, monkeypatch, name):
    """A step's host time is its transfers: the rows' places are one, where no page fills."""
    from decode_attention_value_gb300.cache import CompressedKVCache, RawKVCache

    c = RawKVCache(L, HKV, 3, 4, num_slots=9) if name == "raw" else CompressedKVCache(L, HKV, 3, 4, arena_bytes=1 << 24)
    kv = _kv(2, "cuda")
    c.append([0, 2], kv)
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA, torch.profiler.ProfilerActivity.CPU]) as p:
        c.append([0, 2], kv)
        torch.cuda.synchronize()
    copies = [e for e in p.events() if "Memcpy HtoD" in e.name]
    assert len(copies) <= 1, [e.name for e in p.events()]
    assert c.lens.tolist() == [2, 0, 2]
