"""Chunk attention, step plans and norms without a GPU: host-side refusals, nothing is launched."""
import pytest
import torch


@pytest.fixture(scope="module")
def kvz():
    from decode_attention_value_gb300 import _build

    _build.build()
    import decode_attention_value_gb300 as m

    return m


fake = 1 << 20  # never dereferenced: every call below returns before any launch
INVAL, UNSUP, ALIGN = -1, -2, -3


def test_chunk_attention_refuses(kvz):
    lib = kvz.lib()

    def raw(hkv=8, d=128, T=4, hq=32, q=fake, B=2, start=fake, ids=fake, mp=4, lens=fake, pool=fake, pages=9, window=0,
            sinks=0, out=fake, kind=1, ws=fake, status=fake):
        return lib.kvz_chunk_attention_raw(kvz.Dims(hkv, d, 16), T, hq, q, B, start, ids, mp, lens, pool, pages, window,
                                           sinks, out, kind, ws, 1 << 30, status, None)

    assert raw(d=64) == UNSUP and raw(hkv=0) == INVAL
    assert raw(hq=12) == INVAL and raw(hq=72) == UNSUP and raw(hq=0) == INVAL
    assert raw(T=0, q=None, out=None) == 0 and raw(B=0, start=None) == 0
    for name in ("T", "B", "mp", "pages", "window", "sinks"):
        assert raw(**{name: -1}) == INVAL, name
    assert raw(B=1025) == UNSUP and raw(T=(1 << 24) + 1) == UNSUP and raw(mp=(1 << 26) + 1) == UNSUP
    assert raw(kind=2) == INVAL and raw(kind=-1) == INVAL
    assert raw(pages=1 << 30) == UNSUP
    for name in ("q", "start", "ids", "lens", "pool", "out", "ws", "status"):
        assert raw(**{name: None}) == INVAL, name
    for name in ("q", "pool", "ws"):
        assert raw(**{name: fake + 8}) == ALIGN, name
    assert raw(out=fake + 16) == ALIGN
    for name in ("start", "ids", "lens", "status"):
        assert raw(**{name: fake + 2}) == ALIGN, name


def test_plan_refuses(kvz):
    lib = kvz.lib()

    def plan(B=2, T=4, rows=fake, new=fake, lens=fake, S=3, tables=fake, width=4, free=fake, cap=9, count=fake, start=fake,
             seq=fake, ids=fake, pos=fake, slots=fake, lens_out=fake, free_out=fake, status=fake):
        return lib.kvz_plan_step(B, T, rows, new, lens, S, tables, width, free, cap, count, start, seq, ids, pos, slots,
                                 lens_out, free_out, status, None)

    for name in ("B", "T", "S", "width", "cap"):
        assert plan(**{name: -1}) == INVAL, name
    assert plan(B=1025) == UNSUP and plan(width=(1 << 27)) == UNSUP
    for name in ("rows", "new", "lens", "tables", "free", "count", "start", "seq", "ids", "pos", "slots", "lens_out",
                 "free_out", "status"):
        assert plan(**{name: None}) == INVAL, name
        assert plan(**{name: fake + 2}) == ALIGN, name
    assert lib.kvz_release_pages(0, None, fake, 3, fake, 4, fake, 9, fake, fake, None) == 0
    assert lib.kvz_release_pages(2, None, fake, 3, fake, 4, fake, 9, fake, fake, None) == INVAL
    assert lib.kvz_release_pages(2, fake, fake, 3, fake, 4, fake + 1, 9, fake, fake, None) == ALIGN


def test_bindings_refuse_host_tensors(kvz):
    i = torch.zeros(2, dtype=torch.int32)
    q, pool = torch.zeros((2, 4, 128), dtype=torch.bfloat16), torch.zeros((3, 2, 2, 16, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kvz.chunk_attention_raw(q, i, i.view(2, 1), i, pool, q, i[:1], workspace=i)
    with pytest.raises(ValueError):
        kvz.chunk_attention(q, i, i.view(2, 1), i, i, None, None, pool, q, i[:1])
    with pytest.raises(ValueError):
        kvz.plan_step(i, i, i, i.view(2, 1), i, i[:1], kvz.new_step_plan(2, 4, 1, device="cpu"), i[:1])
    with pytest.raises(ValueError):
        kvz.append_tokens(q, q, i, pool, i[:1], k_norm=i)
