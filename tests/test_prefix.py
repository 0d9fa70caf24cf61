"""kvz_prefix_attention and kvz_prefix_attention_raw without a GPU: host-side refusals (nothing is
launched) and what the binding refuses."""
import pytest
import torch


@pytest.fixture(scope="module")
def kvz():
    from decode_attention_value_gb300 import _build

    _build.build()
    import decode_attention_value_gb300 as m

    return m


E = dict(inval=-1, unsup=-2, align=-3)
FAKE = 1 << 20  # never dereferenced: every call below returns before any launch


def _raw(kvz, hkv=8, d=128, p=16, B=4, hq=32, q=FAKE, groups=2, start=FAKE, pids=FAKE, pp=3, plens=FAKE, ids=FAKE, op=2,
         lens=FAKE, pool=FAKE, pages=9, out=FAKE, kind=0, ws=FAKE, size=0, status=FAKE):
    return kvz.lib().kvz_prefix_attention_raw(kvz.Dims(hkv, d, p), B, hq, q, groups, start, pids, pp, plens, ids, op, lens,
                                              pool, pages, out, kind, ws, size, status, None)


def _coded(kvz, hkv=8, d=128, p=16, B=4, hq=32, q=FAKE, groups=2, start=FAKE, pids=FAKE, pp=3, plens=FAKE, ptail=FAKE,
           ids=FAKE, op=2, lens=FAKE, tail=FAKE, meta=FAKE, mpages=9, arena=FAKE, abytes=4096, pool=FAKE, pages=9,
           out=FAKE, kind=0, ws=FAKE, size=0, status=FAKE):
    return kvz.lib().kvz_prefix_attention(kvz.Dims(hkv, d, p), B, hq, q, groups, start, pids, pp, plens, ptail, ids, op,
                                          lens, tail, meta, mpages, arena, abytes, pool, pages, out, kind, ws, size, status,
                                          None)


@pytest.mark.parametrize("call", [_raw, _coded])
def test_host_rejects_bad_arguments(kvz, call):
    app = lambda **kw: call(kvz, **kw)  # noqa: E731
    assert app(d=64) == E["unsup"] and app(p=32) == E["unsup"]
    assert app(hkv=0) == E["inval"]
    assert app(B=-1) == E["inval"] and app(hq=0) == E["inval"] and app(hq=31) == E["inval"]
    assert app(hq=72) == E["unsup"]  # nine query heads a KV head
    assert app(groups=-1) == E["inval"] and app(groups=257) == E["unsup"]
    assert app(pp=-1) == E["inval"] and app(op=-1) == E["inval"] and app(pages=-1) == E["inval"]
    assert app(pp=1 << 28) == E["unsup"]
    assert app(kind=2) == E["inval"] and app(kind=-1) == E["inval"]
    for name in ("q", "start", "pids", "plens", "ids", "lens", "out", "ws", "status"):
        assert app(**{name: None}) == E["inval"], name
    for name in ("q", "out"):
        assert app(**{name: FAKE + 8}) == E["align"], name
    for name in ("start", "pids", "plens", "ids", "lens", "status"):
        assert app(**{name: FAKE + 2}) == E["align"], name


def test_host_rejects_bad_coded_arguments(kvz):
    app = lambda **kw: _coded(kvz, **kw)  # noqa: E731
    for name in ("ptail", "tail", "meta", "arena"):
        assert app(**{name: None}) == E["inval"], name
    assert app(mpages=-1) == E["inval"]
    assert app(meta=FAKE + 8) == E["align"] and app(arena=FAKE + 128) == E["align"]
    assert app(ptail=FAKE + 2) == E["align"] and app(tail=FAKE + 1) == E["align"]


@pytest.mark.parametrize("call", [_raw, _coded])
def test_an_empty_batch_is_done_at_once(kvz, call):
    assert call(kvz, B=0, q=None, start=None, pids=None, plens=None, ids=None, lens=None, out=None, ws=None, status=None) == 0


def test_workspace_size_refuses_what_the_call_refuses(kvz):
    size = lambda hkv=8, B=4, hq=32, groups=2, pp=3, op=2: kvz.lib().kvz_prefix_attention_workspace_size(  # noqa: E731
        kvz.Dims(hkv, 128, 16), B, hq, groups, pp, op)
    for bad in (dict(groups=-1), dict(groups=257), dict(pp=-1), dict(hq=31), dict(op=-1), dict(B=-1)):
        assert size(**bad) == 0, bad


def test_binding_rejects_cpu_tensors(kvz):
    q = torch.zeros((2, 8, 128), dtype=torch.bfloat16)
    i = torch.zeros((2,), dtype=torch.int32)
    pool = torch.zeros((3, 2, 2, 16, 128), dtype=torch.bfloat16)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError):
        kvz.prefix_attention_raw(q, i, i.view(1, 2), i[:1], i.view(2, 1), i, pool, torch.empty_like(q), i[:1], workspace=ws)
    with pytest.raises(ValueError):
        kvz.prefix_attention(q, i, i.view(1, 2), i[:1], i[:1], i.view(2, 1), i, i, None, None, pool, torch.empty_like(q), i[:1],
                             workspace=ws)
