"""Buffers that a call on a given stream makes for itself come from that stream (no GPU: the allocations
are watched, and the calls end at the host's checks)."""
import contextlib
import types

import pytest
import torch


@pytest.fixture(scope="module")
def kvz():
    from decode_attention_value_gb300 import _build

    _build.build()
    import decode_attention_value_gb300 as m

    return m


def _calls(kvz):
    q = torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    t = i.view(2, 1)
    pool = torch.zeros((3, 2, 2, 16, 128), dtype=torch.bfloat16)
    meta, arena = torch.zeros((3, 2, 2), dtype=torch.int64), torch.zeros(512, dtype=torch.uint8)
    m32, bases, out, st = meta.int(), torch.zeros((2, 2, 2, 128), dtype=torch.uint8), q.float(), i[:1]
    return {
        "append_tokens": lambda **k: kvz.append_tokens(q[:, :2], q[:, 2:], i, pool, st, q=q, **k),
        "prefix_attention": lambda **k: kvz.prefix_attention(q, i, t[:1], i[:1], i[:1], t, i, i, meta, arena, pool, out, st, **k),
        "prefix_attention_raw": lambda **k: kvz.prefix_attention_raw(q, i, t[:1], i[:1], t, i, pool, out, st, **k),
        "decode_attention": lambda **k: kvz.decode_attention(q, t, i, i, meta, arena, pool, out, st, **k),
        "decode_attention_raw": lambda **k: kvz.decode_attention_raw(q, t, i, pool, out, st, **k),
        "ga_decode_attention": lambda **k: kvz.ga_decode_attention(q, t, i, i, m32, arena, bases, pool, out, st, **k),
        "f8_decode_attention": lambda **k: kvz.f8_decode_attention(0, q, t, i, i, m32, arena, bases, pool, out, st, **k),
        "encode_pages": lambda **k: kvz.encode_pages(pool, i, i, i, meta, arena, t, st, **k),
        "encode_sizes": lambda **k: kvz.encode_sizes(pool, i, i, st, **k),
        "ga_encode_pages": lambda **k: kvz.ga_encode_pages(pool, bases, i, i, i, m32, arena, t, st, **k),
        "f8_encode_pages": lambda **k: kvz.f8_encode_pages(0, pool, bases, i, i, i, m32, arena, t, st, **k),
    }


@pytest.mark.parametrize("name", ["append_tokens", "prefix_attention", "prefix_attention_raw", "decode_attention",
                                  "decode_attention_raw", "ga_decode_attention", "f8_decode_attention", "encode_pages",
                                  "encode_sizes", "ga_encode_pages", "f8_encode_pages"])
def test_a_calls_own_buffers_come_from_its_stream(kvz, monkeypatch, name):
    call = _calls(kvz)[name]
    current, made, real = [None], [], torch.empty

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def empty(*a, **k):
        made.append(current[-1])
        return real(*a, **k)

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(kvz, "attention_workspace_size", lambda *a: 64)
    monkeypatch.setattr(kvz, "encode_workspace_size", lambda *a: 64)
    stream = types.SimpleNamespace(cuda_stream=1 << 20)
    for given in (None, stream):
        made.clear()
        with pytest.raises(ValueError):  # tensors on the host
            call(**({} if given is None else {"stream": given}))
        assert made == [given]
    assert current == [None]
