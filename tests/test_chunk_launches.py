"""Chunk attention and plans as dependent launches and on given streams, without a GPU: the sources' loads, and where a
call's own buffers come from."""
import contextlib
import os
import re
import types

import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_attention_value_gb300", "csrc")


@pytest.mark.parametrize("name", ["chunk.cu", "chunk.cuh", "plan.cu"])
def test_no_read_only_loads(name):
    """What an earlier kernel may still write is read by plain loads, which stay behind the wait for it."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.findall(r"__ldg\s*\(|ld\.global\.nc|__restrict__", code)


@pytest.mark.parametrize("coded", [False, True])
def test_a_chunk_calls_workspace_comes_from_its_stream(monkeypatch, coded):
    from decode_attention_value_gb300 import _build

    _build.build()
    import decode_attention_value_gb300 as kvz

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
    q = torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    pool = torch.zeros((3, 2, 2, 16, 128), dtype=torch.bfloat16)
    meta, arena = torch.zeros((3, 2, 2), dtype=torch.int64), torch.zeros(512, dtype=torch.uint8)
    s = types.SimpleNamespace(cuda_stream=7)
    for stream in (s, None):
        made.clear()
        with pytest.raises(ValueError):  # (host tensors)
            if coded:
                kvz.chunk_attention(q, i, i.view(2, 1), i, i, meta, arena, pool, q, i[:1], window=3, stream=stream)
            else:
                kvz.chunk_attention_raw(q, i, i.view(2, 1), i, pool, q, i[:1], window=3, stream=stream)
        assert made == [stream]
