"""Calls on a given stream while another one is current and busy."""
import pytest
import torch

from prefix_case import PrefixCase
from test_gpu_append import _table

pytestmark = pytest.mark.gpu


def test_output_of_an_append_is_no_block_of_the_current_streams():
    """A block freed on the current stream, which a kernel there still writes, is not what another
    stream's call writes its queries to."""
    import decode_attention_value_gb300 as kvz

    T, hq = 4096, 16
    s, st = torch.cuda.Stream(), kvz.new_status()
    q = torch.randn((T, hq, 128), device="cuda").to(torch.bfloat16)
    rope = _table(kvz, 128)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    want = kvz.append_tokens(None, None, None, None, st, q=q, rope=rope, positions=pos)
    late = torch.zeros_like(q)
    torch.cuda.synchronize()
    freed = torch.empty_like(q)  # as large as the output
    at = freed.data_ptr()
    kvz.selftest_late_writer(late, freed, 20_000_000)  # 20 ms on the current stream
    del freed
    got = kvz.append_tokens(None, None, None, None, st, q=q, rope=rope, positions=pos, stream=s)
    assert got.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("kind", ["raw", "coded"])
def test_prefix_attention_on_another_stream_makes_its_workspace_there(kind):
    c = PrefixCase([(20, 700)], [30] * 20, 8, 2, seed=71)
    run = c.run_raw if kind == "raw" else c.run_coded
    want = run()
    s, out = torch.cuda.Stream(), torch.empty_like(want)
    torch.cuda.synchronize()
    base = torch.cuda.memory_stats()["reserved_bytes.all.current"]
    for _ in range(20):  # one block of the stream's, used again and again
        run(out=out, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert torch.cuda.memory_stats()["reserved_bytes.all.current"] - base <= 64 << 20
