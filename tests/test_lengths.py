"""Sequence lengths that the tables cannot name, up to the ends of int32, in every attention call: what the
table names is attended to, the rest flagged, and nothing outside the workspace and the output is written.

In 32 bits a length of 2^31 - 1 has a negative count of pages (2^31 + 14 wraps), and sums of such counts wrap
too; sequences and KV heads found from them are out of range."""
import pytest
import torch

from prefix_case import PAGE, PrefixCase

FAR = [2 ** 31 - 1, 2 ** 31 - 16, 2 ** 30 + 16 * 7 + 15, -1, -2 ** 31]


def test_tables_of_2_31_pages_are_refused():
    from decode_attention_value_gb300 import _build

    _build.build()
    import decode_attention_value_gb300 as kvz

    fake = 1 << 20  # never dereferenced

    def raw(B, pages):
        return kvz.lib().kvz_decode_attention_raw(kvz.Dims(8, 128, 16), B, 32, fake, fake, pages, fake, fake, 9, fake, fake, 0,
                                                  fake, None)

    def coded(B, pages):
        return kvz.lib().kvz_decode_attention(kvz.Dims(8, 128, 16), B, 32, fake, fake, pages, fake, fake, fake, 9, fake, 4096,
                                              fake, 9, fake, fake, 0, fake, None)

    def prefix(B, pages):
        return kvz.lib().kvz_prefix_attention_raw(kvz.Dims(8, 128, 16), B, 32, fake, 1, fake, fake, 1, fake, fake, pages, fake,
                                                  fake, 9, fake, 0, fake, 0, fake, None)

    for call in (raw, coded, prefix):
        assert call(1024, 1 << 21) == -2 and call(2, (1 << 30) - 1) == -2 and call(1, 1 << 27) == -2
        assert call(1024, (1 << 21) - 2) != -2  # (not the table's size: refused later, without a workspace or a GPU)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["raw", "coded"])
@pytest.mark.parametrize("op", ["decode", "overlapped", "prefix"])
@pytest.mark.parametrize("pages", [3, 69])  # own tables of both routes of the prefix calls
@pytest.mark.parametrize("G", [4, 5])
@pytest.mark.parametrize("n", [3, 60])
def test_lengths_at_the_ends_of_int32(kind, op, pages, G, n):
    tail = kind == "coded"
    most = pages * PAGE + (15 if tail else 0)
    own = [(i * 389 + 11) % (most + 1) for i in range(n)]
    far = {i: FAR[i % len(FAR)] for i in range(0, n, 2)}
    for i, L in far.items():  # what the table names of it
        own[i] = 0 if L < 0 else pages * PAGE + (L % PAGE if tail else 0)
    own[1] = most  # (as wide a table in every case)
    c = PrefixCase([(2, 90)], own, 2 * G, 2, seed=91)
    kvz = c.kvz
    if tail:
        c.encode()
    table = c.own_whole if tail else c.page_ids
    assert table.shape[1] == pages
    flags = kvz.ATTN_OVERLAP_PREVIOUS if op == "overlapped" else 0
    size = kvz.prefix_attention_workspace_size(2, n, 2 * G, 1, c.pw, pages) if op == "prefix" else \
        kvz.attention_workspace_size(2, n, 2 * G, pages + tail)
    whole = torch.empty(size + (2 << 20), dtype=torch.uint8, device="cuda")
    ws = whole[1 << 20:][:size]

    def run():
        whole.fill_(0xA5)
        outs = torch.full((n + 64, 2 * G, 128), 3.0, device="cuda")
        out = outs[32: 32 + n]
        if op == "prefix":
            (c.run_coded if tail else c.run_raw)(out=out, workspace=ws)
        elif tail:
            kvz.decode_attention(c.q, table, c.seq_lens, c.tail_page, c.meta, c.arena, c.pool, out, c.status, workspace=ws,
                                 flags=flags)
        else:
            kvz.decode_attention_raw(c.q, table, c.seq_lens, c.pool, out, c.status, workspace=ws, flags=flags)
        torch.cuda.synchronize()
        assert (outs[:32] == 3).all() and (outs[32 + n:] == 3).all()
        assert (whole[: 1 << 20] == 0xA5).all() and (whole[(1 << 20) + size:] == 0xA5).all()
        return out.clone()

    want = run()
    c.check(want, c.reference(prefix=op == "prefix"))
    assert int(c.status.item()) == 0
    c.seq_lens.copy_(torch.tensor([far.get(i, L) for i, L in enumerate(own)], dtype=torch.int32))
    assert torch.equal(run(), want)
    assert int(c.status.item()) == kvz.STATUS_BAD_INDEX
