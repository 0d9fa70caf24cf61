"""Group starts and prefix lengths are checked on every route of the prefix attention calls, also where the
prefix table has no page: bad ones are flagged, and no prefix is read."""
import pytest
import torch

from prefix_case import PrefixCase

pytestmark = pytest.mark.gpu


# own tables: one that the kernel of short prefixes takes, one that it does not, long own tokens
@pytest.mark.parametrize("n,own", [(3, [40, 0, 9]), (700, [20] * 700), (700, [0] * 350 + [300] * 350), (3, [1100, 3, 50])])
@pytest.mark.parametrize("kind", ["raw", "coded"])
def test_starts_and_lengths_of_a_table_without_pages(kind, n, own):
    c = PrefixCase([(1, 0), (2, 0)], own, 8, 2, seed=81)
    assert c.prefix_ids.shape[1] == 0
    run = c.run_raw if kind == "raw" else c.run_coded
    ref = c.reference()
    c.check(run(), ref)
    assert int(c.status.item()) == 0
    starts, lens = c.group_start.clone(), c.prefix_lens.clone()

    def flagged(bits):
        got = run()
        torch.cuda.synchronize()
        assert int(c.status.item()) == bits
        c.status.zero_()
        c.check(got, ref)  # no prefix is read: the own tokens alone

    for bad in ([0, 3, 1], [-1, 1, 3], [0, 1, n + 1]):
        c.group_start.copy_(torch.tensor(bad, dtype=torch.int32))
        flagged(c.kvz.STATUS_BAD_ORDER)
        c.group_start.copy_(starts)
    for bad in ([-1, 0], [0, 2 ** 31 - 1], [0, 17]):  # (raw: 17 tokens, no page; 12-bit: more than the tail)
        c.prefix_lens.copy_(torch.tensor(bad, dtype=torch.int32))
        if kind == "coded":
            c.prefix_tail.fill_(-1)
            if max(bad) > 0:  # what the table cannot name is as if it were 15 tokens of a tail page, here none
                flagged(c.kvz.STATUS_BAD_INDEX | c.kvz.STATUS_BAD_TAIL)
                c.prefix_lens.copy_(lens)
                continue
        flagged(c.kvz.STATUS_BAD_INDEX)
        c.prefix_lens.copy_(lens)
    flagged(0)


@pytest.mark.parametrize("kind", ["raw", "coded"])
@pytest.mark.parametrize("n", [1, 33, 161])
def test_rows_that_fill_no_warp_over_many_blocks(monkeypatch, kind, n):
    """The last warp's lanes without a row keep step while the others add to their partials (every eight
    blocks for fp32 outputs; 626 blocks a KV head are at least 16 a CTA)."""
    monkeypatch.setattr(PrefixCase, "wide", True)
    c = PrefixCase([(n, 80003)], [3] * n, 4, 4, seed=82)
    run = c.run_raw if kind == "raw" else c.run_coded
    ref = c.reference()
    first = run()
    c.check(first, ref)
    c.check(run(dtype=torch.bfloat16), ref)
    assert torch.equal(run(), first)
    assert int(c.status.item()) == 0
