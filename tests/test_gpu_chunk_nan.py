"""Queries that are not finite: their own rows become NaN, however the work is cut, and no other row changes a bit."""
import pytest
import torch

from chunk_case import ChunkCase

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("seqs", [[(1, 100)], [(1, 300)], [(1, 3000)], [(5, 2000)], [(300, 900)], [(300, 300)],
                                  [(1, 2000)] * 64, [(1, 6000)] * 40 + [(200, 5000)]])
def test_a_query_that_is_not_finite(seqs, value):
    for hq, hkv in ((8, 2), (8, 8)):
        c = ChunkCase(seqs, hq, hkv, seed=len(seqs))
        clean = c.q
        t, h = c.T * 3 // 4, 5
        for dtype in (torch.bfloat16, torch.float32):
            for name in ("raw", "coded"):
                c.q = clean
                want = getattr(c, f"run_{name}")(dtype=dtype)
                c.q = clean.clone()
                c.q[t, h, 77] = value  # (keys of both signs: an infinite score of each)
                got = getattr(c, f"run_{name}")(dtype=dtype)
                torch.cuda.synchronize()
                assert int(c.status.item()) == 0
                assert got[t, h].isnan().all(), (hq, hkv, dtype, name)
                got[t, h] = want[t, h]
                assert torch.equal(got, want), (hq, hkv, dtype, name)
