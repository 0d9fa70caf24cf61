"""Workspaces of the prefix attention calls: any 16-byte aligned one of the stated size, whatever stands
around it, on every route (one kernel, the prefix kernel, long own tokens)."""
import pytest
import torch

from prefix_case import PrefixCase

pytestmark = pytest.mark.gpu

ROUTES = {"one-kernel": (False, [(4, 300)], [40, 7, 0, 33]), "prefix-kernel": (True, [(4, 300), (2, 0)], [40, 7, 0, 33, 9, 1]),
          "two-tiles": (True, [(70, 700)], [20] * 70), "long-own": (False, [(3, 200)], [1100, 0, 50])}


@pytest.mark.parametrize("kind", ["raw", "coded"])
@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_workspace_on_any_16_bytes(monkeypatch, kind, route, dtype):
    wide, groups, own = ROUTES[route]
    monkeypatch.setattr(PrefixCase, "wide", wide)
    c = PrefixCase(groups, own, 8, 2, seed=61)
    run = c.run_raw if kind == "raw" else c.run_coded
    want = run(dtype=dtype)
    size = c.kvz.prefix_attention_workspace_size(c.hkv, c.B, c.hq, len(groups), c.pw, c.ow)
    whole = torch.empty(size + 256, dtype=torch.uint8, device="cuda")
    assert whole.data_ptr() % 256 == 0
    for at in (0, 16, 32, 48, 112):
        whole.fill_(0xA5)
        got = run(dtype=dtype, workspace=whole[at: at + size])
        assert torch.equal(got, want), at
        assert bool((whole[:at] == 0xA5).all()) and bool((whole[at + size:] == 0xA5).all()), at
    with pytest.raises(c.kvz.KvzError):
        run(dtype=dtype, workspace=whole[8: 8 + size])
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("groups,own", [([(4, 300)], [40, 7, 0, 33]), ([(3, 200)], [1100, 0, 50])])
def test_the_size_is_needed_on_an_odd_16_bytes(groups, own):
    c = PrefixCase(groups, own, 8, 2, seed=62)
    call = lambda ws: c.kvz.lib().kvz_prefix_attention_raw(  # noqa: E731
        c.kvz.Dims(2, 128, 16), c.B, 8, c.q.data_ptr(), 1, c.group_start.data_ptr(), c.prefix_ids.data_ptr(), c.pw,
        c.prefix_lens.data_ptr(), c.page_ids.data_ptr(), c.ow, c.seq_lens.data_ptr(), c.pool.data_ptr(), c.pool.shape[0],
        out.data_ptr(), 0, ws.data_ptr(), ws.numel(), c.status.data_ptr(), torch.cuda.current_stream().cuda_stream)
    out = torch.empty(c.q.shape, dtype=torch.float32, device="cuda")
    size = c.kvz.lib().kvz_prefix_attention_workspace_size(c.kvz.Dims(2, 128, 16), c.B, 8, 1, c.pw, c.ow)
    whole = torch.empty(size + 64, dtype=torch.uint8, device="cuda")
    assert call(whole[16: 16 + size]) == 0 and call(whole[:size]) == 0
    assert call(whole[16: 15 + size]) != 0  # one byte less: refused, nothing launched
    assert call(whole[16: 16 + size]) == 0
    c.check(out)
