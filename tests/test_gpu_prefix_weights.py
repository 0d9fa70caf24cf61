"""Weights of fp32 outputs in shared-prefix attention, one by one: all kernels hold all their bits.

K and q have one dimension each, so a score is one exact product; the first token of every page scores 0
and the others -8 to 0, so the maximum is 0 everywhere, every rescaling factor is exactly 1, and the first
token's weight is exactly 1.  V is 1 at dimension t % 128 of token t within a window of 128 tokens and 0
elsewhere, so a sum has one term that is not zero: output d over output d0 of the window's first token is
the weight of token d itself, times one rounding."""
import math

import pytest
import torch

from prefix_case import D, PAGE, PrefixCase

pytestmark = pytest.mark.gpu

# relative to the weight: the score times the constant (rounded itself) is off by 2 * 2^-24 at most, ln 2 of
# that in the weight; exp2 by 2 units in the last place, 2^-22; the product with 1 / sum by 2^-24
BOUND = (2 * math.log(2) + 4 + 1) * 2.0 ** -24  # 3.8e-7; without their third part weights are off by up to 2^-17


def _case(groups, own, hq, hkv, window, seed):
    """window: ("prefix" | "own", first token)."""
    c = PrefixCase(groups, own, hq, hkv, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    c.q.zero_()
    c.q[:, :, 0] = (1 + rand(c.B, hq)).to(torch.bfloat16)
    c.pool.zero_()
    c.pool[:, :, 0, :, 0] = (-3.9 * rand(c.pool.shape[0], hkv, PAGE)).to(torch.bfloat16)
    c.pool[:, :, 0, 0, 0] = 0
    where, first = window
    rows = [(c.prefix_ids[0], groups[0][1])] if where == "prefix" else [(c.page_ids[b], n) for b, n in enumerate(own)]
    for ids, n in rows:
        t = torch.arange(first, max(first, min(n, first + D)), device="cuda")
        if len(t):
            c.pool[ids[t // PAGE].long(), :, 1, t % PAGE, t % D] = 1
    return c


def _weights(c, where, first):
    """[B][hq][128] weights of the window's tokens relative to the maximum's, 0 where there is none (sequences
    behind the group have no prefix)."""
    w = torch.zeros((c.B, c.hq, D), dtype=torch.float64, device="cuda")
    for b in range(c.B if where == "own" else c.groups[0][0]):  # (the sequences of the group)
        ids, n = (c.prefix_ids[0], c.groups[0][1]) if where == "prefix" else (c.page_ids[b], c.own[b])
        t = torch.arange(first, max(first, min(n, first + D)), device="cuda")
        k = c.pool[ids[t // PAGE].long(), :, 0, t % PAGE, 0].double()  # [tokens][hkv]
        s = c.q[b, :, 0].double().view(c.hkv, c.G, 1) * k.T[:, None] / math.sqrt(D)
        w[b, :, t % D] = torch.exp(s).flatten(0, 1)
    return w


ROUTES = {  # tables wide enough for the prefix kernel, groups, own lengths, KV heads, windows
    "one kernel": (False, [(4, 300)], [40, 7, 128, 33], 2, [("prefix", 0), ("prefix", 160), ("own", 0)]),
    "prefix kernel": (True, [(4, 700)], [40, 7, 128, 33], 2, [("prefix", 0), ("prefix", 128), ("prefix", 576), ("own", 0)]),
    "two tiles": (True, [(300, 700)], [17] * 300, 1, [("prefix", 128), ("own", 0)]),
    "many blocks": (True, [(300, 20000)], [3] * 300, 8, [("prefix", 0), ("prefix", 1024), ("prefix", 19840)]),
    "long own tokens": (False, [(3, 200)], [1500, 1030, 16], 2, [("prefix", 64), ("own", 0), ("own", 1024)]),
    "longest beside empty": (True, [(2, 200)], [2100, 0, 1025], 3, [("own", 1008), ("prefix", 0)]),
}


@pytest.mark.parametrize("kind", ["raw", "coded"])
@pytest.mark.parametrize("G", [1, 3, 4, 5, 8])
@pytest.mark.parametrize("route", ROUTES)
def test_every_weight_of_an_fp32_output(monkeypatch, kind, G, route):
    wide, groups, own, hkv, windows = ROUTES[route]
    monkeypatch.setattr(PrefixCase, "wide", wide)
    for i, (where, first) in enumerate(windows):
        c = _case(groups, own, G * hkv, hkv, (where, first), seed=10 * G + i)
        got = (c.run_raw() if kind == "raw" else c.run_coded()).double()
        want = _weights(c, where, first)
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0
        one = got[:, :, first % D][..., None]  # weight 1 over the sum
        have = want.sum(-1) > 0  # rows whose sequence has tokens in the window
        rel = ((got / one - want).abs() / want.clamp(min=1e-3))[have]
        assert rel.numel() and rel.max() <= BOUND, (where, first, rel.max().item())
        assert (got[~have] == 0).all()
        # two BF16 parts of these weights would not do
        w = want[have].float()
        high = w.bfloat16().float()
        two = high.double() + (w - high).bfloat16().double()
        assert ((two - w.double()).abs() / w.double().clamp(min=1e-3)).max() > 6 * BOUND
