"""Weights of chunk attention's BF16 outputs: two BF16 parts each, as in the package's other attention calls.

K and q have one dimension each, so a score is one exact product between -8 and 0, and the first token of every page scores
0: every rescaling factor is exactly 1.  V is 1 and -1 at one dimension for two neighbouring tokens, whose keys are two
neighbouring BF16 values, within a window of 256 tokens, and 0 elsewhere: an output is a small difference of two
weights, and what their parts leave out stands beside its own rounding."""
import pytest
import torch

from chunk_case import D, PAGE, ChunkCase

pytestmark = pytest.mark.gpu

# relative to a weight: its exponent, at most 8 / ln 2 = 11.6, is off by 2 * 2^-24 of itself (the constant's rounding and
# its own), which is 16 * 2^-24 of the weight; exp2 by 2 units in the last place, 2^-22; the product with 1 / sum by 2^-23
BOUND = 22 * 2.0 ** -24


def _case(seqs, hq, hkv, first, seed):
    c = ChunkCase(seqs, hq, hkv, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    c.q.zero_()
    c.q[:, :, 0] = (1 + rand(c.T, hq)).to(torch.bfloat16)
    kv = torch.zeros_like(c.clean)
    low = (-3.9 * rand(c.clean.shape[0], hkv, PAGE // 2)).to(torch.bfloat16)
    kv[:, :, 0, 0::2, 0] = low
    kv[:, :, 0, 1::2, 0] = (low.view(torch.int16) - 1).view(torch.bfloat16)  # the value before it
    kv[:, :, 0, 0, 0] = 0
    for b, (_, L) in enumerate(seqs):
        t = torch.arange(first, max(first, min(L, first + 2 * D)), device="cuda")
        kv[c.full_ids[b, t // PAGE].long(), :, 1, t % PAGE, t // 2 % D] = (1.0 - 2 * (t % 2))[:, None].to(torch.bfloat16)
    c.pool, c.clean = torch.where(c.pool.isnan(), c.pool, kv), kv
    return c


@pytest.mark.parametrize("seqs,first", [([(1, 600)], 256), ([(40, 300), (1, 257)], 0), ([(300, 900)], 512),
                                        ([(5, 1999), (200, 200), (1, 31)], 0)])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (10, 2), (16, 2)])
def test_bf16_outputs_keep_16_bits_of_a_weight(hq, hkv, seqs, first):
    c = _case(seqs, hq, hkv, first, seed=hq + first)
    want, size, _, _ = c.reference()
    longest = max(L for _, L in seqs)

    def tol(part):
        # the sum of up to `longest` fp32 weights, and the output's rounding
        return (1 + 2.0 ** -8) * size * (part + BOUND) + (2.0 ** -8 + (longest + 8) * 2.0 ** -24) * want.abs()

    # one part would not do
    one = torch.zeros_like(want)
    for b, (n, L) in enumerate(seqs):
        j, p = torch.arange(L, device="cuda"), torch.arange(L - n, L, device="cuda")
        kv = c.clean[c.full_ids[b, j // PAGE].long(), :, :, j % PAGE].double()  # [L][hkv][2][128]
        rows = slice(c.start[b], c.start[b] + n)
        s = torch.einsum("thg,kh->thgk", c.q[rows, :, 0].double().unflatten(1, (hkv, -1)), kv[:, :, 0, 0]) / D ** 0.5
        w = torch.exp(s).masked_fill((j[None] > p[:, None])[:, None, None], 0.0)
        o = torch.einsum("thgk,khd->thgd", w.float().bfloat16().double(), kv[:, :, 1]) / w.sum(-1, keepdim=True)
        one[rows] = o.flatten(1, 2)
    assert ((one - want).abs() > 2 * tol(2.0 ** -17)).any()

    for name in ("raw", "coded"):
        got = getattr(c, f"run_{name}")().double()
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0
        over = (got - want).abs() - tol(2.0 ** -17)
        assert (over <= 0).all(), (name, over.max().item(), (over > 0).sum().item())
