"""append_tokens with norms: heads whose squares leave fp32's range, weights at its ends, against 64 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu

PAGE, D = 16, 128
BF16 = torch.bfloat16


def _wanted(x, w, eps, ang=None, interleaved=False, rot=0):
    """(value, what its pairs are made of, their weights) in 64 bits."""
    y = x.double() / torch.sqrt(x.double().square().mean(-1, keepdim=True) + eps) * w.double()
    w = w.double().abs().expand_as(y)
    if not rot:
        return y, y.abs(), w
    h = y[..., :rot]
    a, b = (h[..., 0::2], h[..., 1::2]) if interleaved else h.chunk(2, -1)
    r, m = (a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()), a.abs() + b.abs()
    wa, wb = (w[..., :rot][..., 0::2], w[..., :rot][..., 1::2]) if interleaved else w[..., :rot].chunk(2, -1)
    join = (lambda u, t: torch.stack([u, t], -1).flatten(-2)) if interleaved else (lambda u, t: torch.cat([u, t], -1))
    return (torch.cat([join(*r), y[..., rot:]], -1), torch.cat([join(m, m), y[..., rot:].abs()], -1),
            torch.cat([join(wa + wb, wa + wb), w[..., rot:]], -1))


def _close(got, want, size, weight):
    """One rounding to BF16 (2^-8 of a value at most, 2^-134 below the normal ones) of an fp32 value: the mean of 128 squares
    is off by 20 roundings of 2^-24, half of that after the root, four more for root, quotient and products; the
    rotation by 2^-21.  fp32 values below 2^-126 have steps of 2^-149: x over the root mean square is off by half of one
    before it meets its weight; where x was scaled by 2^-68 first (squares beyond fp32's range: the scaled root mean
    square is 2^-4 at least) that is off by as much before it is divided by 2^-4 or more.  2^-150 + 2^-146, under
    2^-145, times the weights."""
    tol = 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * (2.0 ** -21 + 14 * 2.0 ** -24) * size + 2.0 ** -145 * weight + 2.0 ** -133
    assert torch.isfinite(got).all()
    over = (got.double() - want).abs() - tol
    assert (over <= 0).all(), (over.max().item(), (over > 0).sum().item())


def _heads(T, heads, g):
    """Heads of every magnitude that BF16 has, some with a few large values among small ones."""
    x = torch.randn((T, heads, D), generator=g, device="cuda", dtype=torch.float64)
    k = torch.randint(-133, 126, (T, heads, 1), generator=g, device="cuda").double()
    k[:8, 0, 0] = torch.tensor([-133, -127, -64, -51, 59, 63, 120, 125], device="cuda").double()
    spread = torch.where(torch.rand((T, heads, D), generator=g, device="cuda") < 0.1, 0, -40 * (torch.arange(heads, device="cuda") % 2)[None, :, None])
    x = (x.clamp(-1.9, 1.9) * torch.exp2(k) * torch.exp2(spread.double()))
    return x.to(BF16)


@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-40, 1e-30, 1e-6, 1.0, 1e30, 3e38])
@pytest.mark.parametrize("rot,interleaved,dtype", [(0, False, BF16), (128, False, torch.float32), (64, True, BF16)])
def test_heads_of_every_magnitude(eps, rot, interleaved, dtype):
    import decode_attention_value_gb300 as kvz

    T, hq, hkv = 200, 5, 2
    g = torch.Generator(device="cuda").manual_seed(int(rot + 1000 * eps) % 1000)
    q, k, v = _heads(T, hq, g), _heads(T, hkv, g), _heads(T, hkv, g)
    if eps == 0.0:  # (a head of zeros would be NaN, as the formula says)
        for x in (q, k):
            x[..., 0] = torch.where((x == 0).all(-1), torch.full_like(x[..., 0], 2.0 ** -133), x[..., 0])
    qw, kw = (torch.randn((h, D), generator=g, device="cuda").to(dtype) for h in (hq, hkv))
    qw[1], kw[0] = qw[1] * 2.0 ** 120, kw[0] * 2.0 ** -120
    pool = torch.zeros((T // PAGE + 1, hkv, 2, PAGE, D), dtype=BF16, device="cuda")
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    pos = torch.randint(0, 5000, (T,), generator=g, device="cuda", dtype=torch.int32)
    inv = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(rot // 2, 1))
    table, status = kvz.rope_table(inv).cuda() if rot else None, kvz.new_status()
    ang = torch.outer(pos.double(), inv.cuda())[:, None]
    out = kvz.append_tokens(k, v, slots, pool, status, q=q, rope=table, positions=pos if rot else None,
                            interleaved=interleaved, q_norm=qw, k_norm=kw, norm_eps=eps)
    f32 = float(torch.tensor(eps, dtype=torch.float32))  # what the call takes
    for got, x, w in ((out, q, qw), (pool[slots.long() // PAGE, :, 0, slots.long() % PAGE], k, kw)):
        _close(got, *_wanted(x, w, f32, ang, interleaved, rot))
    assert torch.equal(pool[slots.long() // PAGE, :, 1, slots.long() % PAGE], v) and int(status.item()) == 0


def test_heads_that_are_not_finite():
    import decode_attention_value_gb300 as kvz

    q = torch.ones((6, 1, D), dtype=BF16, device="cuda")
    q[0, 0, 5], q[1, 0, 7], q[2, 0, 9], q[3] = float("nan"), float("inf"), -float("inf"), 0.0
    w, status = torch.ones(D, device="cuda"), kvz.new_status()
    for eps in (0.0, 1e-6):
        out = kvz.append_tokens(None, None, None, None, status, q=q, q_norm=w, norm_eps=eps)
        want = (q.float() / torch.sqrt(q.float().square().mean(-1, keepdim=True) + eps)).to(BF16)
        assert torch.equal(out.isnan(), want.isnan())
        assert torch.equal(out.nan_to_num(7.0)[4:], want.nan_to_num(7.0)[4:])
        assert (out[1:3].nan_to_num(0.0) == 0).all()


@pytest.mark.parametrize("T,hq,hkv", [(1, 1, 1), (5003, 32, 8), (16381, 32, 8), (9001, 5, 5)])
@pytest.mark.parametrize("rot,interleaved,per_head,dtype", [(128, False, True, BF16), (64, True, False, torch.float32)])
def test_many_rows_a_block_and_padding_tokens(T, hq, hkv, rot, interleaved, per_head, dtype):
    """Several passes a block with two rows in flight, results of more than 64 MB written past L2, rows without a slot
    among the eight-lane groups of a warp; either operand normed alone too."""
    import decode_attention_value_gb300 as kvz

    g = torch.Generator(device="cuda").manual_seed(T)
    qkv = (torch.randn((T, hq + 2 * hkv, D), generator=g, device="cuda") * 3).to(BF16)
    q, k, v = qkv.split((hq, hkv, hkv), 1)
    qw, kw = (torch.randn(((h, D) if per_head else (D,)), generator=g, device="cuda").to(dtype) for h in (hq, hkv))
    pages = T // PAGE + 3
    slots = torch.randperm(pages * PAGE, generator=g, device="cuda")[:T].to(torch.int32)
    if T > 1:
        slots[torch.rand(T, generator=g, device="cuda") < 0.05] = -1
    live = slots >= 0
    at = slots[live].long()
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda", dtype=torch.int32)
    inv = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
    table, status, ang = kvz.rope_table(inv).cuda(), kvz.new_status(), torch.outer(pos.double(), inv.cuda())[:, None]
    for qn, kn in ((qw, kw), (qw, None), (None, kw)):
        pool = torch.full((pages, hkv, 2, PAGE, D), 77.0, dtype=BF16, device="cuda")
        out = kvz.append_tokens(k, v, slots, pool, status, q=q, rope=table, positions=pos, interleaved=interleaved, q_norm=qn,
                                k_norm=kn)
        if qn is not None:
            _close(out, *_wanted(q, qn, float(torch.tensor(1e-6)), ang, interleaved, rot))
        if kn is not None:
            want = _wanted(k, kn, float(torch.tensor(1e-6)), ang, interleaved, rot)
            _close(pool[at // PAGE, :, 0, at % PAGE], *(x[live] if x.shape[0] == T else x for x in want))
        # an operand without a norm is what the call without norms gives
        bare = torch.full_like(pool, 77.0)
        ref = kvz.append_tokens(k, v, slots, bare, status, q=q, rope=table, positions=pos, interleaved=interleaved)
        if qn is None:
            assert torch.equal(out, ref)
        if kn is None:
            assert torch.equal(pool, bare)
        assert torch.equal(pool[:, :, 1], bare[:, :, 1]) and int(status.item()) == 0
        rows = torch.zeros(pages * PAGE, dtype=torch.bool, device="cuda")
        rows[at] = True
        assert (pool.permute(0, 3, 1, 2, 4).reshape(pages * PAGE, hkv, 2, D)[~rows] == 77.0).all()
