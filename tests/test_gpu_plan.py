"""plan_step and release_pages on the GPU against the same tables worked out on the host, append_tokens with norms
against 64 bits, and a run of all of a chunked step's calls together, eager and captured."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PAGE, D = 16, 128


def _dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _host(rows, new, lens, tables, free, count, width, T):
    lens, tables = lens.copy(), tables.copy()
    start, seq, ids, pos, slots = [0], [], [], [], []
    for r, n in zip(rows, new):
        if r < 0:
            start.append(start[-1]), seq.append(0), ids.append([-1] * width)
            continue
        for t in range(lens[r], lens[r] + n):
            if t % PAGE == 0:
                count -= 1
                tables[r, t // PAGE] = free[count]
            pos.append(t), slots.append(int(tables[r, t // PAGE]) * PAGE + t % PAGE)
        lens[r] += n
        held = -(-lens[r] // PAGE)
        start.append(start[-1] + n), seq.append(lens[r]), ids.append([*tables[r, :held], *[-1] * (width - held)])
    pad = T - len(pos)
    return start, seq, np.array(ids).reshape(-1, width), pos + [0] * pad, slots + [-1] * pad, lens, tables, count


@pytest.mark.parametrize("B,width,most,pad", [(0, 3, 1, 5), (1, 1, 16, 0), (1, 7, 100, 3), (5, 33, 40, 0), (64, 128, 1, 2),
                                              (257, 50, 30, 11), (1024, 20, 9, 0)])
def test_plan_and_release(B, width, most, pad):
    import decode_attention_value_gb300 as kvz

    rng = np.random.default_rng(B + width)
    S = B + 4
    rows = rng.permutation(S)[:B]
    new = rng.integers(0, most + 1, B)
    lens = np.zeros(S, np.int64)
    lens[rows] = rng.integers(0, width * PAGE - most + 1, B)
    tables = np.full((S, width), -1)
    perm, at = rng.permutation(S * width + 50), 0
    for r in rows:
        n = -(-lens[r] // PAGE)
        tables[r, :n], at = perm[at: at + n], at + n
    if B > 3:
        rows[2] = -1  # no request in this place
    free = perm[at:]
    T = int(new[rows >= 0].sum()) + pad
    want = _host(rows, new, lens, tables, free, len(free), width, T)
    d = [_dev(rows), _dev(new), _dev(lens), _dev(tables), _dev(free), _dev([len(free)])]
    status = kvz.new_status()
    for in_place in (False, True):
        out = (None, None) if in_place else (torch.zeros_like(d[2]), torch.zeros_like(d[5]))
        p = kvz.plan_step(*d, kvz.new_step_plan(B, T, width), status, lens_out=out[0], free_out=out[1])
        got = [*p, d[2] if in_place else out[0], d[3], (d[5] if in_place else out[1])]
        for name, a, b in zip(("q_start", "seq_lens", "page_ids", "positions", "slots", "lens", "tables", "free"),
                              (got[0], got[1], got[2], got[3], got[4], got[5], got[6], got[7]), want):
            assert np.array_equal(a.cpu().numpy().reshape(-1), np.asarray(b).reshape(-1)), name
    assert int(status.item()) == 0
    live = rows[rows >= 0]
    back = sum(-(-want[5][r] // PAGE) for r in live)
    if want[7] + back > len(free):  # a free list without room for all pages: refused, nothing changes
        kvz.release_pages(d[0], d[2], d[3], d[4], d[5], status)
        assert int(status.item()) == kvz.STATUS_BAD_INDEX and int(d[5].item()) == want[7]
        assert np.array_equal(d[2].cpu().numpy(), want[5]) and np.array_equal(d[3].cpu().numpy(), want[6])
        status.zero_()
    # all pages come back to one that has
    d[4] = torch.cat([d[4], _dev([-1] * int(back))])
    kvz.release_pages(d[0], d[2], d[3], d[4], d[5], status)
    count = int(d[5].item())
    assert count == want[7] + back and int(status.item()) == 0
    assert sorted(d[4][:count].tolist()) == sorted([*free[:want[7]], *(x for r in live for x in want[6][r] if x >= 0)])
    assert (d[2][_dev(live).long()] == 0).all() and (d[3][_dev(live).long()] == -1).all()


def test_steps_that_cannot_be_taken_change_nothing():
    import decode_attention_value_gb300 as kvz

    base = dict(rows=[1, 0], new=[20, 3], lens=[5, 30, 0], free=[9, 8, 7, 6], count=[4], T=30)
    for change, bit in ((dict(count=[0]), kvz.STATUS_ARENA_FULL), (dict(T=22), kvz.STATUS_BAD_INDEX),
                        (dict(rows=[1, 1]), kvz.STATUS_BAD_ORDER), (dict(rows=[1, 3]), kvz.STATUS_BAD_INDEX),
                        (dict(rows=[-2, 1]), kvz.STATUS_BAD_INDEX), (dict(new=[-1, 3]), kvz.STATUS_BAD_INDEX),
                        (dict(new=[2 ** 31 - 1, 3]), kvz.STATUS_BAD_INDEX), (dict(lens=[5, -1, 0]), kvz.STATUS_BAD_INDEX),
                        (dict(new=[35, 3]), kvz.STATUS_BAD_INDEX), (dict(count=[5]), kvz.STATUS_BAD_INDEX),
                        (dict(count=[-1]), kvz.STATUS_BAD_INDEX)):
        c = {**base, **change}
        tables = _dev([[3, -1, -1, -1], [1, 2, -1, -1], [-1] * 4])
        lens, count, status = _dev(c["lens"]), _dev(c["count"]), kvz.new_status()
        plan = kvz.new_step_plan(2, c["T"], 4)
        for t in plan:
            t.fill_(55)
        before = tables.clone()
        p = kvz.plan_step(_dev(c["rows"]), _dev(c["new"]), lens, tables, _dev(c["free"]), count, plan, status)
        assert int(status.item()) == bit, change
        assert lens.tolist() == c["lens"] and count.tolist() == c["count"] and torch.equal(tables, before), change
        assert not p.q_start.any() and not p.seq_lens.any() and (p.page_ids == -1).all() and (p.slots == -1).all(), change


@pytest.mark.parametrize("rot,interleaved,per_head,dtype", [(128, False, False, torch.bfloat16), (64, True, True, torch.float32),
                                                            (0, False, True, torch.bfloat16), (96, False, False, torch.float32)])
@pytest.mark.parametrize("T", [1, 37, 700])
def test_norms(T, rot, interleaved, per_head, dtype):
    import decode_attention_value_gb300 as kvz

    hq, hkv, eps = 6, 2, 1e-5
    g = torch.Generator(device="cuda").manual_seed(T + rot)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    q, k, v = (rand(T, h, D).mul(3).to(torch.bfloat16) for h in (hq, hkv, hkv))
    q[0, 0] = 0  # a head of zeros stays one
    qw, kw = (rand(*((h, D) if per_head else (D,))).to(dtype) for h in (hq, hkv))
    pool = torch.zeros((T // PAGE + 2, hkv, 2, PAGE, D), dtype=torch.bfloat16, device="cuda")
    slots = torch.randperm(pool.shape[0] * PAGE, generator=g, device="cuda")[:T].to(torch.int32)
    pos = torch.randint(0, 5000, (T,), generator=g, device="cuda", dtype=torch.int32)
    n = rot // 2
    inv = 10000.0 ** (-torch.arange(n, dtype=torch.float64) / max(n, 1))
    table, status = kvz.rope_table(inv).cuda() if rot else None, kvz.new_status()
    ang = torch.outer(pos.double(), inv.cuda())[:, None]

    def turned(x, w):
        y = x.double() * torch.rsqrt(x.double().square().mean(-1, keepdim=True) + eps) * w.double()
        h = y[..., :rot]
        a, b = (h[..., 0::2], h[..., 1::2]) if interleaved else h.chunk(2, -1)
        r, m = (a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()), a.abs() + b.abs()
        join = (lambda u, t: torch.stack([u, t], -1).flatten(-2)) if interleaved else (lambda u, t: torch.cat([u, t], -1))
        return torch.cat([join(*r), y[..., rot:]], -1), torch.cat([join(m, m), y[..., rot:].abs()], -1)

    for qn, kn in ((qw, kw), (qw, None), (None, kw)):
        out = kvz.append_tokens(k, v, slots, pool, status, q=q, rope=table, positions=pos if rot else None,
                                interleaved=interleaved, q_norm=qn, k_norm=kn, norm_eps=eps)
        at = slots.long()
        for name, got, x, w in (("q", out, q, qn), ("k", pool[at // PAGE, :, 0, at % PAGE], k, kn)):
            if w is None:
                continue
            want, size = turned(x, w)
            # one rounding to bf16 (2^-8 of the value at most) of an fp32 value: the norm's sum of 128 squares is off by
            # 19 roundings of 2^-24, half of that after the root, four more for root, quotient and products; rotation 2^-21
            tol = 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * (2.0 ** -21 + 14 * 2.0 ** -24) * size
            assert ((got.double() - want).abs() <= tol).all(), name
        assert torch.equal(pool[at // PAGE, :, 1, at % PAGE], v) and int(status.item()) == 0


def test_a_chunked_step_end_to_end():
    """plan, append with norms, attention, step after step, against attention over the whole sequences in 64 bits."""
    import decode_attention_value_gb300 as kvz

    hq, hkv, width, S = 8, 2, 12, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    lens, tables = _dev([0] * S), torch.full((S, width), -1, dtype=torch.int32, device="cuda")
    free, count, status = torch.randperm(40, device="cuda").to(torch.int32), _dev([40]), kvz.new_status()
    pool = torch.full((40, hkv, 2, PAGE, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    table = kvz.rope_table(10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).cuda()
    w = torch.rand(D, generator=g, device="cuda") + 0.5
    T = 80
    rows, new, plan = _dev([2, 0, 1]), _dev([0, 0, 0]), kvz.new_step_plan(3, T, width)
    q, k, v = (torch.zeros((T, h, D), dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
    out = torch.zeros_like(q)
    ws = torch.empty(kvz.chunk_attention_workspace_size(hkv, T, hq, 3, width), dtype=torch.uint8, device="cuda")
    qr = torch.empty_like(q)

    def step():
        kvz.plan_step(rows, new, lens, tables, free, count, plan, status)
        kvz.append_tokens(k, v, plan.slots, pool, status, q=q, q_out=qr, rope=table, positions=plan.positions, q_norm=w, k_norm=w)
        kvz.chunk_attention_raw(qr, plan.q_start, plan.page_ids, plan.seq_lens, pool, out, status, workspace=ws)

    step()  # an empty one
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    total = [0, 0, 0]
    for i, n in enumerate(([50, 17, 1], [1, 1, 1], [30, 0, 49], [1, 20, 1], [1, 1, 1])):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        new.copy_(_dev(n))
        if i % 2:
            graph.replay()
        else:
            step()
        total = [a + b for a, b in zip(total, n)]
        assert int(status.item()) == 0 and plan.seq_lens.tolist() == total
        for b in range(3):
            L, lo, hi = total[b], int(plan.q_start[b]), int(plan.q_start[b + 1])
            j = torch.arange(L, device="cuda")
            kv = pool[plan.page_ids[b, j // PAGE].long(), :, :, j % PAGE].double()
            p = torch.arange(L - (hi - lo), L, device="cuda")
            for h in range(hq):
                s = qr[lo:hi, h].double() @ kv[:, h // 4, 0].T / math.sqrt(D)
                p_ = torch.softmax(s.masked_fill(j[None] > p[:, None], -math.inf), -1)
                want, size = p_ @ kv[:, h // 4, 1], p_ @ kv[:, h // 4, 1].abs()
                # weights and output rounded to BF16, 2^-8 each; scores in fp32
                assert ((out[lo:hi, h].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1.01 * (2.0 ** -8 + 2.0 ** -14) * size).all()
