"""append_tokens and the prefix attention calls together, as a decode loop uses them: prompts into
pages, then steps that append every sequence's token and attend behind the shared prompt, eager and
captured into one graph."""
import pytest
import torch

from prefix_case import PAGE, PrefixCase
from test_gpu_append import _angles, _close, _rotated, _table

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, params=[False, True], ids=["narrow", "wide"])
def both_ways(request, monkeypatch):
    """Short prefixes are read with the own tokens; tables wide enough for long ones send them through the
    prefix kernel.  Every test runs both ways."""
    monkeypatch.setattr(PrefixCase, "wide", request.param)


@pytest.mark.parametrize("kind,steps", [("raw", 21), ("coded", 15)])
@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_decode_behind_shared_prompts(kind, steps, graph, dtype):
    import decode_attention_value_gb300 as kvz

    groups, hq, hkv = [(3, 150), (2, 70)], 8, 2
    B = sum(n for n, _ in groups)
    c = PrefixCase(groups, [steps] * B, hq, hkv, seed=31)
    c.pool.fill_(float("nan"))  # only what is appended may be read
    table, g = _table(kvz, 128), torch.Generator(device="cuda").manual_seed(77)
    new = lambda n, h: torch.randn((n, h, 128), generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    for i, (_, P) in enumerate(groups):  # the prompts, from a fused projection's output
        t = torch.arange(P, device="cuda")
        slots = (c.prefix_ids[i][t // PAGE] * PAGE + t % PAGE).to(torch.int32)
        kv = new(P, 2 * hkv)
        kvz.append_tokens(kv[:, :hkv], kv[:, hkv:], slots, c.pool, c.status, rope=table, positions=t.to(torch.int32))
    c.own = [1] * B
    if kind == "coded":
        c.encode()  # (own tokens stay in their raw tail pages: at most 15)
    q, k, v = new(B, hq), new(B, hkv), new(B, hkv)
    slots, pos = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    out = torch.empty(c.q.shape, dtype=dtype, device="cuda")
    ws = torch.empty(kvz.prefix_attention_workspace_size(hkv, B, hq, len(groups), c.pw, c.ow), dtype=torch.uint8, device="cuda")

    def step():
        kvz.append_tokens(k, v, slots, c.pool, c.status, q=q, q_out=c.q, rope=table, positions=pos)
        (c.run_raw if kind == "raw" else c.run_coded)(out=out, workspace=ws)

    base = torch.tensor([P for n, P in groups for _ in range(n)], dtype=torch.int32, device="cuda")
    captured = None
    for s in range(steps):
        for x in (q, k, v):
            x.copy_(new(B, x.shape[1]))
        pos.copy_(base + s)
        slots.copy_(c.page_ids[:, s // PAGE] * PAGE + s % PAGE)
        c.own = [s + 1] * B
        c.seq_lens.fill_(s + 1)
        if graph and captured is None:
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured):
                step()
        captured.replay() if graph else step()
        torch.cuda.synchronize()
        ang = _angles(table, pos)
        _close(c.q, *_rotated(q, ang, 128, False), "q")
        at = c.pool[c.page_ids[:, s // PAGE].long(), :, :, s % PAGE]
        _close(at[:, :, 0], *_rotated(k, ang, 128, False), "k")
        assert torch.equal(at[:, :, 1], v)
        c.check(out, what=f"step {s}")
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("kind", ["raw", "coded"])
def test_no_sequences_no_own_pages_no_groups(kind):
    c = PrefixCase([(3, 40)], [0, 0, 0], 8, 2, seed=32)
    got = c.run_raw() if kind == "raw" else c.run_coded()
    c.check(got)
    import decode_attention_value_gb300 as kvz

    none = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.empty((0, 8, 128), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")
    kvz.prefix_attention_raw(q, none(1), none(0, 4), none(0), none(0, 2), none(0), c.pool, torch.empty_like(q), c.status,
                             workspace=ws)
    kvz.prefix_attention_raw(q, none(1), none(0, 4), none(0), none(0, 2), none(0), c.pool, torch.empty_like(q), c.status)
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("kind", ["raw", "coded"])
@pytest.mark.parametrize("own", [37, 1100])
def test_own_lengths_past_the_table(kind, own):
    """A length that the table cannot name: what it can name is attended to, the rest flagged, at once."""
    c = PrefixCase([(3, 90)], [own, 33, 0], 8, 2, seed=33)
    want = c.reference()
    (c.run_raw if kind == "raw" else c.run_coded)()
    assert int(c.status.item()) == 0
    # (12-bit: a length past the table whose tail has the same tokens)
    width = c.ow if kind == "raw" else c.own_whole.shape[1]
    c.own[0] = width * PAGE + (0 if kind == "raw" else own % PAGE)
    c.seq_lens[0] = c.own[0] + 5 * PAGE
    if kind == "raw" and own % PAGE:
        c.pool[c.page_ids[0, own // PAGE], :, :, own % PAGE:] = 0.5
    want = c.reference()
    got = (c.run_raw if kind == "raw" else c.run_coded)()
    assert int(c.status.item()) == c.kvz.STATUS_BAD_INDEX
    c.check(got, want)
    for far in (2 ** 31 - 1, -3):
        if own > 1024:
            break  # (the split kernel's lengths: as in the plain calls)
        c.status.zero_()
        c.seq_lens[0] = far
        got = (c.run_raw if kind == "raw" else c.run_coded)()
        assert int(c.status.item()) == c.kvz.STATUS_BAD_INDEX
        if far < 0:
            c.own[0] = 0
        elif kind == "coded":
            c.own[0] = width * PAGE + far % PAGE
            continue  # (its tail page's further rows are no tokens: NaN)
        c.check(got, c.reference())
