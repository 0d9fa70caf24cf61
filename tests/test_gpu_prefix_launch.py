"""append_tokens and the prefix attention calls are launched while the kernel before them ends: whatever
that kernel still writes (a late writer: it lets its dependents begin, waits, then writes) they must see,
eagerly and in CUDA graphs, also behind copies, fills and joined streams."""
import pytest
import torch

from prefix_case import PrefixCase
from test_gpu_append import _table

pytestmark = pytest.mark.gpu

DELAY_NS = 50_000  # far longer than the kernels' start


@pytest.fixture(autouse=True, params=[False, True], ids=["narrow", "wide"])
def both_ways(request, monkeypatch):
    """Short prefixes are read with the own tokens; tables wide enough for long ones send them through the
    prefix kernel.  Every test runs both ways."""
    monkeypatch.setattr(PrefixCase, "wide", request.param)


@pytest.fixture(scope="module")
def kvz():
    import decode_attention_value_gb300 as m

    return m


def _replayed(step, graph, reset):
    """step() once: called, or captured and replayed twice."""
    if not graph:
        reset()
        torch.cuda.synchronize()
        step()
    else:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        for _ in range(2):
            reset()
            torch.cuda.synchronize()
            g.replay()
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["raw", "coded"])
@pytest.mark.parametrize("groups,own", [([(4, 300), (2, 1000)], [40, 7, 0, 33, 16, 1]), ([(40, 300)], [20] * 40),
                                        ([(2, 90)], [1100, 3, 50]), ([], [40, 0, 9])])
@pytest.mark.parametrize("what", ["q", "seq_lens", "prefix_lens", "pool", "page_ids"])
@pytest.mark.parametrize("graph", [False, True])
def test_prefix_attention_sees_a_late_writer(kvz, kind, groups, own, what, graph):
    c = PrefixCase(groups, own, 8, 2, seed=41)
    run = c.run_raw if kind == "raw" else c.run_coded
    want = run()
    if what == "page_ids" and kind == "coded":
        name = "own_whole"
    else:
        name = what
    live = getattr(c, name)
    bytes_ = live.numel() * live.element_size()
    if bytes_ == 0:
        pytest.skip("nothing to write")
    # the writer moves 16 bytes at a time: a padded copy that the call's tensor is the front of
    pad = (bytes_ + 15) // 16 * 16
    true, late = (torch.zeros(pad, dtype=torch.uint8, device="cuda") for _ in range(2))
    true[:bytes_] = live.contiguous().view(-1).view(torch.uint8)
    setattr(c, name, late[:bytes_].view(live.dtype).view(live.shape))
    out = torch.empty_like(want)
    ws = torch.empty(kvz.prefix_attention_workspace_size(c.hkv, c.B, c.hq, len(groups), c.pw, c.ow), dtype=torch.uint8,
                     device="cuda")

    def step():
        kvz.selftest_late_writer(true, late, DELAY_NS)
        run(out=out, workspace=ws)

    def reset():
        out.fill_(7)
        late.zero_()

    _replayed(step, graph, reset)
    assert torch.equal(out, want)
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("what", ["k", "v", "q", "slots", "positions", "rope"])
def test_append_sees_a_late_writer(kvz, what, graph):
    T, hq, hkv = 300, 8, 2
    g = torch.Generator(device="cuda").manual_seed(5)
    new = lambda h: torch.randn((T, h, 128), generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    a = dict(k=new(hkv), v=new(hkv), q=new(hq), rope=_table(kvz, 128),
             slots=torch.randperm(320, generator=g, device="cuda")[:T].to(torch.int32),
             positions=torch.randint(0, 1 << 20, (T,), generator=g, device="cuda").to(torch.int32))
    pool, st = torch.zeros((20, hkv, 2, 16, 128), dtype=torch.bfloat16, device="cuda"), kvz.new_status()

    def call(a, q_out):
        kvz.append_tokens(a["k"], a["v"], a["slots"], pool, st, q=a["q"], q_out=q_out, rope=a["rope"],
                          positions=a["positions"])

    want_q, got_q = torch.empty_like(a["q"]), torch.empty_like(a["q"])
    call(a, want_q)
    want = pool.clone()
    late = dict(a, **{what: torch.zeros_like(a[what])})

    def step():
        kvz.selftest_late_writer(a[what], late[what], DELAY_NS)
        call(late, got_q)

    def reset():
        pool.zero_()
        got_q.zero_()
        late[what].zero_()

    _replayed(step, graph, reset)
    assert torch.equal(got_q, want_q) and torch.equal(pool, want)
    assert int(st.item()) == 0


def test_captured_behind_copies_fills_and_joined_streams(kvz):
    """A decode step in a graph whose nodes before the calls are a copy, a fill and another stream's work."""
    c = PrefixCase([(3, 200)], [17, 5, 30], 8, 2, seed=43)
    k = torch.randn((3, 2, 128), device="cuda").to(torch.bfloat16)
    q0, q1 = c.q.clone(), torch.zeros_like(c.q)
    slots = torch.tensor([int(c.page_ids[i, n // 16]) * 16 + n % 16 for i, n in enumerate(c.own)], dtype=torch.int32,
                         device="cuda")
    pos = torch.tensor([200 + n for n in c.own], dtype=torch.int32, device="cuda")
    table, out, half = _table(kvz, 128), torch.empty_like(c.q, dtype=torch.float32), torch.empty_like(k)
    ws = torch.empty(kvz.prefix_attention_workspace_size(2, 3, 8, 1, c.pw, c.ow), dtype=torch.uint8, device="cuda")
    before = c.pool.clone()
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            half.copy_(k * 0.5)
        q1.copy_(q0)  # a copy node
        c.seq_lens.add_(1)
        main.wait_stream(side)  # two dependencies
        kvz.append_tokens(half, k, slots, c.pool, c.status, q=q1, q_out=c.q, rope=table, positions=pos)
        out.zero_()  # a fill node
        side.wait_stream(main)
        with torch.cuda.stream(side):
            half.mul_(2)
        main.wait_stream(side)
        c.run_raw(out=out, workspace=ws)

    lens = c.seq_lens.clone()
    step()
    torch.cuda.synchronize()
    c.own = [n + 1 for n in c.own]
    want = out.clone()
    c.check(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        c.pool.copy_(before)
        c.seq_lens.copy_(lens)
        out.fill_(9)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert int(c.status.item()) == 0
