"""plan_step, release_pages, append_tokens with norms and chunk attention are launched while the kernel before them ends:
whatever that kernel still writes (a late writer: it lets its dependents begin, waits, then writes) they must see, eagerly
and in CUDA graphs, on the current stream and on others."""
import pytest
import torch

from chunk_case import ChunkCase
from test_gpu_append import _table

pytestmark = pytest.mark.gpu

DELAY_NS = 50_000  # far longer than the kernels' start
PAGE, D = 16, 128


def _dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _late(live):
    """The writer moves 16 bytes at a time: (true bytes, late ones, a tensor like live that is the front of these)."""
    n = live.numel() * live.element_size()
    true, late = (torch.zeros((n + 15) // 16 * 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    true[:n] = live.contiguous().view(-1).view(torch.uint8)
    return true, late, late[:n].view(live.dtype).view(live.shape)


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


@pytest.mark.parametrize("seqs", [[(1, 300)], [(1, 3000)] * 40, [(200, 900), (1, 70), (5, 400)]])
@pytest.mark.parametrize("what", ["q", "q_start", "seq_lens", "page_ids", "pool", "tail_page", "meta", "arena"])
@pytest.mark.parametrize("graph", [False, True])
def test_chunk_attention_sees_a_late_writer(seqs, what, graph):
    c = ChunkCase(seqs, 8, 2, window=500, sinks=20, seed=41)
    for kind in ("raw", "coded"):
        if kind == "raw" and what in ("tail_page", "meta", "arena"):
            continue
        c.encode()
        run = c.run_raw if kind == "raw" else c.run_coded
        want = run()
        name = "whole" if what == "page_ids" and kind == "coded" else what
        kept = getattr(c, name)
        true, late, view = _late(kept)
        size = c.kvz.chunk_attention_workspace_size(c.hkv, c.T, c.hq, len(seqs), c.width, coded=True)
        ws, out = torch.empty(size, dtype=torch.uint8, device="cuda"), torch.empty_like(want)
        setattr(c, name, view)

        def step():
            c.kvz.selftest_late_writer(true, late, DELAY_NS)
            run(out=out, workspace=ws)

        def reset():
            out.fill_(77)
            late.zero_()

        _replayed(step, graph, reset)
        setattr(c, name, kept)
        assert torch.equal(out, want) and int(c.status.item()) == 0


def _plan_inputs():
    g = torch.Generator().manual_seed(3)
    B, S, width = 40, 50, 30
    lens = torch.randint(0, 300, (S,), generator=g)
    perm = torch.randperm(S * width + 800, generator=g)
    tables = torch.where(torch.arange(width)[None] < (-(-lens // PAGE))[:, None], perm[: S * width].view(S, width), -1)
    return dict(rows=torch.randperm(S, generator=g)[:B], new=torch.randint(1, 80, (B,), generator=g), lens=lens,
                tables=tables, free=perm[S * width:], count=torch.tensor([800])), B, width


@pytest.mark.parametrize("what", ["rows", "new", "lens", "tables", "free", "count"])
@pytest.mark.parametrize("graph", [False, True])
def test_plans_and_releases_see_a_late_writer(what, graph):
    import decode_attention_value_gb300 as kvz

    host, B, width = _plan_inputs()
    T = int(host["new"].sum()) + 5
    status = kvz.new_status()

    def plan(d, p):
        kvz.plan_step(d["rows"], d["new"], d["lens"], d["tables"], d["free"], d["count"], p, status)
        return [*p, d["lens"], d["tables"], d["count"]]

    def release(d, p):
        kvz.release_pages(d["rows"], d["lens"], d["tables"], d["free"], d["count"], status)
        return [d["lens"], d["tables"], d["free"], d["count"]]

    for call in (plan, release):
        if call is release:
            if what == "new":
                continue
            host = {**host, "free": torch.cat([host["free"], torch.full((2000,), -1)])}  # room for what comes back
        start = {k: _dev(v.tolist()) for k, v in host.items()}
        want = [x.clone() for x in call({k: v.clone() for k, v in start.items()}, kvz.new_step_plan(B, T, width))]
        d, p = {k: v.clone() for k, v in start.items()}, kvz.new_step_plan(B, T, width)
        true, late, d[what] = _late(start[what])
        outs = []

        def step():
            kvz.selftest_late_writer(true, late, DELAY_NS)
            outs[:] = call(d, p)

        def reset():
            for k in d:
                d[k].copy_(start[k]) if k != what else late.zero_()
            for t in p:
                t.fill_(55)

        _replayed(step, graph, reset)
        assert int(status.item()) == 0
        for i, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), (call.__name__, i)


@pytest.mark.parametrize("what", ["q", "k", "qw", "kw", "slots"])
@pytest.mark.parametrize("graph", [False, True])
def test_norms_see_a_late_writer(what, graph):
    import decode_attention_value_gb300 as kvz

    T, hq, hkv = 300, 8, 2
    g = torch.Generator(device="cuda").manual_seed(5)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    a = dict(q=new(T, hq, D), k=new(T, hkv, D), qw=new(hq, D), kw=new(D),
             slots=torch.randperm(320, generator=g, device="cuda")[:T].to(torch.int32))
    v, rope, pos = new(T, hkv, D), _table(kvz, 128), torch.arange(T, device="cuda", dtype=torch.int32)
    pool, st = torch.zeros((20, hkv, 2, PAGE, D), dtype=torch.bfloat16, device="cuda"), kvz.new_status()

    def call(a, out):
        kvz.append_tokens(a["k"], v, a["slots"], pool, st, q=a["q"], q_out=out, rope=rope, positions=pos, q_norm=a["qw"],
                          k_norm=a["kw"])

    want_q, got_q = torch.empty_like(a["q"]), torch.empty_like(a["q"])
    call(a, want_q)
    want = pool.clone()
    true, late, view = _late(a[what])
    b = dict(a, **{what: view})

    def step():
        kvz.selftest_late_writer(true, late, DELAY_NS)
        call(b, got_q)

    def reset():
        pool.zero_()
        got_q.zero_()
        late.zero_()

    _replayed(step, graph, reset)
    assert torch.equal(got_q, want_q) and torch.equal(pool, want) and int(st.item()) == 0


def test_a_step_on_another_stream_behind_its_writer():
    """plan, append and attention on a stream that is given, behind 5 ms of that stream's own work, with the current
    stream idle; the attention's workspace is the stream's."""
    import decode_attention_value_gb300 as kvz

    hq, hkv, width, T, B = 8, 2, 30, 200, 3
    g = torch.Generator(device="cuda").manual_seed(6)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v, w = new(T, hq, D), new(T, hkv, D), new(T, hkv, D), new(D)
    rope, rows, counts = _table(kvz, 128), _dev([2, 0, 1]), _dev([150, 1, 49])
    s = torch.cuda.Stream()

    def step(stream, counts):
        lens, tables = _dev([40, 16, 0]), _dev([[90, 91, 92] + [-1] * 27, [93] + [-1] * 29, [-1] * 30])
        free, count, st = torch.arange(80, dtype=torch.int32, device="cuda"), _dev([80]), kvz.new_status()
        pool = torch.ones((100, hkv, 2, PAGE, D), dtype=torch.bfloat16, device="cuda")
        plan, out, qr = kvz.new_step_plan(B, T, width), torch.zeros_like(q), torch.empty_like(q)
        torch.cuda.synchronize()
        if stream is not None:
            kvz.selftest_late_writer(*late, 5_000_000, stream=stream)
        kvz.plan_step(rows, counts, lens, tables, free, count, plan, st, stream=stream)
        kvz.append_tokens(k, v, plan.slots, pool, st, q=q, q_out=qr, rope=rope, positions=plan.positions, q_norm=w, k_norm=w,
                          stream=stream)
        kvz.chunk_attention_raw(qr, plan.q_start, plan.page_ids, plan.seq_lens, pool, out, st, stream=stream)
        kvz.release_pages(rows[:2], lens, tables, free, count, st, stream=stream)
        (stream or torch.cuda.current_stream()).synchronize()
        assert int(st.item()) == 0
        return [*plan, pool, out, lens, tables, free, count]

    late = None
    want = step(None, counts)
    true, late_bytes, view = _late(counts)
    late = (true, late_bytes)
    for _ in range(3):
        late_bytes.zero_()
        for a, b in zip(step(s, view), want):
            assert torch.equal(a, b)


def test_two_calls_at_once_on_two_streams():
    a = ChunkCase([(1, 5000)] * 30, 8, 2, seed=1)
    b = ChunkCase([(400, 1500), (1, 800)], 8, 2, window=300, seed=2)
    for kind in ("run_raw", "run_coded"):
        want = [getattr(c, kind)() for c in (a, b)]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        outs = [[torch.full_like(w, 77.0) for w in want] for _ in range(5)]
        torch.cuda.synchronize()
        for got in outs:
            for c, s, o in zip((a, b), streams, got):
                getattr(c, kind)(out=o, stream=s)
        torch.cuda.synchronize()
        for got in outs:
            assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert int(a.status.item()) == 0 and int(b.status.item()) == 0
