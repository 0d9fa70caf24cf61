"""kvz_prefix_attention_raw and kvz_prefix_attention against attention in 64 bits: group shapes,
lengths around pages and blocks, head layouts, empty rows, bad pages, streams and graphs."""
import pytest
import torch

from prefix_case import D, PAGE, PrefixCase

pytestmark = pytest.mark.gpu

BOTH = ["raw", "coded"]


@pytest.fixture(autouse=True, params=[False, True], ids=["narrow", "wide"])
def both_ways(request, monkeypatch):
    """Short prefixes are read with the own tokens; tables wide enough for long ones send them through the
    prefix kernel.  Every test runs both ways."""
    monkeypatch.setattr(PrefixCase, "wide", request.param)


def run(case, kind, **kw):
    out = case.run_raw(**kw) if kind == "raw" else case.run_coded(**kw)
    torch.cuda.synchronize()
    assert not int(case.status.item()) & case.kvz.STATUS_TIMEOUT
    return out


def own_lens(n, top, seed=0):
    return [(i * 2654435761 + seed * 97 + 11) % (top + 1) for i in range(n)]


@pytest.mark.parametrize("kind", BOTH)
@pytest.mark.parametrize("prefix", [1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1000, 4111])
def test_prefix_lengths(kind, prefix):
    c = PrefixCase([(6, prefix)], own_lens(6, 40, prefix), 8, 2, seed=prefix)
    rel = c.check(run(c, kind), what=f"prefix {prefix}")
    assert int(c.status.item()) == 0 and rel < 1e-4


@pytest.mark.parametrize("kind", BOTH)
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("hkv,n", [(1, 3), (2, 33), (3, 64)])
def test_head_layouts(kind, G, hkv, n):
    c = PrefixCase([(n, 700)], own_lens(n, 70, G), G * hkv, hkv, seed=G)
    c.check(run(c, kind, dtype=torch.bfloat16))
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("kind", BOTH)
@pytest.mark.parametrize("n,G", [(16, 4), (50, 4)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_blocks_a_cta(kind, n, G, dtype):
    """Long prefixes over many KV heads: every ring of the kernel wraps several times."""
    c = PrefixCase([(n, 40003), (2, 9000)], own_lens(n + 2, 20), 8 * G, 8, seed=n)
    ref = c.reference()
    c.check(run(c, kind, dtype=dtype), ref)
    first = run(c, kind, dtype=dtype)
    for _ in range(4):
        assert torch.equal(first, run(c, kind, dtype=dtype))
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("kind", BOTH)
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 65, 130, 300])
def test_group_sizes(kind, n):
    """Rows that fill no tile, one tile, two tiles of a CTA, and several of those."""
    c = PrefixCase([(n, 515)], own_lens(n, 33, n), 8, 2, seed=n)
    c.check(run(c, kind))
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("kind", BOTH)
@pytest.mark.parametrize("G", [1, 2, 4, 7])
@pytest.mark.parametrize("top", [1023, 1024, 1040, 2100])
def test_long_own_tokens(kind, G, top):
    """Own tokens on both sides of where they are split over CTAs, ragged, with empty ones."""
    own = own_lens(9, top, G)
    own[2], own[5], own[8] = top, 0, 1
    c = PrefixCase([(3, 200), (4, 0), (1, 31)], own, 2 * G, 2, seed=top + G)
    ref = c.reference()
    c.check(run(c, kind), ref)
    c.check(run(c, kind, dtype=torch.bfloat16), ref)
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("kind", BOTH)
@pytest.mark.parametrize("groups", [[(3, 400), (1, 17), (9, 1300), (2, 128)], [(70, 300), (2, 900), (40, 1)],
                                    [(4, 0), (0, 500), (5, 260), (0, 0)], [(1, 50)] * 40])
def test_groups_of_different_sizes(kind, groups):
    n = sum(g for g, _ in groups)
    c = PrefixCase(groups, own_lens(n + 5, 50, n), 10, 2, seed=n, lead=3)  # three sequences before, two behind
    c.check(run(c, kind))
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("kind", BOTH)
def test_most_groups(kind):
    c = PrefixCase([(1, 1 + i % 40) for i in range(256)], own_lens(256, 20), 2, 1, seed=5)
    c.check(run(c, kind))
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("kind", BOTH)
@pytest.mark.parametrize("prefix,n", [(5000, 5), (2049, 40)])
def test_uniform_weights_count_every_token_once(kind, prefix, n):
    """K = 0: the output is the mean of V; small integers make every sum exact."""
    ints = lambda shape, g: torch.randint(-8, 9, shape, generator=g, device="cuda").float()  # noqa: E731
    zero = lambda shape, g: torch.zeros(shape, device="cuda")  # noqa: E731
    c = PrefixCase([(n, prefix), (3, 77)], own_lens(n + 4, 90), 16, 4, seed=1, k=zero, v=ints)
    want, _ = c.reference()
    got = run(c, kind).double()
    # weights 1 and integer sums are exact; a reciprocal and a product round.  The mean in 64 bits, a
    # sum of at most 5090 rounded products of at most 8 / 5090 (where the values cancel it is all
    # rounding): off by at most 5090 half-steps of 8, 5090 * 8 * 2^-53 < 2^-37
    assert ((got - want).abs() <= 2.0 ** -22 * want.abs() + 2.0 ** -37).all()


@pytest.mark.parametrize("kind", BOTH)
def test_growing_scores_move_the_maximum(kind):
    """Scores that rise along the prefix, far past 2^8 between blocks: the output is rescaled."""
    def rising(shape, g):
        return torch.randn(shape, generator=g, device="cuda")

    c = PrefixCase([(40, 3000)], own_lens(40, 30), 8, 2, seed=3, k=rising)
    ramp = torch.arange(c.pw, device="cuda")[:, None, None, None] / c.pw * 12
    direction = c.q[0, 0].float()  # every query sees a ramp of its own sign and size
    ids = c.prefix_ids[0].long()
    k = c.pool[ids, :, 0].float() + ramp * direction / direction.norm()
    c.pool[ids, :, 0] = k.to(torch.bfloat16)
    if 3000 % PAGE:
        c.pool[ids[-1], :, :, 3000 % PAGE:] = float("nan")
    c.check(run(c, kind))


@pytest.mark.parametrize("kind", BOTH)
def test_rows_without_tokens_are_zero(kind):
    c = PrefixCase([(2, 0), (3, 300)], [0, 5, 0, 0, 4, 0], 8, 2, seed=7)
    got = run(c, kind)
    c.check(got)
    assert torch.equal(got[0], torch.zeros_like(got[0])) and torch.equal(got[5], torch.zeros_like(got[5]))
    none = PrefixCase([], [3, 0, 40], 8, 2, seed=8)
    none.check(run(none, kind))
    assert int(none.status.item()) == 0 and int(c.status.item()) == 0


@pytest.mark.parametrize("kind", BOTH)
def test_own_tokens_alone_equal_decode_attention(kind):
    """Without prefixes: the same partials as the plain calls, merged in another order."""
    c = PrefixCase([(5, 0)], [100, 0, 37, 16, 260], 8, 2, seed=9)
    got = run(c, kind)
    out = torch.empty_like(got)
    if kind == "raw":
        c.kvz.decode_attention_raw(c.q, c.page_ids, c.seq_lens, c.pool, out, c.status)
    else:
        c.kvz.decode_attention(c.q, c.own_whole, c.seq_lens, c.tail_page, c.meta, c.arena, c.pool, out, c.status)
    # the merges differ by a few fp32 roundings of sums of at most 16 partials
    assert ((got - out).abs() <= 2.0 ** -19 * out.abs().amax()).all()


@pytest.mark.parametrize("kind", BOTH)
def test_bad_pages_are_left_out_and_flagged(kind):
    c = PrefixCase([(4, 700), (2, 90)], [20] * 6, 8, 2, seed=11)
    run(c, kind)
    assert int(c.status.item()) == 0
    table = c.prefix_ids if kind == "raw" else c.prefix_whole
    for bad in (c.pool.shape[0], -5, 2 ** 31 - 1):
        keep = table[0, 9].clone()
        table[0, 9] = bad
        got = run(c, kind)
        assert int(c.status.item()) == c.kvz.STATUS_BAD_INDEX
        table[0, 9] = keep
        c.status.zero_()
        ids = c.prefix_ids[0].clone()
        shared = c.reference(skip_prefix=())  # rows of the second group are untouched
        assert torch.equal(c.prefix_ids[0], ids)
        want = PrefixCase.reference(c, skip_prefix=(9,))
        # page 9 of group 0 is left out; the second group has no page 9
        c.check(got, want)
        assert (shared[0][4:] == want[0][4:]).all()


def test_every_page_of_a_prefix_bad():
    c = PrefixCase([(3, 200)], [0, 9, 40], 8, 2, seed=12)
    c.prefix_ids.fill_(-1)
    got = run(c, "raw")
    assert int(c.status.item()) == c.kvz.STATUS_BAD_INDEX
    c.check(got, c.reference(prefix=False))


def test_unusable_metadata_and_tails():
    c = PrefixCase([(4, 700)], [20, 33, 0, 16], 8, 2, seed=13)
    run(c, "coded")
    page = int(c.prefix_whole[0, 3])
    for group in (0xFFFFFFFF, (0x90 << 32) | 5, (0xFFFFFF00 << 0)):
        keep = c.meta[page].clone()
        c.meta[page] = torch.tensor(group, dtype=torch.int64)
        got = run(c, "coded")
        assert int(c.status.item()) == c.kvz.STATUS_BAD_META
        c.meta[page] = keep
        c.status.zero_()
        c.check(got, c.reference(skip_prefix=(3,)))
    c.prefix_tail[0] = -1
    got = run(c, "coded")
    assert int(c.status.item()) == c.kvz.STATUS_BAD_TAIL
    c.check(got, c.reference(skip_prefix=(700 // PAGE,)))
    c.prefix_tail[0] = c.pool.shape[0]
    c.status.zero_()
    run(c, "coded")
    assert int(c.status.item()) == c.kvz.STATUS_BAD_INDEX


@pytest.mark.parametrize("kind", BOTH)
def test_lengths_out_of_range(kind):
    c = PrefixCase([(2, 320), (2, 100)], [10] * 4, 8, 2, seed=14)
    want = c.reference()
    run(c, kind)
    c.prefix_lens[0] = 2 ** 31 - 1 if kind == "raw" else 320  # past the table: all of it
    got = run(c, kind)
    assert int(c.status.item()) == (c.kvz.STATUS_BAD_INDEX if kind == "raw" else 0)
    c.check(got, want)
    c.status.zero_()
    c.prefix_lens[0] = -7
    got = run(c, kind)
    assert int(c.status.item()) == c.kvz.STATUS_BAD_INDEX
    c.groups[0] = (2, 0)
    c.check(got, c.reference())


@pytest.mark.parametrize("kind", BOTH)
@pytest.mark.parametrize("start", [[0, 3, 2, 4], [-1, 1, 2, 4], [0, 1, 2, 5]])
def test_group_starts_out_of_order(kind, start):
    c = PrefixCase([(1, 100), (1, 50), (2, 70)], [10, 20, 30, 40], 8, 2, seed=15)
    run(c, kind)
    c.group_start.copy_(torch.tensor(start, dtype=torch.int32))
    got = run(c, kind)
    assert int(c.status.item()) == c.kvz.STATUS_BAD_ORDER
    c.check(got, c.reference(prefix=False))


@pytest.mark.parametrize("kind", BOTH)
def test_infinities_and_nan_behind_the_last_token(kind):
    """Rows of the last pages behind a sequence's end (NaN in PrefixCase) and infinite values
    there change nothing."""
    c = PrefixCase([(5, 1 + 128 * 3)], [1, 17, 33, 0, 15], 8, 2, seed=16)
    a = run(c, kind)
    for ids, lens in ((c.prefix_ids, [385]), (c.page_ids, c.own)):
        for r, n in enumerate(lens):
            if n % PAGE:
                c.pool[ids[r, n // PAGE], :, :, n % PAGE:] = float("inf")
    assert torch.equal(a, run(c, kind))
    c.check(a)


@pytest.mark.parametrize("kind", BOTH)
def test_same_bits_again_on_streams_and_in_graphs(kind):
    c = PrefixCase([(20, 2000), (3, 300)], own_lens(23, 64), 16, 4, seed=17)
    want = run(c, kind)
    size = c.kvz.prefix_attention_workspace_size(4, 23, 16, 2, c.pw, c.ow)
    w1, w2 = (torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    o1, o2 = torch.empty_like(want), torch.empty_like(want)
    torch.cuda.synchronize()
    for _ in range(5):  # two calls at once, a workspace each
        (c.run_raw if kind == "raw" else c.run_coded)(out=o1, workspace=w1, stream=s1)
        (c.run_raw if kind == "raw" else c.run_coded)(out=o2, workspace=w2, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(o1, want) and torch.equal(o2, want)
    with torch.cuda.stream(s1):  # workspace of the call's own
        o3 = run(c, kind)
    assert torch.equal(o3, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        (c.run_raw if kind == "raw" else c.run_coded)(out=o1, workspace=w1)
        (c.run_raw if kind == "raw" else c.run_coded)(out=o2, workspace=w1)  # one workspace, one after the other
    for step in range(3):
        o1.fill_(7)
        o2.fill_(7)
        c.q.copy_(c.q.flip(0) if step else c.q)
        c.seq_lens[0] = c.own[0] = 0 if step == 2 else c.own[0]  # lengths are read at replay
        g.replay()
        assert torch.equal(o1, run(c, kind)) and torch.equal(o2, o1)
    assert int(c.status.item()) == 0


def test_prefix_pages_may_be_a_sequences_own():
    c = PrefixCase([(3, 96)], [40, 5, 0], 8, 2, seed=18)
    c.page_ids[1, :3] = c.prefix_ids[0, :3]
    c.own[1] = 48
    c.seq_lens[1] = 48
    c.check(run(c, "raw"))


def test_table_offsets_past_32_bits():
    """A pool of more than 2^31 elements: pages past the 4 GiB mark hold the prefix."""
    c = PrefixCase([(4, 500)], [20] * 4, 8, 2, seed=19)
    want = c.run_raw()
    P, big = c.pool.shape[0], 600000  # 600000 pages of 16 KB: 9.8 GB
    pool = torch.empty((big, 2, 2, PAGE, D), dtype=torch.bfloat16, device="cuda")
    pool[big - P:] = c.pool
    c.prefix_ids += big - P
    c.page_ids += big - P
    c.pool = pool
    assert torch.equal(c.run_raw(), want)


def test_binding_refusals():
    import decode_attention_value_gb300 as kvz

    c = PrefixCase([(2, 40), (1, 20)], [10] * 3, 8, 2, seed=20)
    c.run_coded()
    raw = dict(q=c.q, group_start=c.group_start, prefix_ids=c.prefix_ids, prefix_lens=c.prefix_lens,
               page_ids=c.page_ids, seq_lens=c.seq_lens, raw_pool=c.pool, out=torch.empty_like(c.q), status=c.status)
    for name, bad in (("q", c.q.float()), ("q", c.q[:, :, :64]), ("q", c.q.cpu()), ("q", c.q.transpose(0, 1)),
                      ("group_start", c.group_start[:2]), ("group_start", c.group_start.long()),
                      ("prefix_ids", c.prefix_ids[:1]), ("prefix_ids", c.prefix_ids[0]),
                      ("prefix_lens", c.prefix_lens.long()), ("page_ids", c.page_ids[:2]),
                      ("page_ids", c.page_ids.t()), ("seq_lens", c.seq_lens[:2]), ("raw_pool", c.pool[:, :1]),
                      ("raw_pool", c.pool.float()), ("out", torch.empty_like(c.q).half()),
                      ("out", torch.empty_like(c.q)[:2]), ("status", c.status.cpu()),
                      ("workspace", torch.empty(64, device="cuda"))):
        with pytest.raises(ValueError):
            kvz.prefix_attention_raw(**{**raw, name: bad})
    with pytest.raises(kvz.KvzError):
        kvz.prefix_attention_raw(**{**raw, "workspace": torch.empty(64, dtype=torch.uint8, device="cuda")})
    coded = dict(q=c.q, group_start=c.group_start, prefix_ids=c.prefix_whole, prefix_lens=c.prefix_lens,
                 prefix_tail=c.prefix_tail, page_ids=c.own_whole, seq_lens=c.seq_lens, tail_page=c.tail_page,
                 meta=c.meta, arena=c.arena, raw_pool=c.pool, out=torch.empty_like(c.q), status=c.status)
    for name, bad in (("prefix_tail", c.prefix_tail[:1]), ("tail_page", c.tail_page[:2]), ("meta", c.meta.int()),
                      ("meta", c.meta[:, :1]), ("arena", c.arena.view(torch.int16)), ("raw_pool", c.pool[:, :, :1])):
        with pytest.raises(ValueError):
            kvz.prefix_attention(**{**coded, name: bad})
    assert int(c.status.item()) == 0
