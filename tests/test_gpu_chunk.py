"""kvz_chunk_attention and kvz_chunk_attention_raw on the GPU against attention in 64 bits: chunk lengths, contexts,
head layouts, windows and first tokens, padding, pages that are not there."""
import pytest
import torch

from chunk_case import ChunkCase

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def _both(case, dtype):
    ref = case.reference()
    for name in ("raw", "coded"):
        out = getattr(case, f"run_{name}")(dtype=dtype)
        torch.cuda.synchronize()
        assert int(case.status.item()) == 0, name
        case.check(out, ref, name)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,L", [(1, 1), (1, 15), (1, 16), (1, 17), (1, 128), (1, 129), (1, 700), (2, 2), (5, 260),
                                 (16, 16), (31, 31), (32, 130), (64, 64), (65, 65), (128, 128), (127, 400), (300, 300),
                                 (257, 1025)])
def test_one_sequence(n, L, dtype):
    _both(ChunkCase([(n, L)], 8, 2, seed=n + L), dtype)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (3, 1), (4, 4), (10, 2), (6, 1), (7, 1), (16, 2)])
@pytest.mark.parametrize("n,L", [(1, 333), (43, 200), (150, 390)])
def test_head_layouts(hq, hkv, n, L):
    _both(ChunkCase([(n, L)], hq, hkv, seed=hq), BF16)
    _both(ChunkCase([(n, L)], hq, hkv, seed=hq), F32)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (100, 0), (100, 130), (128, 64), (300, 20), (129, 3),
                                          (5000, 9), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_windows(window, sinks, dtype):
    _both(ChunkCase([(1, 900), (70, 70), (5, 1030), (200, 777), (1, 3), (0, 40)], 8, 2, window=window, sinks=sinks), dtype)


def test_mixed_batches_with_padding_and_empty_sequences():
    seqs = [(0, 0), (1, 1), (0, 55), (3, 3), (1, 640), (90, 600), (0, 0), (1, 17), (33, 2000), (1, 1500), (7, 7), (0, 16)]
    for dtype in (BF16, F32):
        _both(ChunkCase(seqs, 20, 4, lead=5, trail=9, seed=3, wide=2), dtype)


def test_tokens_before_the_first_see_nothing():
    _both(ChunkCase([(9, 4), (40, 0), (300, 12), (1, 5)], 8, 2, seed=4), BF16)
    _both(ChunkCase([(9, 4), (40, 0), (300, 12), (1, 5)], 8, 2, window=3, seed=4), F32)


def test_many_sequences():
    seqs = [(1 + (i % 3 == 0) * (i % 7), 1 + (i * 37) % 200 + 8) for i in range(1024)]
    _both(ChunkCase(seqs, 4, 1, seed=5), BF16)


def test_large_and_small_scores():
    for ks in (0.0, 0.02, 8.0):
        _both(ChunkCase([(40, 500), (1, 300)], 8, 2, seed=6, k_scale=ks, v_scale=30.0), BF16)
        _both(ChunkCase([(40, 500), (1, 300)], 8, 2, seed=6, k_scale=ks, v_scale=30.0), F32)


def test_bad_pages_are_left_out_and_flagged():
    import decode_attention_value_gb300 as kvz

    for bad in (-1, -5, 2 ** 31 - 1, -2 ** 31):
        case = ChunkCase([(20, 300), (1, 200)], 8, 2, seed=8)
        case.encode()
        skip = [(0, 3), (0, 17), (1, 12), (1, 0)]
        for b, p in skip:
            case.page_ids[b, p] = bad
            if p < case.whole.shape[1]:
                case.whole[b, p] = bad
        case.tail_page[1] = bad if bad != -1 else 2 ** 30
        ref = case.reference(skip)
        for name, dtype in (("raw", BF16), ("coded", F32), ("raw", F32), ("coded", BF16)):
            case.status.zero_()
            out = getattr(case, f"run_{name}")(dtype=dtype)
            torch.cuda.synchronize()
            assert int(case.status.item()) == kvz.STATUS_BAD_INDEX
            case.check(out, ref, f"{name} {bad}")


def test_bad_metadata_of_one_head_leaves_out_that_heads_page():
    import decode_attention_value_gb300 as kvz

    case = ChunkCase([(20, 300)], 8, 2, seed=9)
    case.encode()
    case.meta[case.full_ids[0, 5], 1, 0] = -1
    out = case.run_coded(dtype=F32)
    torch.cuda.synchronize()
    assert int(case.status.item()) == kvz.STATUS_BAD_META
    whole, part = case.reference(), case.reference([(0, 5)])
    mixed = [torch.cat([a[:, :4], b[:, 4:]], 1) for a, b in zip(whole[:3], part[:3])] + [whole[3]]
    case.check(out, mixed)


def test_lengths_and_starts_out_of_range():
    import decode_attention_value_gb300 as kvz

    case = ChunkCase([(20, 300), (3, 90)], 8, 2, seed=10)
    case.encode()
    good = {n: getattr(case, f"run_{n}")() for n in ("raw", "coded")}
    lens, starts = case.seq_lens.clone(), case.q_start.clone()
    for s in ([5, 3, 23], [-1, 20, 23], [0, 20, 24], [0, 2 ** 31 - 1, 23], [-2 ** 31, 0, 23]):
        case.q_start = torch.tensor(s, dtype=torch.int32, device="cuda")
        for n in ("raw", "coded"):
            case.status.zero_()
            out = getattr(case, f"run_{n}")()
            assert int(case.status.item()) == kvz.STATUS_BAD_ORDER and (out == 77.0).all(), (s, n)
    case.q_start = starts
    for bad in (-5, -2 ** 31):
        case.seq_lens = torch.tensor([300, bad], dtype=torch.int32, device="cuda")
        for n in ("raw", "coded"):
            case.status.zero_()
            out = getattr(case, f"run_{n}")()
            assert int(case.status.item()) == kvz.STATUS_BAD_INDEX
            assert torch.equal(out[:20], good[n][:20]) and (out[20:] == 0).all()
    # beyond the table: cut to it
    case.pool, case.seq_lens = case.clean, torch.tensor([2 ** 31 - 1, 90], dtype=torch.int32, device="cuda")
    case.status.zero_()
    out = case.run_raw()
    assert int(case.status.item()) & kvz.STATUS_BAD_INDEX and torch.equal(out[20:], good["raw"][20:])
    case.seq_lens = lens
    case.status.zero_()
    assert torch.equal(case.run_raw(), good["raw"]) and int(case.status.item()) == 0


def test_the_same_call_twice_and_captured_gives_the_same_bits():
    seqs = [(1, 3000), (150, 1500), (1, 20), (600, 600)]
    for window in (0, 256):
        case = ChunkCase(seqs, 16, 4, window=window, sinks=8 if window else 0, seed=11)
        for name in ("raw", "coded"):
            run = getattr(case, f"run_{name}")
            a, b = run(), run()
            assert torch.equal(a, b)
            size = case.kvz.chunk_attention_workspace_size(4, case.T, 16, len(seqs), case.width, coded=True)
            ws = torch.empty(size, dtype=torch.uint8, device="cuda")
            out = torch.full_like(a, 77.0)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                run(out=out, workspace=ws)
            for _ in range(3):
                out.fill_(77.0)
                ws.fill_(255)
                g.replay()
                assert torch.equal(out, a)
