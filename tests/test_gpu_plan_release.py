"""release_pages on the GPU: rows with entries that hold no page, the order pages come back in, and what it refuses."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PAGE = 16


def _dev(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("B,width", [(1, 1), (3, 70), (40, 33), (1024, 9)])
def test_entries_that_hold_no_page_are_passed_over(B, width):
    """Pages behind a sliding window are gone: -1, or another number that no slot can name."""
    import decode_attention_value_gb300 as kvz

    rng = np.random.default_rng(B)
    S = B + 5
    rows = rng.permutation(S)[:B]
    lens = np.zeros(S, np.int64)
    lens[rows] = rng.integers(0, width * PAGE + 1, B)
    lens[rows[0]] = width * PAGE
    tables = rng.permutation(S * width).reshape(S, width)
    gone = rng.random((S, width)) < 0.5
    gone[rows[0], : width // 2 + 1] = True
    tables = np.where(gone, rng.choice([-1, -7, -2 ** 31, 2 ** 31 - 1, 2 ** 27], (S, width)), tables)
    if B > 3:
        rows[1] = -1
    back = []
    for r in rows[rows >= 0]:
        mine = tables[r, : -(-lens[r] // PAGE)]
        back += [x for x in mine[::-1] if 0 <= x < 2 ** 27]
    free = [900001, 900002]
    d_lens, d_tables, count, status = _dev(lens), _dev(tables), _dev([2]), kvz.new_status()
    pages = _dev([*free, *[-9] * len(back)])  # room for them and no more
    kvz.release_pages(_dev(rows), d_lens, d_tables, pages, count, status)
    assert int(status.item()) == 0 and int(count.item()) == 2 + len(back)
    assert pages.tolist() == [*free, *back]
    for r in rows[rows >= 0]:
        tables[r, : -(-lens[r] // PAGE)] = -1
        lens[r] = 0
    assert np.array_equal(d_lens.cpu().numpy(), lens) and np.array_equal(d_tables.cpu().numpy(), tables)


def test_a_window_given_back_then_the_rest_and_taken_again():
    import decode_attention_value_gb300 as kvz

    lens, tables = _dev([100, 0]), _dev([[3, 9, 4, 1, 8, 2, 7, -1], [-1] * 8])
    free, count, status = _dev([6] + [-1] * 9), _dev([1]), kvz.new_status()
    # a caller gives back the pages behind a window of 40 tokens himself
    free[1:4], count[0] = tables[0, :3].clone(), 4
    tables[0, :3] = -1
    kvz.release_pages(_dev([0]), lens, tables, free, count, status)
    assert int(count.item()) == 8 and sorted(free[:8].tolist()) == [1, 2, 3, 4, 6, 7, 8, 9] and (tables == -1).all()
    plan = kvz.new_step_plan(1, 128, 8)
    kvz.plan_step(_dev([1]), _dev([128]), lens, tables, free, count, plan, status)
    assert int(status.item()) == 0 and int(count.item()) == 0
    assert sorted(plan.page_ids[0].tolist()) == [1, 2, 3, 4, 6, 7, 8, 9] and (plan.slots >= 0).all()


def test_releases_that_are_refused_change_nothing():
    import decode_attention_value_gb300 as kvz

    base = dict(rows=[1, 0], lens=[5, 30, 0], count=[2])
    for change, bit in ((dict(rows=[1, 1]), kvz.STATUS_BAD_ORDER), (dict(rows=[0, 3]), kvz.STATUS_BAD_INDEX),
                        (dict(rows=[-2, 0]), kvz.STATUS_BAD_INDEX), (dict(rows=[2 ** 31 - 1, 0]), kvz.STATUS_BAD_INDEX),
                        (dict(lens=[-1, 30, 0]), kvz.STATUS_BAD_INDEX), (dict(lens=[5, 65, 0]), kvz.STATUS_BAD_INDEX),
                        (dict(lens=[5, 2 ** 31 - 1, 0]), kvz.STATUS_BAD_INDEX), (dict(lens=[-2 ** 31, 30, 0]), kvz.STATUS_BAD_INDEX),
                        (dict(count=[-1]), kvz.STATUS_BAD_INDEX), (dict(count=[3]), kvz.STATUS_BAD_INDEX),
                        (dict(count=[6]), kvz.STATUS_BAD_INDEX)):
        c = {**base, **change}
        tables = _dev([[3, -1, -1, -1], [1, 2, -1, -1], [-1] * 4])
        lens, count, free, status = _dev(c["lens"]), _dev(c["count"]), _dev([9, 8, -1, -1, -1]), kvz.new_status()
        before = tables.clone()
        kvz.release_pages(_dev(c["rows"]), lens, tables, free, count, status)
        assert int(status.item()) == bit, change
        assert lens.tolist() == c["lens"] and count.tolist() == c["count"], change
        assert torch.equal(tables, before) and free.tolist() == [9, 8, -1, -1, -1], change
    # and the same call with nothing wrong
    lens, tables, count, free = _dev(base["lens"]), _dev([[3, -1, -1, -1], [1, 2, -1, -1], [-1] * 4]), _dev([2]), _dev([9, 8, -1, -1, -1])
    status = kvz.new_status()
    kvz.release_pages(_dev(base["rows"]), lens, tables, free, count, status)
    assert int(status.item()) == 0 and count.tolist() == [5] and free.tolist() == [9, 8, 2, 1, 3]
    assert lens.tolist() == [0, 0, 0] and (tables == -1).all()
