"""plan_step takes no step whose new tokens would get a page that no slot can name, and minds no other page."""
import pytest
import torch

pytestmark = pytest.mark.gpu

PAGE = 16


def _dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _run(lens, tables, free, rows=(0, 2), new=(20, 33), in_place=True):
    import decode_attention_value_gb300 as kvz

    d = [_dev(rows), _dev(new), _dev(lens), _dev(tables), _dev(free), _dev([len(free)])]
    plan, status = kvz.new_step_plan(2, 64, 4), kvz.new_status()
    for t in plan:
        t.fill_(55)
    out = {} if in_place else dict(lens_out=torch.full_like(d[2], 55), free_out=torch.full_like(d[5], 55))
    kvz.plan_step(*d, plan, status, **out)
    return plan, int(status.item()), out.get("lens_out", d[2]).tolist(), out.get("free_out", d[5]).tolist(), d[3].tolist()


LENS, FREE = [21, 0, 0], [30, 31, 2 ** 27 - 1, 32, 33]
TABLES = [[-1, 7, -1, -1], [-1] * 4, [-1] * 4]  # the first page stands behind a window and is gone


@pytest.mark.parametrize("in_place", [True, False])
def test_the_largest_page_and_a_page_that_is_gone(in_place):
    plan, status, lens, count, tables = _run(LENS, TABLES, FREE, in_place=in_place)
    assert status == 0 and lens == [41, 0, 33] and count == [1]
    assert tables[0] == [-1, 7, 33, -1] and tables[2] == [32, 2 ** 27 - 1, 31, -1]
    assert plan.slots.tolist()[:20] == [7 * PAGE + i for i in range(5, 16)] + [33 * PAGE + i for i in range(9)]
    assert plan.slots.tolist()[36:53] == [(2 ** 27 - 1) * PAGE + i for i in range(16)] + [31 * PAGE]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("bad", [-1, -2 ** 31, 2 ** 27, 2 ** 31 - 1])
def test_a_page_without_slots_refuses_the_step(bad, in_place):
    import decode_attention_value_gb300 as kvz

    for where in ("last", 1, 2, 3, 4):
        tables, free = [list(r) for r in TABLES], list(FREE)
        if where == "last":
            tables[0][1] = bad
        else:
            free[where] = bad
        plan, status, lens, count, after = _run(LENS, tables, free, in_place=in_place)
        assert status == kvz.STATUS_BAD_INDEX, where
        assert lens == LENS and count == [5] and after == tables, where
        assert not plan.q_start.any() and not plan.seq_lens.any() and not plan.positions.any()
        assert (plan.page_ids == -1).all() and (plan.slots == -1).all()
    # a free page that the step does not take, and a last page without room, may be anything
    plan, status, *_ = _run(LENS, TABLES, [bad, *FREE[1:]], in_place=in_place)
    assert status == 0 and (plan.slots[:53] >= 0).all()
    plan, status, *_ = _run([32, 0, 0], [[-1, bad, -1, -1], *TABLES[1:]], FREE, in_place=in_place)
    assert status == 0 and (plan.slots[:53] >= 0).all()


def test_a_place_without_new_tokens_minds_no_page():
    plan, status, lens, count, _ = _run(LENS, [[-1, -1, -1, -1], *TABLES[1:]], FREE, new=(0, 33))
    assert status == 0 and lens == [21, 0, 33] and count == [2]
    # and many pages at once, the bad one the last taken
    import decode_attention_value_gb300 as kvz

    n = 5000
    for bad in (False, True):
        free = torch.randperm(n, device="cuda").to(torch.int32)
        free[0] = -1 if bad else free[0]
        lens, tables, count, status = _dev([0]), torch.full((1, n), -1, dtype=torch.int32, device="cuda"), _dev([n]), kvz.new_status()
        plan = kvz.new_step_plan(1, n * PAGE, n)
        kvz.plan_step(_dev([0]), _dev([n * PAGE]), lens, tables, free, count, plan, status)
        assert int(status.item()) == (kvz.STATUS_BAD_INDEX if bad else 0)
        assert (int(lens.item()), int(count.item())) == ((0, n) if bad else (n * PAGE, 0))
        if not bad:
            assert torch.equal(tables[0], free.flip(0)) and torch.equal(plan.slots, (tables[0, :, None] * PAGE + _dev(list(range(PAGE)))).flatten())
