"""Loops of plan.cu over tokens, rows and free pages end where these are near 2^31: read from the source, and run."""
import os
import re

import pytest
import torch

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_attention_value_gb300", "csrc", "plan.cu")


def test_loops_over_caller_counts_step_in_unsigned_bits():
    """A signed count of steps of 8192 wraps past 2^31 - 8192, to places before the tensor."""
    with open(SRC) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    loops = re.findall(r"for \((\w+) \w+ = (?:at|tid); \w+ < ([^;]*(?:P\.tokens|P\.num_rows|all\[1\])[^;]*); ", code)
    assert len(loops) == 3
    for kind, bound in loops:
        assert kind == "uint32_t" and "(uint32_t)" in bound


@pytest.mark.gpu
def test_a_plan_of_almost_two_to_the_31_tokens():
    import decode_attention_value_gb300 as kvz

    T, dev = 2 ** 31 - 1, lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    plan, status = kvz.new_step_plan(1, T, 2), kvz.new_status()
    plan.positions.fill_(55)
    lens = dev([3])
    kvz.plan_step(dev([0]), dev([20]), lens, dev([[7, -1]]), dev([9]), dev([1]), plan, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and lens.tolist() == [23]
    assert plan.slots[:20].tolist() == [7 * 16 + i for i in range(3, 16)] + [9 * 16 + i for i in range(7)]
    assert not plan.positions[20:].any() and bool((plan.slots[20:] == -1).all())
