"""Instructions that want the whole warp (.aligned) stand where its lanes have met, read from the sources."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_attention_value_gb300", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_plan_cluster_barrier_takes_threads_one_by_one():
    """Lanes come to it from a loop over the rows, of which some have one turn more."""
    code = _code("plan.cu")
    assert "barrier.cluster.arrive.release;" in code and "barrier.cluster.wait.acquire;" in code
    assert ".aligned" not in code


def test_chunk_lanes_without_a_row_meet_the_others_before_tensor_memory():
    """What only lanes with a row do ends in a __syncwarp() before the next load or store of tensor memory and before
    the next instruction that waits for the other stream."""
    code = _code("chunk.cu")
    places = [m.end() for m in re.finditer(r"\blane < rows\b", code)]
    assert len(places) >= 6
    for at in places:
        nxt = re.search(r"\btmem_(ld|st)\d+\(|\bmeet\(\)|__syncwarp\(\)", code[at:])
        line = code[:at].count("\n") + 1
        assert nxt and nxt.group(0) == "__syncwarp()", (line, nxt and nxt.group(0))
