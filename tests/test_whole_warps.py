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
