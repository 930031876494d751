"""What the biased linears' kernels have to hold to and no run on a GPU can show, read from their source."""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "backward_split_linear_gb300", "csrc", "linear.cu")


def test_barriers_of_a_pair_are_waited_on_at_cluster_scope():
    """The other CTA of a pair arrives on these barriers, or its loads' bytes do."""
    text = open(SOURCE).read()
    waits = re.findall(r"(mbar_wait\w*)\((?:leader \? )?(\w+)\(", text)
    shared = [(call, bar) for call, bar in waits if bar in ("full_bar", "empty_bar", "tfull_bar", "tempty_bar")]
    assert len(shared) >= 10
    for call, bar in shared:
        assert call.startswith("mbar_wait_cluster"), (call, bar)
