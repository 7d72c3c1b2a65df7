"""Stores into another CTA's shared memory come after a barrier of the cluster, as that CTA must have
started: read from the kernels' source, since on a GPU a cluster's CTAs start together and a missing
barrier hardly ever shows."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "activation_sparse_ffn_threshold_b200", "csrc")


def kernels():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for body in text.split("__global__")[1:]:
            if "st.shared::cluster" in body:
                yield pytest.param(body, id=os.path.basename(path) + re.search(r"\b(k_\w+)\(", body).group(1))


def as_run(body, apart):
    """The source with the statements that stand under a condition on where the exchange lies resolved."""
    def chosen(m):
        return m.group(2) if (m.group(1) == "") == apart else m.group(3) or ""
    return re.sub(r"if \((!?)P\.apart\)\s*([^;{}]*;)(?:\s*else\s*([^;{}]*;))?", chosen, body)


@pytest.mark.parametrize("apart", [True, False])
@pytest.mark.parametrize("body", list(kernels()))
def test_a_cluster_barrier_stands_before_the_first_remote_store(body, apart):
    before = as_run(body, apart).split("st.shared::cluster")[0]
    both = "cluster_arrive();" in before and "cluster_wait();" in before.split("cluster_arrive();", 1)[1]
    assert both or "cluster_sync_all();" in before
