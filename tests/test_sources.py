"""Rules of the kernels that no run shows: read from their sources."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "block_sparse_paged_msa_gb300", "csrc")
REMOTE = re.compile(r"map_shared_rank|\bmapa\b|\bld\.shared::cluster|\bst\.shared::cluster"
                    r"|\bst\.async")


def _code(path):
    """A source without its comments."""
    text = re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def _kernels(text):
    """The texts from one __global__ to the next."""
    return text.split("__global__")[1:]


def _remote_kernels():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        for i, body in enumerate(_kernels(_code(path))):
            if REMOTE.search(body):
                yield pytest.param(body, id=f"{os.path.basename(path)[:-3]}-{i}")


@pytest.mark.parametrize("body", list(_remote_kernels()))
def test_another_blocks_shared_memory_is_touched_after_a_cluster_barrier(body):
    """A block of a cluster that has not started has no shared memory yet: before the
    first access to another block's comes a cluster barrier of all its threads (an
    arrival and a wait)."""
    first = REMOTE.search(body).start()
    before = body[:first]
    if "cluster.sync();" in before:
        return
    assert "cluster_arrive();" in before and "cluster_wait();" in before
    assert before.index("cluster_arrive();") < before.index("cluster_wait();")
    # no thread leaves between the two without the other half
    between = before[before.index("cluster_arrive();"):before.rindex("cluster_wait();")]
    leaves = [m.start() for m in re.finditer(r"\breturn;", between)]
    waits = [m.start() for m in re.finditer(r"cluster_wait\(\);", between)]
    assert len(waits) >= len(leaves) and all(w < x for w, x in zip(waits, leaves))
