"""Instructions of the `.aligned` form take a warp whose lanes are together.  Where
lanes may have parted on the way there (a loop whose length depends on the lane, one
lane that arrives on a barrier, a store of some rows) the warp is brought together
first: held here by reading, since what a parted warp does is not defined."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_attention_sequence_chunked_gb300",
                    "csrc")


def _lines(name):
    """The statements of a source, without comments and blank lines."""
    text = open(os.path.join(CSRC, name)).read()
    text = re.sub(r"//[^\n]*", "", text)
    return [s.strip() for s in text.splitlines() if s.strip()]


def test_cluster_barriers_stand_in_one_place():
    users = [f for f in sorted(os.listdir(CSRC)) if any("barrier.cluster" in s for s in _lines(f))]
    assert users == ["gdn_cluster.cuh"]


def test_cluster_barriers_bring_their_warp_together():
    lines = _lines("gdn_cluster.cuh")
    at = [i for i, s in enumerate(lines) if "barrier.cluster" in s]
    assert len(at) == 2 and all(lines[i - 1] == "__syncwarp();" for i in at)


@pytest.mark.parametrize("name,count", [("gdn_window_fwd.cu", 1), ("gdn_window_bwd.cu", 3)])
def test_window_kernels_bring_their_warps_together(name, count):
    """Before tensor memory is allocated (behind the offsets' checks) and before a
    barrier of some warps (behind one lane's arrival)."""
    lines = _lines(name)
    at = [i for i, s in enumerate(lines) if "tmem_alloc(" in s or "named_bar(" in s]
    assert len(at) == count and all(lines[i - 1] == "__syncwarp();" for i in at)


def test_rows_stored_between_loads_of_tensor_memory():
    """The gradients' fp32 sums: some lanes store a row between two loads."""
    lines = _lines("gdn_window_bwd.cu")
    store = lines.index("if (j < joined) {")
    end = next(i for i in range(store, len(lines)) if lines[i] == "__syncwarp();")
    assert not any("tmem_ld" in s or "store_rows" in s for s in lines[store:end])


def test_the_steps_products_follow_a_uniform_branch():
    """Rescaling between the scores and the second product hangs on the warp's vote."""
    lines = _lines("gdn_window_step.cu")
    assert any(s.startswith("if (__any_sync(0xffffffffu, f != 1.f))") for s in lines)
    assert not any(s.startswith("if (f != 1.f)") for s in lines)
