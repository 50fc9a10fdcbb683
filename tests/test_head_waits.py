"""Every wait of the kernels has a limit: none of them meets a whole grid through
the library's barrier, whose wait has none."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ctc_prefix_beam_gb300", "csrc")


def test_no_wait_without_a_limit():
    files = glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    assert len(files) > 8
    for f in files:
        with open(f) as h:
            assert not re.search(r"cooperative_groups|this_grid|grid_group|barrier_sync_count", h.read()), f
