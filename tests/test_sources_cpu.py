"""What the kernels' sources may not hold."""
import glob
import os

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "long_context_split_gb300", "csrc")


def test_no_copy_or_commit_goes_to_several_ctas():
    """Every CTA fetches its own tiles: the library serves processes that run beside others on the
    machine's GPUs, and a copy to several CTAs is kept out of those."""
    files = glob.glob(os.path.join(CSRC, "*"))
    assert len(files) > 20
    for path in files:
        with open(path) as f:
            assert ".multicast" not in f.read(), path
