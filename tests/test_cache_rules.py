"""Rules of the key/value cache's sources that a run cannot show reliably: what they guard against would be a race or stale
data on the GPU, so they are checked in the text."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_weight_matvec_hq_gb300", "csrc")


def source(path):
    """A source file without its comments."""
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S))


def test_no_load_is_of_memory_that_nobody_writes():
    """Kernels start while the one in front of them still runs, which may write what they read: their wait orders plain
    loads, and nothing says that it orders those of the read-only form."""
    paths = sorted(glob.glob(os.path.join(CSRC, "*.cu*")))
    assert len(paths) > 8
    for path in paths:
        assert not re.findall(r"ld\.global(?:\.\w+)*\.nc\b|\b__ldg\b|\b__ldg\(", source(path)), path
