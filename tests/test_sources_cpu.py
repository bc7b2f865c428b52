"""What the sources of liblr must not hold, read from their text."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_delta_rule_fwd_gb300", "csrc")


def sources():
    """(name, text without comments) of every source and header of the kernels."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        with open(path) as f:
            yield os.path.basename(path), re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_no_copy_is_sent_to_several_ctas():
    """The library is one for every process: its tensor maps cover whatever pointer a
    caller passes, which need not be this GPU's own memory."""
    found = [name for name, text in sources() if "multicast" in text]
    assert not found
