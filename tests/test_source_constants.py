"""The number of SMs is asked of the device: in the kernels' sources it stands only where that question
may go unanswered (a machine without a driver, where only sizes are computed)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "piecewise_attention_diffusion_b200", "csrc")


def test_the_cards_size_is_asked_for():
    files = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))
    assert files
    for path in files:
        code = re.sub(r"//.*", "", open(path).read())
        code = code.replace("return n > 0 ? n : 148;", "")
        assert not re.search(r"\b148\b", code), os.path.basename(path)
