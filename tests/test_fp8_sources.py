"""Properties of the 8-bit kernels' sources that no run shows reliably."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_diffusion_transformer_b200", "csrc")


def test_no_load_that_asks_for_constant_memory():
    """Every 8-bit kernel may run beside the previous kernel of its stream, which may still be writing
    what this one reads after its wait. ld.global.nc (__ldg, const __restrict__) is defined only for
    memory that nothing writes during the kernel's life."""
    files = sorted(glob.glob(os.path.join(CSRC, "opq_fp8*.cu*")))
    assert len(files) >= 5
    for path in files:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)
        for word in (r"\b__ldg\b", r"global\.nc\b", r"\b__restrict__\b", r"\btex1Dfetch\b"):
            assert not re.search(word, code), (os.path.basename(path), word)
