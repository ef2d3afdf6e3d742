"""Rules that the CUDA sources keep, read as text (no GPU)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "codebook_token_sampling_gb300", "csrc")


def test_no_copy_is_multicast():
    """The library is loaded by programs of several GPUs: no bulk or tensor copy goes to more
    than one CTA's shared memory."""
    found = [path for path in glob.glob(os.path.join(CSRC, "*.cu*"))
             for copy in re.findall(r"cp\.(?:reduce\.)?async\.bulk[^;]*;", open(path).read()) if "multicast" in copy]
    assert not found
