"""Rules that every kernel source keeps."""
import glob
import os
import re

from mixture_experts_layer_57_b200 import build


def test_no_read_only_loads():
    # Kernels start while the one before them may still be writing (programmatic dependent launch), so
    # no tensor is read-only for a kernel's whole lifetime, which the non-coherent load path asks for;
    # its loads may also be moved above the wait.
    files = glob.glob(os.path.join(build.CSRC, "*.cu*"))
    assert len(files) >= 15
    for path in files:
        found = re.findall(r"__ldg\w*\(|ld\.global\.nc", open(path).read())
        assert not found, (os.path.basename(path), found)
