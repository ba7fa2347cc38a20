"""Latent attention on the host: promises of the calls that need no GPU to be checked."""
import glob
import os
import re

import pytest

from linear_attention_06_gb300 import build as kbuild


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(kbuild.CSRC, "kda_latent_*.cu*"))), ids=os.path.basename)
def test_overlapped_kernels_read_nothing_as_read_only_data(path):
    """These kernels may be resident while the kernel before them still writes what they read, so no load of theirs
    may go through the read-only path, which promises memory that nobody writes while the kernel lives."""
    with open(path) as f:
        code = re.sub(r"//.*", "", f.read())
    assert not re.search(r"__ldg\b|ld\.global(\.\w+)*\.nc|__restrict__", code)
