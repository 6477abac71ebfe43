"""Kernels that start while their predecessor drains read nothing through the
read-only path: what they read may have been written meanwhile."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "static_kv_cache_gb300", "csrc")


def test_no_read_only_loads():
    files = sorted(glob.glob(os.path.join(CSRC, "*.cu*")))
    assert files
    for f in files:
        with open(f) as src:
            for i, line in enumerate(src, 1):
                code = line.split("//")[0]
                assert not re.search(r"__ldg\b|\.nc\b|__restrict", code), f"{os.path.basename(f)}:{i}: {line.strip()}"
