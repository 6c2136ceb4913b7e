"""What the library's sources must not hold, whatever the GPU."""

import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_load_writes_another_block():
    """A bulk load with cluster multicast must only ever read this GPU's own
    memory, which a library that takes its callers' addresses, and that runs on
    several GPUs are served with, cannot know: there is none."""
    files = sorted(glob.glob(os.path.join(ROOT, "mla_latent_kv_append_gb300", "csrc", "*.cu*")))
    assert files
    for f in files:
        code = re.sub(r"//[^\n]*", "", open(f, encoding="utf-8").read())
        assert ".multicast" not in code, os.path.basename(f)
