"""Kernels here start while the ones before them still run (programmatic
dependent launch).  What those may write is not read-only for a kernel's whole
life, so it must not come through the non-coherent load path."""

import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# the weights of the projections, which include/mla.h documents as read during the launch overlap
CONSTANT = {"decode.cu": ["__ldg(w + c * (kDv / 2))"] * 2,
            "absorb.cu": ["const uint16_t* __restrict__ w_uk", "const uint16_t* __restrict__ w_uv"] * 2}


def test_non_coherent_loads_are_of_constant_data():
    files = sorted(glob.glob(os.path.join(ROOT, "mla_latent_kv_append_gb300", "csrc", "*.cu*")))
    assert files
    for f in files:
        code = re.sub(r"//[^\n]*", "", open(f, encoding="utf-8").read())
        rest = code
        for use in CONSTANT.get(os.path.basename(f), []):
            assert use in rest, use
            rest = rest.replace(use, "", 1)
        assert "__ldg" not in rest and "ld.global.nc" not in rest and ".nc." not in rest, os.path.basename(f)
        # a read-only restrict pointer lets the compiler take that path by itself
        assert not re.search(r"const\s+\w+\s*\*\s*__restrict__", rest), os.path.basename(f)
