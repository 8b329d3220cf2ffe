"""Shared memory that a kernel reads in 16-byte pieces declares that alignment.

A float array without it may start at any multiple of four bytes; where it lies
is the compiler's choice, which other arrays' sizes change.
"""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "deltanet_sequence_mixing_b200", "csrc")


@pytest.mark.parametrize("name", sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*.cu"))))
def test_declared(name):
    text = open(os.path.join(CSRC, name)).read()
    if not re.search(r"reinterpret_cast<(const )?(float4|uint4)\s*\*>", text):
        return
    for decl in re.findall(r"extern __shared__ [^;]*;", text):
        # bytes are rounded up to the swizzle's 1024 by hand
        assert "__align__(" in decl or "uint8_t smem_raw[]" in decl or "tsolve_smem_raw[]" in decl, decl
    for array in re.findall(r"reinterpret_cast<(?:const )?float4\s*\*>\(&(\w+)\[", text):
        decls = [d for d in re.findall(r"__shared__ [^;]*;", text) if re.search(r"\b%s\[" % array, d)]
        assert decls and all("__align__(16)" in d for d in decls), (array, decls)
