"""Shared arrays of elements narrower than a word say their alignment: wider accesses to them are
aligned by their declaration, not by where the compiler happens to place them (read from the
sources; no GPU needed).  Dynamic shared memory is aligned by its kernels."""
from __future__ import annotations

import glob
import os
import re

import mixture_experts_ffn_renorm_gb300 as m

CSRC = os.path.join(os.path.dirname(os.path.abspath(m.__file__)), "csrc")


def test_narrow_shared_arrays_are_aligned():
    narrow = re.compile(r"^(?!.*\bextern\b)(?!.*__align__).*__shared__\s+(?:u?int8_t|u?int16_t|char|__half|__nv_bfloat16)\b")
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        for n, line in enumerate(open(path), 1):
            if narrow.match(line):
                found.append(f"{os.path.basename(path)}:{n}: {line.strip()}")
    assert not found, found
