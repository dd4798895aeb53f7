"""Local arrays of the CUDA sources that are read or written in 16-byte words are declared so.

A local array has its element's alignment and no more; where the compiler keeps it in memory, a
16-byte access to one of BF16 values can be off its alignment and fault.
"""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "rank_binary_factorization_b200", "csrc")
WIDE = r"(?:u?int4|float4|double2|u?longlong2)"


def _unaligned_locals(src):
    src = re.sub(r"//.*", "", src)
    bad = []
    for m in re.finditer(rf"reinterpret_cast<(?:const )?{WIDE} \*>\((&?)(\w+)\b(\[?)", src):
        ref, name, element = m.groups()
        if element and not ref:         # an element that is itself an address
            continue
        # the nearest declaration of an array of that name before the cast
        decls = list(re.finditer(rf"([^;{{}}\n]*)\b{name}\[[^\];]*\](?:\[[^\];]*\])*\s*(?=[;,=])", src[:m.start()]))
        decls = [d for d in decls if re.match(r"\s*(?:__align__\(\d+\) |__shared__ |constexpr |const )*\w[\w:]* (?!.*[=(])", d.group(1))]
        if decls:
            d = decls[-1].group(1)
            if "__align__(" not in d and not re.search(rf"\b{WIDE}\b", d):
                bad.append((name, d.strip()))
    return bad


def test_the_check_sees_what_it_is_for():
    assert _unaligned_locals("T v[16];\nreinterpret_cast<const uint4 *>(v)[0];")
    assert not _unaligned_locals("__align__(16) T v[16];\nreinterpret_cast<const uint4 *>(v)[0];")
    assert not _unaligned_locals("uint4 raw[2];\nreinterpret_cast<const uint4 *>(raw)[0];")
    assert not _unaligned_locals("void f(const T *p) { reinterpret_cast<const uint4 *>(p)[0]; }")


@pytest.mark.parametrize("name", sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*.cu*"))))
def test_local_arrays_read_in_wide_words_are_aligned(name):
    assert not _unaligned_locals(open(os.path.join(CSRC, name)).read())
