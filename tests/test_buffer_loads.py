"""Bounds of the kernels' raw buffer loads, read from the sources.

The hardware's bounds check is promised for the vector offset and the immediate
only.  A kernel that leaves it to the check which rows are there must therefore
put the row into the vector offset: the scalar offset of every raw buffer load
is the literal 0."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(p for ext in ("hip", "h") for p in
                 glob.glob(os.path.join(ROOT, "ternary_weight_matmul_amd", "csrc", "*." + ext)))
# the place of the scalar offset among the arguments
CALL = re.compile(r"__builtin_amdgcn_(raw_buffer_load_\w+|raw_ptr_buffer_load_lds|raw_buffer_store_\w+)\s*\(")
PLACE = {"raw_buffer_load": 2, "raw_ptr_buffer_load_lds": 4, "raw_buffer_store": 3}


def arguments(text, start):
    """The arguments of a call whose opening bracket is just before `start`."""
    depth, args, begin = 0, [], start
    for i in range(start, len(text)):
        c = text[i]
        if c in "([{":
            depth += 1
        elif c in ")]}":
            if depth == 0:
                return args + [text[begin:i].strip()]
            depth -= 1
        elif c == "," and depth == 0:
            args.append(text[begin:i].strip())
            begin = i + 1
    raise AssertionError("unbalanced brackets")


def scalar_offsets(text):
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
    for m in CALL.finditer(text):
        place = next(v for k, v in PLACE.items() if m.group(1).startswith(k))
        yield arguments(text, m.end())[place]


def test_the_reader_finds_scalar_offsets():
    text = "f(__builtin_amdgcn_raw_buffer_load_b128(rsrc(p + u, n), at(i, 4), 8 * b, 0)); // __builtin_amdgcn_raw_buffer_load_b8(r, 1, 2, 0)"
    assert list(scalar_offsets(text)) == ["8 * b"]


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_scalar_offsets_are_zero(path):
    with open(path) as f:
        assert all(s == "0" for s in scalar_offsets(f.read()))


def test_there_are_buffer_loads_to_check():
    found = 0
    for path in SOURCES:
        with open(path) as f:
            found += len(list(scalar_offsets(f.read())))
    assert found >= 10
