"""What the CUDA sources may not contain, read as text."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "comm_overlap_gb300", "csrc")
FILES = sorted(f for pattern in ("*.cu", "*.cuh", "*.h") for f in glob.glob(os.path.join(CSRC, pattern)))


def code(path):
    """The file without its comments."""
    with open(path, encoding="utf-8") as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_bulk_copies_are_not_multicast(path):
    """The library also runs on several GPUs and takes any device address: no copy goes to other CTAs' memory by
    multicast.  (A barrier's multicast arrive, tcgen05.commit, is no copy.)"""
    for asm in re.findall(r"\basm\b[^;]*?\((.*?)\)\s*;", code(path), flags=re.S):
        text = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', asm))
        assert not ("cp.async.bulk" in text and ".multicast" in text), text


@pytest.mark.parametrize("path", [f for f in FILES if "pdl_wait()" in code(f)], ids=os.path.basename)
def test_dependent_kernels_read_with_ordinary_loads(path):
    """A kernel that starts before its predecessor has ended may not declare what it reads read-only: such a load may
    come from a stale line, or be moved before the wait."""
    text = code(path)
    for word in (r"\b__ldg\b", r"\b__restrict__\b", r"\.nc\b"):
        assert not re.search(word, text), word
