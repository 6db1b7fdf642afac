"""LDS arrays of the rule's kernels state the alignment that their 16-byte reads and sends need; without it the
compiler may place them at any multiple of an element.  CPU only: the declarations are read from the source."""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tree_masked_gated_amd", "csrc",
                      "rule_kernels.hpp")


def test_arrays_of_small_elements_are_aligned():
    text = re.sub(r"//.*", "", open(SOURCE).read())
    arrays = [d for d in re.findall(r"__shared__([^;]*);", text) if "[" in d and not re.match(r"\s*double\b", d)]
    assert len(arrays) >= 8
    assert not [d for d in arrays if "aligned(16)" not in d]
