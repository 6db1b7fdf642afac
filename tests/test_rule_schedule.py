"""The rows that the rule's scans request ahead: the header that the kernels walk, run on the CPU
(rule_schedule_model.cpp)."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "tree_masked_gated_amd", "csrc")


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("schedule") / "model")
    p = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", CSRC, os.path.join(HERE, "rule_schedule_model.cpp"),
                        "-o", exe], capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
    return lambda *args: subprocess.run([exe, *map(str, args)], capture_output=True, text=True)


@pytest.mark.parametrize("walk", ["forward", "back"])
def test_no_row_past_the_sequence_is_requested(model, walk):
    lengths = [0, 1, 2, 5, 63, 64, 65, 127, 128, 129, 200, 4096, 6727]
    p = model(walk, *lengths)
    assert p.returncode == 0 and f"{len(lengths)} lengths, 0 faults" in p.stdout, p.stdout
