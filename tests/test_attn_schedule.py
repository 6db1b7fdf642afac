"""The order of sends, waits, barriers and reads in the tree attention's tile loops: the header that the
kernel walks, run on the CPU against a model of LDS (attn_schedule_model.cpp)."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "tree_masked_gated_amd", "csrc")


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("schedule") / "model")
    p = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wno-unknown-pragmas", "-I", CSRC,
                        os.path.join(HERE, "attn_schedule_model.cpp"), "-o", exe], capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
    return lambda *args: subprocess.run([exe, *map(str, args)], capture_output=True, text=True)


@pytest.mark.parametrize("uneven", [0, 1])
@pytest.mark.parametrize("loop,slots", [("turns", 3), ("step", 2), ("step", 3)])
def test_every_read_is_waited_for(model, loop, slots, uneven):
    """1 to 24 tiles: each read finds its tile, from every wave that sends a part of it."""
    p = model(loop, slots, uneven, "none")
    assert p.returncode == 0 and "72 runs, 0 faults" in p.stdout, p.stdout


def test_values_read_ahead_need_a_wait_of_their_own(model):
    """Without the wait that ends a first half, the leading waves read V before the trailing waves' share
    of it has arrived."""
    p = model("turns", 3, 0, "wait_k")
    assert p.returncode == 1 and "V of tile 3: read before it has arrived" in p.stdout, p.stdout


@pytest.mark.parametrize("loop,slots", [("turns", 3), ("step", 3)])
def test_the_model_misses_a_dropped_wait(model, loop, slots):
    p = model(loop, slots, 0, "wait_sent")
    assert p.returncode == 1 and "read before it has arrived" in p.stdout, p.stdout
