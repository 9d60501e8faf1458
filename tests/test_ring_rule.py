"""The rule of the rings in shared memory, compiled for the host: a set of warps that takes every so many-th use of a ring waits on
barriers whose every use is its own. A parity tells a use only from the one before on its barrier."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "post_weight_quantization_gb300", "csrc")


@pytest.fixture(scope="module")
def barriers_for(tmp_path_factory):
    d = tmp_path_factory.mktemp("ring")
    (d / "ring.cpp").write_text('#include "ring.h"\nextern "C" int barriers(int places, int step) { return gptq::barriers_for(places, step); }\n')
    subprocess.run([os.environ.get("CXX") or "g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(d / "ring.cpp"), "-o", str(d / "ring.so")],
                   check=True)
    return ctypes.CDLL(str(d / "ring.so")).barriers


def sees_every_use(barriers, step, uses=600):
    """Whether a set that waits for every step-th use has waited for the one before on the barrier each time."""
    waited = set(range(0, uses, step))
    return all(n - barriers in waited for n in waited if n >= barriers)


def test_each_barrier_is_one_sets(barriers_for):
    for places in range(1, 13):
        for step in range(1, 13):
            b = barriers_for(places, step)
            assert b >= places and sees_every_use(b, step), (places, step, b)
            assert not any(sees_every_use(n, step) for n in range(places, b)), (places, step, b)     # and none too many


def test_three_places_and_a_step_of_two(barriers_for):
    assert not sees_every_use(3, 2) and barriers_for(3, 2) == 4
    assert barriers_for(2, 2) == 2 and barriers_for(4, 2) == 4 and barriers_for(3, 4) == 4 and barriers_for(3, 1) == 3


def test_a_copy_that_lands_late_is_taken_for_another(barriers_for):
    """What the rule keeps away, step by step: three places, a set that takes blocks 0, 2, 4, ... and another for the rest. Block 1
    is still on its way when the first set asks for block 4, which comes into block 1's place."""
    def ready_after(landings, barriers):
        uses = [0] * barriers                                # uses of each barrier that are complete
        for block in landings:
            uses[block % barriers] += 1
        return lambda block: uses[block % barriers] % 2 != block // barriers % 2     # a parity: the present use is not that one
    ready = ready_after([0, 2], 3)
    assert ready(0) and ready(2) and not ready(1)
    assert ready(4)                                          # wrongly: its place has not even block 1
    ready = ready_after([0, 2], barriers_for(3, 2))
    assert ready(0) and ready(2) and not ready(1) and not ready(4)
