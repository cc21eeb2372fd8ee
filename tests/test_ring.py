"""The copies that a staged row kernel still has to wait for when it gives up (csrc/ring.h), against a
step-by-step model of the kernel's ring for every place where it can stop.  Runs on the CPU."""
import ctypes
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_layer_48_b200", "csrc")
SOURCE = """
#include "ring.h"
extern "C" int issued(int lost, int stages, int steps) { return moe::ring_issued(lost, stages, steps); }
extern "C" int oldest(int issued, int stages) { return moe::ring_oldest(issued, stages); }
extern "C" int slot(int j, int stages) { return moe::ring_slot(j, stages); }
extern "C" int parity(int j, int stages) { return (int)moe::ring_parity(j, stages); }
"""


@pytest.fixture(scope="module")
def ring(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("ring")
    (d / "ring.cc").write_text(SOURCE)
    subprocess.run([cxx, "-shared", "-fPIC", "-I", CSRC, str(d / "ring.cc"), "-o", str(d / "ring.so")], check=True)
    return ctypes.CDLL(str(d / "ring.so"))


def _model(stages, steps, lost):
    """Phases of every stage's barrier that copies were issued for, and those waited for, when the
    wait of step `lost` gives up and the block goes through its other steps without copies."""
    issued = [[] for _ in range(stages)]     # parities, in order
    waited = [0] * stages

    def fetch(slot):
        issued[slot].append(len(issued[slot]) & 1)

    for s in range(min(stages, steps)):
        fetch(s)
    for i in range(steps):
        slot = i % stages
        if i < lost:
            waited[slot] += 1
            if i + stages < steps:
                fetch(slot)
    return issued, waited


@pytest.mark.parametrize("stages", [1, 2, 3, 4])
def test_a_block_that_gives_up_waits_for_what_it_issued(ring, stages):
    for steps in range(1, 14):
        for lost in range(steps):
            issued, waited = _model(stages, steps, lost)
            n = ring.issued(lost, stages, steps)
            assert n == sum(map(len, issued)), (stages, steps, lost)
            drained = [(ring.slot(j, stages), ring.parity(j, stages)) for j in range(ring.oldest(n, stages), n)]
            # one wait a stage at most, for the last phase that a copy was issued for: that parity is
            # complete only when the copy has landed, and every earlier phase was complete before
            assert len({s for s, _ in drained}) == len(drained)
            for s, parity in drained:
                assert parity == issued[s][-1], (stages, steps, lost, s)
            for s in range(stages):
                assert len(issued[s]) - waited[s] <= 1
                if len(issued[s]) > waited[s]:
                    assert s in {d for d, _ in drained}, (stages, steps, lost, s)


def test_the_old_rule_would_have_missed_copies():
    """Parities told from where the block's own reading had got to, which moves on after it gave up:
    what the model has to catch."""
    missed = 0
    for stages in (2, 3, 4):
        for steps in range(1, 9):
            for lost in range(steps):
                issued, waited = _model(stages, steps, lost)
                slot, phase = steps % stages, (steps // stages) & 1
                for s in range(stages):
                    parity = phase ^ 1 if s < slot else phase
                    missed += len(issued[s]) > waited[s] and parity != issued[s][-1]
    assert missed > 0
