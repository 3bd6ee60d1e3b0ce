"""The drain of a pair of CTAs that gives up: csrc/drain.cuh compiled for the
CPU, against a model of the barriers it waits on."""
import ctypes
import itertools
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "dropless_grouped_gemm_gb300", "csrc")


@pytest.fixture(scope="module")
def drain(tmp_path_factory):
    d = tmp_path_factory.mktemp("drain")
    src = d / "drain.cpp"
    src.write_text('#include "drain.cuh"\n'
                   'extern "C" int drain(unsigned f, unsigned s, unsigned n, unsigned i) {\n'
                   "  const moe::StageDrain d = moe::stage_drain(f, s, n, i);\n"
                   "  return d.wait | d.parity << 1 | d.arrive << 2 | d.make_up << 3;\n}\n")
    so = str(d / "drain.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", so], check=True)
    f = ctypes.CDLL(so).drain

    def call(first, second, stages, stage):
        r = f(first, second, stages, stage)
        return {"wait": r & 1, "parity": r >> 1 & 1, "arrive": r >> 2 & 1, "make_up": r >> 3 & 1}
    return call


class Barrier:
    """One arrival a phase; the phase ends when it is there and no byte is due."""

    def __init__(self):
        self.phase, self.pending, self.due = 0, 1, 0

    def _step(self):
        if self.pending == 0 and self.due == 0:
            self.phase, self.pending = self.phase + 1, 1

    def arrive(self, expect):
        assert self.pending == 1, "a second arrival in a phase"
        self.pending, self.due = 0, self.due + expect
        self._step()

    def bytes(self, n):
        self.due -= n
        self._step()

    def passed(self, parity):
        return self.phase & 1 != parity


def _give_up(drain, stages, used, first, second, rng):
    """Loads of both CTAs in their order, those before `used` landed; then the
    drain, with the others landing one by one in any order."""
    bars = [Barrier() for _ in range(stages)]
    for j in range(used):
        bars[j % stages].arrive(2)
        bars[j % stages].bytes(1)
        bars[j % stages].bytes(1)
    flying = []
    for j in range(used, max(first, second)):
        if j < first:
            bars[j % stages].arrive(2)
            flying.append(j % stages)
        if j < second:
            flying.append(j % stages)
    rng.shuffle(flying)
    early = rng.randrange(len(flying) + 1)
    for s in flying[:early]:
        bars[s].bytes(1)
    late = flying[early:]
    plan = [drain(first, second, stages, s) for s in range(stages)]
    for b, p in zip(bars, plan):
        if p["make_up"]:
            b.bytes(1)
        if p["arrive"]:
            b.arrive(1)
    while True:
        for s in range(stages):
            done = not plan[s]["wait"] or bars[s].passed(plan[s]["parity"])
            assert done == (s not in late), (stages, used, first, second, s, late)
        if not late:
            return
        bars[late.pop()].bytes(1)


@pytest.mark.parametrize("stages", [1, 2, 4, 6])
def test_waits_for_every_copy_in_flight_and_for_nothing_else(drain, stages):
    rng = random.Random(stages)
    for used in range(3 * stages + 1):
        for x, y in itertools.product(range(stages + 1), repeat=2):
            for _ in range(4):
                _give_up(drain, stages, used, used + x, used + y, rng)


def test_one_cta_alone(drain):
    for stages in (3, 4, 11):
        for n in range(40):
            for s in range(stages):
                loads = len([j for j in range(n) if j % stages == s])
                assert drain(n, n, stages, s) == {"wait": int(loads > 0), "parity": (loads - 1) & 1,
                                                  "arrive": 0, "make_up": 0}
