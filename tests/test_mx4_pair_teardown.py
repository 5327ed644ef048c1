"""How a pair of CTAs of the 4-bit product leaves when its roles stop at any
point (csrc/mx4_settle.h), on the host: the stage barriers and the copies of a
pair are played through in random order, the roles stop where chance has it, and
the leader then has to know of every copy in flight, of either CTA, when it lands.
"""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from conftest import ROOT

ROLES, ARRIVALS, BYTES = 6, 5, 65536  # the leader's producer and four scale warps arrive

SHIM = """
#include "%s"
extern "C" void debt(const uint32_t *steps, uint32_t i, uint32_t bytes, uint32_t *arrivals, int32_t *tx)
{
    const exl3::MxDebt d = exl3::mx_debt(steps, i, bytes);
    *arrivals = d.arrivals;
    *tx = d.tx;
}
extern "C" void range(const uint32_t *steps, uint32_t stages, uint32_t *first, uint32_t *end)
{
    exl3::mx_debt_range(steps, stages, *first, *end);
}
extern "C" int roles() { return exl3::kMxRoles; }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("settle")
    src = d / "shim.cpp"
    src.write_text(SHIM % os.path.join(ROOT, "trellis_coded_bit_b200", "csrc", "mx4_settle.h"))
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-O1", "-shared", "-fPIC", "-o", str(d / "shim.so"), str(src)],
                   check=True)
    so = ctypes.CDLL(str(d / "shim.so"))
    assert so.roles() == ROLES
    return so


class Barrier:
    def __init__(self):
        self.pending, self.tx, self.phase = ARRIVALS, 0, 0

    def change(self, arrivals=0, tx=0):
        assert arrivals <= self.pending
        self.pending -= arrivals
        self.tx += tx
        if self.pending == 0 and self.tx == 0:
            self.pending, self.phase = ARRIVALS, self.phase + 1


class Pair:
    """Barriers full[stage] of the leader, the copies in flight as (step, CTA)."""

    def __init__(self, rng, stages, total):
        self.rng, self.stages, self.total = rng, stages, total
        self.full = [Barrier() for _ in range(stages)]
        self.steps, self.consumed, self.flying = [0] * ROLES, 0, []

    def land(self):
        step, _ = self.flying.pop(self.rng.randrange(len(self.flying)))
        self.full[step % self.stages].change(tx=-BYTES)

    def role(self, r):
        i = self.steps[r]
        if i == self.total or i - self.stages >= self.consumed:
            return
        bar = self.full[i % self.stages]
        if r == 0:
            bar.change(arrivals=1, tx=2 * BYTES)
        if r < 2:
            self.flying.append((i, r))
        else:
            bar.change(arrivals=1)
        self.steps[r] += 1

    def play(self, moves, living):
        for _ in range(moves):
            what = self.rng.randrange(ROLES + 2)
            if what < ROLES:
                if what in living:
                    self.role(what)
            elif what == ROLES:
                if self.flying:
                    self.land()
            elif "mma" in living and self.full[self.consumed % self.stages].phase > self.consumed // self.stages:
                self.consumed += 1

    def wait(self, step):
        """The wait for a step's phase: copies land meanwhile.  False: it never completes."""
        while self.full[step % self.stages].phase <= step // self.stages:
            if not self.flying:
                return False
            self.land()
        return True


def stopped_pair(seed):
    rng = random.Random(seed)
    pair = Pair(rng, rng.randint(2, 5), rng.randint(1, 14))
    living = list(range(ROLES)) + ["mma"]
    rng.shuffle(living)
    while living:  # one after the other stops, some at once
        pair.play(rng.choice([0, 1, 5, 40]), living)
        living.pop()
    return pair


def test_every_copy_has_landed(lib):
    seen = set()
    for seed in range(20000):
        pair = stopped_pair(seed)
        steps = (ctypes.c_uint32 * ROLES)(*pair.steps)
        first, end, arrivals, tx = ctypes.c_uint32(), ctypes.c_uint32(), ctypes.c_uint32(), ctypes.c_int32()
        lib.range(steps, pair.stages, ctypes.byref(first), ctypes.byref(end))
        for i in range(first.value, end.value):
            lib.debt(steps, i, BYTES, ctypes.byref(arrivals), ctypes.byref(tx))
            bar = pair.full[i % pair.stages]
            bar.change(tx=tx.value)
            for _ in range(arrivals.value):
                bar.change(arrivals=1)
            seen.add((arrivals.value, tx.value))
            assert pair.wait(i), (seed, i, pair.steps)
            assert all(step != i for step, _ in pair.flying)
        assert not pair.flying, (seed, pair.steps)
    # stopped in every way: either producer ahead, any number of arrivals missing
    assert {t for _, t in seen} == {0, BYTES, -BYTES} and {a for a, _ in seen} == set(range(ARRIVALS + 1))


def test_the_leaders_own_steps_are_not_enough():
    """Waiting for the steps that the leader itself began leaves copies of the
    other CTA in flight: what the counts of both are for."""
    left = 0
    for seed in range(20000):
        pair = stopped_pair(seed)
        for i in range(max(0, pair.steps[0] - pair.stages), pair.steps[0]):
            if pair.full[i % pair.stages].phase <= i // pair.stages:
                pair.flying = [f for f in pair.flying if f[0] != i]  # landed, or waited for until the limit
        left += bool(pair.flying)
    assert left > 0
