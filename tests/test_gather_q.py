"""The hand-over of the queries in the gathered readout (csrc/gather_q.h) on the CPU:
whatever the order of copies, conversions and products, a role passes a wait only
when the phase that it waits for is complete, and none waits for ever."""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_fp4_csa2_gb300", "csrc")
WARPS = 8   # row warps, and the arrivals of a phase of q_ready


@pytest.fixture(scope="module")
def q(tmp_path_factory):
    d = tmp_path_factory.mktemp("gather_q")
    src = d / "q.cpp"
    src.write_text('#include "gather_q.h"\nextern "C" {\nint waits() { return csa2::kQWaits; }\n'
                   "int of_ready(unsigned n, int i) { return csa2::q_wait(n, i).ready; }\n"
                   "unsigned phase(unsigned n, int i) { return csa2::q_wait(n, i).phase; }\n}\n")
    so = d / "q.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", f"-I{CSRC}", str(src), "-o", str(so)], check=True)
    return ctypes.CDLL(str(so))


class Barrier:
    def __init__(self, count):
        self.count, self.arrived = count, 0

    def phases(self):
        return self.arrived // self.count

    def passes(self, phase):
        """mbarrier.try_wait.parity for this phase."""
        return (self.phases() - 1) % 2 == phase % 2


class Cta:
    """One CTA's roles as generators that yield what they wait for: (barrier, phase)."""

    def __init__(self, steps, waits):
        self.steps, self.waits = steps, waits
        self.raw, self.ready, self.q_free = Barrier(1), Barrier(WARPS), Barrier(1)
        self.rows, self.slot_free = [Barrier(WARPS) for _ in range(2)], [Barrier(1) for _ in range(2)]
        self.events = [self.raw]   # asynchronous completions on their way (the first token's copy)

    def row_warp(self):
        g = 0
        for n, steps in enumerate(self.steps):
            for s in range(steps):
                if g > 1:
                    yield self.slot_free[g & 1], (g >> 1) - 1
                self.rows[g & 1].arrived += 1
                if s == 0 and n:
                    for ready, phase in self.waits(n):
                        yield (self.ready if ready else self.raw), phase
                    self.ready.arrived += 1
                g += 1

    def softmax(self):
        yield self.raw, 0
        self.ready.arrived += WARPS

    def score(self):
        g = 0
        for n, steps in enumerate(self.steps):
            if n:
                yield self.q_free, n - 1
                self.events.append(self.raw)
            yield self.ready, n
            for s in range(steps):
                yield self.rows[g & 1], g >> 1
                self.events.append(self.slot_free[g & 1])   # (S, softmax and the second product of this step)
                if s == steps - 1:
                    self.events.append(self.q_free)
                g += 1


def simulate(steps, waits, rng, late):
    """Runs the roles in random order, `late`: copies land only when nothing else can
    go on.  The waits that ended too early, and whether every role came to its end."""
    cta = Cta(steps, waits)
    roles = [cta.row_warp() for _ in range(WARPS)] + [cta.softmax(), cta.score()]
    at = [next(r, None) for r in roles]
    early = []
    while any(at) or cta.events:
        moves = [("role", i) for i, w in enumerate(at) if w and w[0].passes(w[1])]
        events = [("event", i) for i, b in enumerate(cta.events)
                  # (products of one barrier end in order: only its first one)
                  if cta.events.index(b) == i and not (late and b is cta.raw and moves)]
        if not moves and not events:
            return early, False
        what, i = rng.choice(moves + events)
        if what == "event":
            cta.events.pop(i).arrived += 1
            continue
        barrier, phase = at[i]
        if barrier.phases() <= phase:
            early.append((i, phase))
        at[i] = next(roles[i], None)
    return early, True


CASES = [[1, 1], [1, 3, 1], [1] * 7, [2, 1, 1, 2], [3, 1, 1, 4, 1], [10, 10]]


@pytest.mark.parametrize("late", [False, True])
@pytest.mark.parametrize("steps", CASES, ids=str)
def test_waits_are_exact(q, steps, late):
    rng = random.Random(len(steps))
    for _ in range(200):
        early, ended = simulate(steps, lambda n: [(q.of_ready(n, i), q.phase(n, i)) for i in range(q.waits())], rng, late)
        assert not early and ended


def test_model_sees_a_missing_wait(q):
    """With the wait for the copy alone the model finds conversions before the copy."""
    rng, found = random.Random(1), False
    for _ in range(200):
        found |= bool(simulate([1, 1], lambda n: [(False, n)], rng, True)[0])
    assert found
