"""The slot protocol of the dense readout's ring (csrc/dense_ring.h) on the CPU:
whatever the order in which the releases of different slots arrive, a wait for
round r - 1 ends only when that round has been released."""
import ctypes
import os
import random
import subprocess

import pytest

SLOTS = 8   # and as many dequantising warps
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_fp4_csa2_gb300", "csrc")


@pytest.fixture(scope="module")
def ring(tmp_path_factory):
    d = tmp_path_factory.mktemp("ring")
    src = d / "ring.cpp"
    src.write_text('#include "dense_ring.h"\nextern "C" {\nint sets() { return csa2::kRingSets; }\n'
                   "unsigned set_of(unsigned r) { return csa2::ring_set(r); }\n"
                   "unsigned parity_of(unsigned r) { return csa2::ring_parity(r); }\n}\n")
    so = d / "ring.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", f"-I{CSRC}", str(src), "-o", str(so)], check=True)
    return ctypes.CDLL(str(so))


def rounds_of(segments):
    """The rounds of segments of the given steps: K(0), then K(i + 1) and V(i)."""
    out = []
    for n in segments:
        out.append("K")
        for i in range(n):
            out += ["K", "V"] if i + 1 < n else ["V"]
    return out


class Ring:
    """One CTA's barriers.  Products end in order; the release of (round, slot)
    arrives at its barrier any time after that."""

    def __init__(self, sets, set_of, parity_of):
        self.set_of, self.parity_of = set_of, parity_of
        self.phases = [[0] * SLOTS for _ in range(sets)]   # completed phases of each barrier
        self.released = set()

    def arrive(self, r, s):
        self.phases[self.set_of(r)][s] += 1
        self.released.add((r, s))

    def passes(self, r, s):
        """mbarrier.try_wait.parity for the release of round r."""
        return (self.phases[self.set_of(r)][s] - 1) % 2 == self.parity_of(r)


def simulate(kinds, ring, rng, held):
    """Runs the warps, the issuing thread and the arrivals in random order; the
    releases that `held` names arrive only when nothing else can go on.
    Returns the waits that ended too early."""
    n = len(kinds)
    at = [(0, 0)] * SLOTS                    # each warp: (round, half of a K round)
    filled = [[0] * SLOTS for _ in range(n)]
    issued, pending, late = (0, 0), [], []
    early = []

    def ready(r, slots):
        if r == 0:
            return True
        if not all(ring.passes(r - 1, s) for s in slots):
            return False
        early.extend((r, s) for s in slots if (r - 1, s) not in ring.released)
        return True

    while True:
        moves = [("warp", w) for w in range(SLOTS) if at[w][0] < n]
        if issued[0] < n:
            moves.append(("issue", 0))
        moves += [("arrive", i) for i in range(len(pending))]
        rng.shuffle(moves)
        for what, i in moves:
            if what == "warp":
                r, half = at[i]
                if kinds[r] == "K":
                    slots = range(4 * half, 4 * half + 4)
                    if not ready(r, slots):
                        continue
                    for s in slots:
                        filled[r][s] += 1
                    at[i] = (r, 1) if half == 0 else (r + 1, 0)
                else:
                    if not ready(r, [i]):
                        continue
                    filled[r][i] += SLOTS
                    at[i] = (r + 1, 0)
            elif what == "issue":
                r, s = issued
                if filled[r][s] < SLOTS:
                    continue
                (late if (r, s) in held else pending).append((r, s))
                issued = (r, s + 1) if s + 1 < SLOTS else (r + 1, 0)
            else:
                ring.arrive(*pending.pop(i))
            break
        else:
            if not late:
                break
            ring.arrive(*late.pop(0))
        if early:
            return early
    assert all(a == (n, 0) for a in at) and issued == (n, 0), "the protocol stands still"
    return early


SEGMENTS = [[1], [1, 1, 1, 1], [4], [2, 1, 3], [3, 2, 2, 5]]


@pytest.mark.parametrize("segments", SEGMENTS)
def test_no_wait_ends_early(ring, segments):
    kinds = rounds_of(segments)
    for seed in range(12):
        simulate(kinds, Ring(ring.sets(), ring.set_of, ring.parity_of), random.Random(seed), ())
    for r in range(len(kinds)):
        for s in range(SLOTS):
            for held in ({(r, s)}, {(r, i) for i in range(SLOTS) if i != s}, {(r, i) for i in range(s, SLOTS)}):
                early = simulate(kinds, Ring(ring.sets(), ring.set_of, ring.parity_of), random.Random(r * SLOTS + s), held)
                assert not early, f"round {early[0][0]}, slot {early[0][1]}: filled before the round before was read"


def test_one_barrier_per_slot_is_not_enough():
    """The simulation finds the early wait that a single barrier per slot allows."""
    kinds = rounds_of([4])
    found = [simulate(kinds, Ring(1, lambda r: 0, lambda r: r % 2), random.Random(s), {(r, s)})
             for r in range(len(kinds)) for s in range(SLOTS)]
    assert any(found)
