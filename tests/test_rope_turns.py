"""The window writer's RoPE phases (csrc/rope_turns.h) on the CPU, against exact
arithmetic: behind by less than 2^-39 rad for every position below 2^22, next
to zeros of cos and sin too."""
import ctypes
import os
import subprocess
from fractions import Fraction

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_fp4_csa2_gb300", "csrc")


@pytest.fixture(scope="module")
def rope(tmp_path_factory):
    d = tmp_path_factory.mktemp("rope")
    (d / "rope.cpp").write_text('''#include "rope_turns.h"
extern "C" {
void steps(float theta, unsigned long long *out) {
  const csa2::RopeTurns t = csa2::rope_turns(theta);
  for (int j = 0; j < csa2::kRopePairs; ++j) out[j] = t.step[j];
}
float phase(unsigned long long step, long long p, unsigned *quarter) { return csa2::rope_phase(step, p, *quarter); }
}
''')
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", f"-I{CSRC}", str(d / "rope.cpp"), "-o", str(d / "rope.so")],
                   check=True)
    lib = ctypes.CDLL(str(d / "rope.so"))
    lib.steps.argtypes = [ctypes.c_float, ctypes.POINTER(ctypes.c_ulonglong)]
    lib.phase.argtypes, lib.phase.restype = [ctypes.c_ulonglong, ctypes.c_longlong, ctypes.POINTER(ctypes.c_uint)], ctypes.c_float
    return lib


def inverse_two_pi(bits=320):
    """floor(2^bits / (2 pi)) by Machin's formula in integers."""
    one = 1 << (bits + 64)

    def atan_inv(n):
        total, term, k = 0, one // n, 0
        while term:
            total += (-1) ** k * (term // (2 * k + 1))
            term //= n * n
            k += 1
        return total
    pi = 4 * (4 * atan_inv(5) - atan_inv(239))
    return (one << bits) // (2 * pi)


INV_TWO_PI, BITS = inverse_two_pi(), 320


def turns(inv, p):
    """p * inv / (2 pi) modulo one, exact but for 2^-270."""
    m, e = np.float32(inv).item().as_integer_ratio()
    return Fraction(p * m * INV_TWO_PI, e << BITS) % 1


@pytest.mark.parametrize("theta", [10000.0, 500000.0, 1.5, 3e38])
def test_phase(rope, theta):
    steps = (ctypes.c_ulonglong * 32)()
    rope.steps(theta, steps)
    rng = np.random.default_rng(3)
    worst = 0.0
    for j in range(32):
        inv = np.float32(np.float64(np.float32(theta)) ** (-2.0 * j / 64))
        at = [0, 1, 2, (1 << 22) - 1, (1 << 21) + 1, *rng.integers(0, 1 << 22, 60).tolist()]
        if theta == 10000.0:   # rotations next to a quarter turn: results of 1.6e-8 and the like
            at += {16: [2970533], 26: [3078233]}.get(j, [])
        for p in at:
            q = ctypes.c_uint(99)
            rest = rope.phase(steps[j], p, ctypes.byref(q))
            assert q.value < 4 and abs(rest) <= 0.25
            got = Fraction(q.value, 4) + Fraction(rest) / 2
            err = (got - turns(inv, p) + Fraction(1, 2)) % 1 - Fraction(1, 2)
            # the rounding of the rest to fp32 aside
            err = max(abs(err) - abs(Fraction(rest)) / 2 / 2 ** 24, 0) * 2 * Fraction(355, 113)
            worst = max(worst, float(err))
    assert worst <= 2.0 ** -39, worst


def test_steps_are_floors(rope):
    steps = (ctypes.c_ulonglong * 32)()
    rope.steps(10000.0, steps)
    for j in range(32):
        inv = np.float32(10000.0 ** (-2.0 * j / 64))
        exact = turns(inv, 1) * 2 ** 64
        assert 0 <= exact - steps[j] < 1 + Fraction(1, 2 ** 20)
