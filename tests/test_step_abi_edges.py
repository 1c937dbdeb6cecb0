"""More host-side refusals of the slot maps, without a GPU."""
import ctypes

import pytest

from test_step_abi import INVALID, c2  # noqa: F401

NAMES = ["ctx", "new", "cu", "tok", "pos", "swa", "ecu", "epos", "slot", "vis", "len"]
SIZES = {"cu": 12, "ecu": 12, "vis": 8, "len": 8, "tok": 40, "pos": 80, "swa": 80, "epos": 80, "slot": 80}   # bytes, batch 2, 10 places


@pytest.mark.parametrize("name", SIZES)
@pytest.mark.parametrize("length", ["ctx", "new"])
def test_slot_map_outputs_apart_from_the_lengths(c2, name, length):  # noqa: F811
    """Outputs that share a word with the lengths, which other CTAs may still read: the same
    memory (lengths updated in place), the output's last word, the lengths' last one."""
    at = {n: 0x10000 * (i + 1) for i, n in enumerate(NAMES)}   # never dereferenced: the checks fail first
    for where in (0, SIZES[name] - 4, -4):
        a = at | {length: at[name] + where}
        out = (ctypes.c_void_p * 9)(*[a[n] for n in NAMES[2:]])
        assert c2.lib().csa2_slot_map(2, a["ctx"], a["new"], 1, 100, 128, 10, 10, ctypes.addressof(out), None) == INVALID
        assert c2.last_launch_count() == 0
