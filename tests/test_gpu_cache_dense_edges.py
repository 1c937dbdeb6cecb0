"""Edges of the window writer, the read-backs and the dense readouts."""
import math

import pytest
import torch

from test_gpu_cache_dense import D, c2  # noqa: F401

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------- writing
@pytest.mark.parametrize("n", [6, 1500])
def test_swa_write_nan_beside_zeros(c2, n):  # noqa: F811
    """A row that holds nothing but NaNs and zeros keeps its NaNs: also one that
    RoPE makes of two infinities (inf x cos 0 - inf x sin 0)."""
    lat = torch.zeros(n, D, device="cuda")
    lat[0] = math.nan
    lat[1, 7] = math.nan
    lat[2, 510] = -math.nan
    lat[3, 448:450] = math.inf
    lat[4, 3] = -0.0
    pos = torch.zeros(n, dtype=torch.int64, device="cuda")
    swa = torch.full((n, D), 0x5A, dtype=torch.uint8, device="cuda")
    scale = torch.full((n,), -3.0, device="cuda")
    c2.swa_quant_write(lat.bfloat16(), torch.arange(n, device="cuda"), swa, scale, pos=pos)
    assert c2.get_device_status() == 0
    # the rotation of pair 255 makes a NaN of both its channels
    want = torch.zeros(n, D, dtype=torch.bool, device="cuda")
    want[0] = True
    want[1, 7] = True
    want[2, 510:] = True
    want[3, 448:450] = True
    assert torch.equal((swa & 127) == 127, want) and (swa[~want] == 0).all()
    out = torch.empty(1, n, D, dtype=torch.bfloat16, device="cuda")
    c2.swa_read(swa.view(1, n, D), scale.view(1, n), out)
    assert torch.equal(torch.isnan(out[0]), want) and (out[0][~want] == 0).all()
