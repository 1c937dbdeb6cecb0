"""Edges of the window writer, the read-backs and the dense readouts."""
import math

import pytest
import torch

from test_gpu_cache_dense import (D, ENTRY, H, attend64, c2, check_out, entries, gen, kv64, prefix_inputs, prefix_ref,  # noqa: F401
                                  queries, run_cross, run_prefix)

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


# ----------------------------------------------------------------- reading
def bf16_of(v):
    """64-bit values rounded once to bf16 (nearest even), as 64-bit values."""
    step = torch.exp2((torch.frexp(v).exponent - 8).clamp_min(-133).double())
    r = torch.round(v / step) * step
    return torch.where(r.abs() > float(torch.finfo(torch.bfloat16).max), torch.copysign(torch.full_like(r, math.inf), r), r)


def test_swa_read_rounds_once(c2):  # noqa: F811
    """Scales that put code x scale next to the middle of two bf16 values, from
    subnormal products to the largest, and every finite code."""
    g = gen(130)
    codes = torch.tensor([c for c in range(256) if c & 127 != 127], dtype=torch.uint8, device="cuda")
    val = codes.view(torch.float8_e4m3fn).double()
    n = 4000
    pick = torch.randint(0, codes.numel(), (n,), generator=g, device="cuda")
    mid = (torch.randint(128, 256, (n,), generator=g, device="cuda").double() + 0.5) * torch.exp2(
        torch.randint(-140, 120, (n,), generator=g, device="cuda").double())
    mid[:8] = torch.tensor([0.0, 2.0 ** -149, 2.0 ** -134, 3.4e38, 0.094815336 * 11, 0.88920456 * 11, 1.0, 2.0 ** -126], dtype=torch.float64)
    pick[4:6] = int((val == 11).nonzero()[0])
    scale = torch.where(val[pick] != 0, mid / val[pick].abs().clamp_min(2.0 ** -9), mid).float().abs()
    swa = codes[torch.randint(0, codes.numel(), (n, D), generator=g, device="cuda")]
    swa[:, :codes.numel()] = codes
    swa[:, 300:400] = codes[pick][:, None]
    out = torch.empty(1, n, D, dtype=torch.bfloat16, device="cuda")
    c2.swa_read(swa.view(1, n, D), scale.view(1, n), out)
    exact = swa.view(torch.float8_e4m3fn).double() * scale.double()[:, None]   # 28 bits
    want = bf16_of(exact)
    nan = torch.isnan(want)   # zero codes under the few scales that overflow to infinity
    assert torch.equal(torch.isnan(out[0]), nan)
    assert torch.equal(out[0].double()[~nan], want[~nan])
    assert torch.equal(torch.signbit(out[0])[~nan], torch.signbit(exact)[~nan])
    # the case is worth its name: a product rounded to fp32 first gives other values
    assert (exact.float().bfloat16().double() != want)[~nan].any()


def test_swa_read_infinities_and_nans(c2):  # noqa: F811
    swa = torch.zeros(1, 3, D, dtype=torch.uint8, device="cuda")
    swa[..., 1], swa[..., 2], swa[..., 3] = 0x38, 0xB8, 0x7F   # 1, -1, NaN
    out = torch.empty(1, 3, D, dtype=torch.bfloat16, device="cuda")
    c2.swa_read(swa, torch.tensor([[1.0, math.inf, math.nan]], device="cuda"), out)
    assert out[0, 0, 1] == 1 and out[0, 0, 2] == -1 and torch.isnan(out[0, 0, 3])
    assert out[0, 1, 1] == math.inf and out[0, 1, 2] == -math.inf and torch.isnan(out[0, 1, [0, 3]]).all()
    assert torch.isnan(out[0, 2]).all()


# ------------------------------------------------------------------- dense
# factors on the queries (of the head's sharpness, 0.5 to 3) and the entries'
# standard deviation: next to no logits at all, the usual ones, one key that takes
# everything, logits past 2^28 (where a step of fp32 is whole powers of e)
SCALES = [(1e-3, 1.0), (1.0, 0.01), (0.05, 100.0), (300.0, 30.0), (20000.0, 800.0)]


@pytest.mark.parametrize("q_scale,std", SCALES)
def test_cross_attn_of_any_size(c2, q_scale, std):  # noqa: F811
    n, T = 1500, 3
    kv = entries(c2, n, 100, std)
    q = (queries((1, T), 101).float() * q_scale).clamp(-65000, 65000).bfloat16()
    out, lse = run_cross(c2, q, kv.view(1, n, ENTRY), torch.tensor([n], dtype=torch.int32, device="cuda"), n)
    assert c2.get_device_status() == 0
    check_out(out, lse, *attend64(q[0].double().view(-1, D), kv64(kv)))


@pytest.mark.parametrize("q_scale,std", SCALES)
def test_prefix_attn_of_any_size(c2, q_scale, std):  # noqa: F811
    p, q, pre, kv, idx, swa, sc, sl = prefix_inputs(c2, 3, 900, 64, 16, 110, [(64, 16), (0, 0), (5, 1)])
    pre = entries(c2, 900, 111, std)
    kv = entries(c2, kv.shape[0] * kv.shape[1], 112, std).view_as(kv)
    sc = sc * std
    q = (q.float() * q_scale).clamp(-65000, 65000).bfloat16()
    args = (q, pre, kv, idx, swa, sc, sl)
    out, lse = run_prefix(c2, p, *args)
    assert c2.get_device_status() == 0
    check_out(out, lse, *prefix_ref(*args))


@pytest.mark.parametrize("prefix", [False, True])
def test_logits_past_two_to_the_29(c2, prefix):  # noqa: F811
    """Queries and entries near the ends of their ranges: each head's logit for
    one key, or for two equal ones, is about 3e9, the others' far below, and the
    output is that key."""
    n, K = 700, 64
    g = gen(120)
    sign = torch.where(torch.rand(H, D, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    lat = torch.randn(n, D, generator=g, device="cuda") * 20
    at = torch.randperm(n - 1, generator=g, device="cuda")[:H]
    lat[at] = sign * 2000
    lat[n - 1] = lat[at[0]]            # head 0 has two
    pre = torch.zeros(n, ENTRY, dtype=torch.uint8, device="cuda")
    rows = torch.arange(n, device="cuda")
    c2.kv_quant_write(lat.bfloat16(), None, 1, torch.zeros_like(rows), rows, pre)
    q = (sign * 60000).bfloat16()[None]
    if prefix:
        p, _, _, kv, idx, swa, sc, sl = prefix_inputs(c2, 1, 0, K, 8, 121)
        args = (q, pre, kv, idx, swa, sc, sl)
        out, lse = run_prefix(c2, p, *args)
        ref = prefix_ref(*args)
    else:
        out, lse = run_cross(c2, q[None], pre[None], torch.tensor([n], dtype=torch.int32, device="cuda"), n)
        ref = attend64(q[0].double(), kv64(pre))
    assert c2.get_device_status() == 0
    check_out(out, lse, *ref)
