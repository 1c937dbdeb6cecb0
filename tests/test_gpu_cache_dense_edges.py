"""Edges of the window writer, the read-backs and the dense readouts: NaNs among
zeros, exact rounding, queries and entries of any size, offsets past 2^32 bytes,
calls behind the kernels that write their inputs, in graphs and with events."""
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


# ----------------------------------------------- offsets past 2^32 bytes
def test_cross_attn_and_read_past_4_gib(c2):  # noqa: F811
    """18 million entries (5.2 GB): sequence 5 starts past 2^32 bytes."""
    B, cap = 6, 3_000_000
    kv = torch.zeros(B, cap, ENTRY, dtype=torch.uint8, device="cuda")
    tail = entries(c2, 700, 140)
    kv[5, :700] = tail
    kv[0, :700] = tail.flip(0)   # what 32-bit offsets would reach, among others
    kv[5, cap - 3:] = tail[:3]
    q = queries((B, 1), 141)
    out, lse = run_cross(c2, q, kv, torch.tensor([0, 0, 0, 0, 0, 700], dtype=torch.int32, device="cuda"), 700)
    r, rl = attend64(q[5, 0].double(), kv64(tail))
    check_out(out[5], lse[5], r, rl)
    idx = torch.tensor([[cap - 1, 0, 699]] * B, dtype=torch.int32, device="cuda")
    back = torch.empty(B, 3, D, dtype=torch.bfloat16, device="cuda")
    c2.kv_read(kv, back, idx=idx)
    assert c2.get_device_status() == 0
    assert torch.equal(back[5].double(), kv64(tail[[2, 0, 699]]))


def test_prefix_of_15_million_entries(c2):  # noqa: F811
    """A prefix past 2^32 bytes whose last entries alone are not zero, with logits 0 for the others."""
    n = 15_000_000
    pre = torch.zeros(n, ENTRY, dtype=torch.uint8, device="cuda")
    tail = entries(c2, 700, 150, 2.0)
    pre[n - 700:] = tail
    p, q, _, kv, idx, swa, sc, sl = prefix_inputs(c2, 2, 0, 64, 16, 151, [(64, 16), (0, 0)])
    out, lse = run_prefix(c2, p, q, pre, kv, idx, swa, sc, sl)
    assert c2.get_device_status() == 0
    r, rl = prefix_ref(q, tail, kv, idx, swa, sc, sl)
    total = torch.logaddexp(rl, torch.full_like(rl, math.log(n - 700)))
    check_out(out, lse, r * torch.exp(rl - total)[..., None], total)


def test_window_rows_past_4_gib(c2):  # noqa: F811
    rows = 9_000_000   # 4.6 GB
    swa = torch.zeros(rows, D, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(rows, device="cuda")
    lat = torch.randn(3, D, generator=gen(160), device="cuda").bfloat16()
    at = torch.tensor([rows - 1, 8_500_000, 5], device="cuda")
    c2.swa_quant_write(lat, at, swa, scale)
    want = torch.zeros(3, D, dtype=torch.uint8, device="cuda"), torch.zeros(3, device="cuda")
    c2.swa_quant_write(lat, torch.arange(3, device="cuda"), *want)
    assert torch.equal(swa[at], want[0]) and torch.equal(scale[at], want[1])
    assert int(scale.count_nonzero()) == 3
    small, big = (torch.empty(1, 3, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c2.swa_read(want[0][None], want[1][None], small)
    c2.swa_read(swa[None], scale[None], big, idx=at.int()[None])
    assert c2.get_device_status() == 0 and torch.equal(small, big)


def test_indexer_keys_past_4_gib(c2):  # noqa: F811
    rows = 68_000_000   # code plane 4.35 GB, then the exponents
    ik = c2.indexer_k_fp4_cache(rows)
    k = torch.randn(3, 128, generator=gen(170), device="cuda").bfloat16()
    at = torch.tensor([rows - 1, 67_500_000, 5], device="cuda")
    c2.indexer_k_quant(k, at, ik)
    few = c2.indexer_k_fp4_cache(4)
    c2.indexer_k_quant(k, torch.arange(3, device="cuda"), few)
    small, big = (torch.empty(1, 3, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c2.indexer_k_read(few, small)
    c2.indexer_k_read(ik, big, idx=at.int()[None])
    assert c2.get_device_status() == 0 and torch.equal(small, big) and (big != 0).any()


# --------------------------------------- streams, graphs and neighbours
class Written:
    """Inputs of a prefix call that kernels right before it write: the query, the
    prefix's entries, the own entries and the window rows."""

    def __init__(self, c2, seed):  # noqa: F811
        self.c2, self.n, self.B, self.K, self.W = c2, 6000, 5, 64, 16
        self.p, self.q, self.pre, self.kv, self.idx, self.swa, self.sc, self.sl = prefix_inputs(c2, self.B, self.n, self.K, self.W, seed)
        self.lat = torch.zeros(self.n, D, dtype=torch.bfloat16, device="cuda")
        self.own = torch.zeros(self.kv.shape[0] * self.kv.shape[1], D, dtype=torch.bfloat16, device="cuda")
        self.win = torch.zeros(self.B * self.W, D, dtype=torch.bfloat16, device="cuda")
        self.qs = torch.zeros_like(self.q)
        self.at = [torch.arange(x.shape[0], device="cuda") for x in (self.lat, self.own, self.win)]
        self.out = torch.empty(self.B, H, D, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.empty(self.B, H, device="cuda")
        self.ws = c2.workspace(c2.OP_PREFIX, self.B, self.n, self.p)

    def fill(self, seed):
        g = gen(seed)
        for x in (self.lat, self.own, self.win, self.qs):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))

    def steps(self, last):
        """The writes in an order that ends with `last`, each a function."""
        c2, s = self.c2, self  # noqa: F811
        writes = {"q": lambda: s.q.copy_(s.qs),
                  "window": lambda: c2.swa_quant_write(s.win, s.at[2], s.swa, s.sc, pos=s.at[2]),
                  "own": lambda: c2.kv_quant_write(s.own, None, 1, s.at[1], s.at[1], s.kv),
                  "prefix": lambda: c2.kv_quant_write(s.lat, None, 1, s.at[0], s.at[0], s.pre)}
        call = lambda: c2.prefix_attn(s.p, s.q, s.pre, s.kv, s.idx, s.swa, s.sc, s.sl, s.out, s.ws, lse=s.lse)  # noqa: E731
        return [writes[k] for k in writes if k != last] + [writes[last], call]

    def result(self):
        return self.out.clone(), self.lse.clone()


@pytest.mark.parametrize("last", ["q", "window", "own", "prefix"])
def test_prefix_attn_behind_the_kernel_that_writes_its_inputs(c2, last):  # noqa: F811
    w = Written(c2, 180)
    for i in range(12):
        w.fill(181 + i)
        for f in w.steps(last):
            f()
            torch.cuda.synchronize()
        want = w.result()
        for x in (w.q, w.swa, w.sc, w.kv, w.pre, w.out, w.lse):
            x.zero_()
        for f in w.steps(last):
            f()
        for a, b in zip(w.result(), want):
            assert torch.equal(a, b)
    assert c2.get_device_status() == 0


@pytest.mark.parametrize("last", ["q", "prefix"])
def test_prefix_attn_in_a_graph(c2, last):  # noqa: F811
    """Writes and readout captured together and replayed on new inputs; two
    replays in a row share the workspace."""
    w = Written(c2, 200)
    w.fill(201)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        for f in w.steps(last):
            f()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            for f in w.steps(last):
                f()
    for i in range(6):
        w.fill(202 + i)
        for f in w.steps(last):
            f()
            torch.cuda.synchronize()
        want = w.result()
        for x in (w.q, w.swa, w.sc, w.kv, w.pre, w.out, w.lse):
            x.zero_()
        w.ws.fill_(0xFF)
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(w.result(), want):
            assert torch.equal(a, b)
    assert c2.get_device_status() == 0


def test_prefix_attn_with_profile_events(c2):  # noqa: F811
    """Events around the own part's kernel come between the two launches."""
    w = Written(c2, 220)
    w.fill(221)
    steps = w.steps("prefix")
    for f in steps:
        f()
    want = w.result()
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    b.record()
    c2.set_profile_events(1, a, b)   # the sparse readout
    try:
        for _ in range(5):
            w.pre.zero_()
            for f in steps:
                f()
            for x, y in zip(w.result(), want):
                assert torch.equal(x, y)
            assert a.elapsed_time(b) > 0
    finally:
        c2.set_profile_events(1, None, None)
    assert c2.get_device_status() == 0
