"""The FP8 window writer, the cache read-backs and the dense readouts
(cross_attn, prefix_attn) against plain 64-bit implementations on the host or
the GPU's fp64 units.

Tolerances.  A read-back is one product rounded to bf16: exact for main-KV
entries (6 significant bits) and MXFP4 keys (2), half a bf16 step (2^-8
relative) for window rows.  A written code may sit one E4M3 step from the
64-bit one only where x / scale lies within 2^-20 of a rounding border
(relative: RoPE's cos and sin to 2 ulp, three fp32 roundings of a rotation
and two divisions are below 16 x 2^-24).  A dense readout rounds each P to
fp16, independently for each key, so an output of standard deviation s over
its channels is off by 2^-11 / sqrt(3) s, and by five times that at the worst
of some 10^5 values; the row's largest of 512 channels is above 2 s, so 2^-9
of it is twice what five deviations need, which leaves room for the fp16
partials (2^-11 of a value).  The output's own rounding to bf16 adds 2^-8 of
each value.  The log-sum-exp is fp32 over fp32 logits: 2e-5 of it (or of 1).
"""
import ctypes
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

D, H, ENTRY = 512, 64, 288


@pytest.fixture(scope="module")
def c2():
    import sparse_attention_fp4_csa2_gb300.build as b
    b.build()
    import sparse_attention_fp4_csa2_gb300 as c
    return c


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def e2m1_64(b):
    c = torch.stack([b & 15, b >> 4], -1).flatten(-2).long()
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64,
                       device=b.device)
    return lut[c]


def kv64(kv):
    return e2m1_64(kv[..., :256]) * kv[..., 256:].contiguous().view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)


def entries(c2, rows, seed, std=1.0):
    """Main-KV entries written by the library itself from N(0, std^2) latents."""
    kv = torch.zeros(rows, ENTRY, dtype=torch.uint8, device="cuda")
    if rows:
        lat = (torch.randn(rows, D, generator=gen(seed), device="cuda") * std).bfloat16()
        at = torch.arange(rows, device="cuda")
        c2.kv_quant_write(lat, None, 1, at, at.clone(), kv)
    return kv


def queries(shape, seed):
    sharp = torch.linspace(0.5, 3.0, H, device="cuda").unsqueeze(-1)
    return (torch.randn(*shape, H, D, generator=gen(seed), device="cuda") * sharp).bfloat16()


def attend64(q, keys):
    """q [rows, 512], keys [n, 512] in 64 bits -> (out, lse)."""
    if keys.shape[0] == 0:
        return torch.zeros_like(q), torch.full(q.shape[:1], -math.inf, dtype=torch.float64, device=q.device)
    x = q @ keys.T / math.sqrt(D)
    lse = torch.logsumexp(x, -1)
    return torch.exp(x - lse[:, None]) @ keys, lse


def check_out(out, lse, ref, ref_lse):
    o, r = out.double().reshape(-1, D), ref.reshape(-1, D)
    tol = r.abs() * 2.0 ** -8 + r.abs().amax(-1, keepdim=True) * 2.0 ** -9
    assert torch.isfinite(o).all()
    assert ((o - r).abs() <= tol).all(), f"off by {((o - r).abs() - tol).max().item()}"
    l, rl = lse.double().reshape(-1), ref_lse.reshape(-1)
    empty = torch.isinf(rl)
    assert torch.equal(torch.isneginf(l), empty)
    err = (l - rl)[~empty].abs()
    assert (err <= 2e-5 * rl[~empty].abs().clamp_min(1.0)).all(), f"lse off by {err.max().item()}"


# ----------------------------------------------------------------- writing
def rotate64(x, pos, theta=10000.0):
    inv = torch.tensor([np.float32(theta ** (-2.0 * j / 64)) for j in range(32)], dtype=torch.float64, device=x.device)
    ang = pos.double()[:, None] * inv
    a, b = x[:, 448::2], x[:, 449::2]
    c, s = ang.cos(), ang.sin()
    return torch.cat([x[:, :448], torch.stack([a * c - b * s, a * s + b * c], -1).flatten(1)], 1)


@pytest.mark.parametrize("n,rows,rope,std", [(1, 1, True, 1.0), (3, 128, False, 1e-3), (33, 4096, True, 50.0),
                                             (1025, 1500, True, 1.0), (5000, 5001, False, 1.0)])
def test_swa_write(c2, n, rows, rope, std):
    lat = (torch.randn(n, D, generator=gen(n), device="cuda") * std).bfloat16()
    if n > 2:
        lat[1] = 0
        lat[2, 5:] = 0
    slot = torch.randperm(rows, generator=gen(1), device="cuda")[:n]
    pos = torch.randint(0, 1 << 22, (n,), generator=gen(2), device="cuda") if rope else None
    if rope:
        pos[0] = (1 << 22) - 1
    swa = torch.full((rows, D), 0x5A, dtype=torch.uint8, device="cuda")
    scale = torch.full((rows,), -3.0, device="cuda")
    c2.swa_quant_write(lat, slot, swa, scale, pos=pos)
    assert c2.last_launch_count() == 1 and c2.get_device_status() == 0
    x = lat.double() if pos is None else rotate64(lat.double(), pos)
    s = x.abs().amax(-1) / 448
    got = scale[slot].double()
    assert ((got - s).abs() <= s * 16 * 2.0 ** -24).all()
    y = torch.where(s[:, None] > 0, x / s[:, None].clamp_min(1e-300), torch.zeros_like(x))
    codes = swa[slot].view(torch.float8_e4m3fn).double()
    lo = (y - y.abs() * 2.0 ** -20).float().to(torch.float8_e4m3fn).double()
    hi = (y + y.abs() * 2.0 ** -20).float().to(torch.float8_e4m3fn).double()
    assert ((codes == lo) | (codes == hi)).all()
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[slot] = False
    assert (swa[rest] == 0x5A).all() and (scale[rest] == -3.0).all()


def test_swa_write_matches_torch_without_rope(c2):
    """Without RoPE every step is one IEEE operation: bit-exact against torch's cast."""
    lat = torch.randn(300, D, generator=gen(9), device="cuda").bfloat16()
    swa = torch.zeros(300, D, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(300, device="cuda")
    c2.swa_quant_write(lat, torch.arange(300, device="cuda"), swa, scale)
    s = lat.float().abs().amax(-1) / torch.full((), 448.0, device="cuda")
    assert torch.equal(scale, s)
    assert torch.equal(swa, (lat.float() / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8))


def test_swa_write_every_bf16_value(c2):
    """Every finite bf16 value, signed zeros and subnormals among them, in rows
    of like magnitudes: the codes and scales of torch's IEEE division and cast."""
    v = torch.arange(65536, device="cuda").to(torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[torch.isfinite(v)]
    v = v[v.float().abs().argsort()]
    v = torch.cat([v, v[-(-v.numel() % D):]]).view(-1, D) if v.numel() % D else v.view(-1, D)
    n = v.shape[0]
    swa = torch.zeros(n, D, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(n, device="cuda")
    c2.swa_quant_write(v.contiguous(), torch.arange(n, device="cuda"), swa, scale)
    s = v.float().abs().amax(-1) / torch.full((), 448.0, device="cuda")
    assert torch.equal(scale, s)
    live = s > 0
    y = (v.float()[live] / s[live][:, None]).clamp(-448, 448)
    assert torch.equal(swa[live], y.to(torch.float8_e4m3fn).view(torch.uint8))
    assert (swa[~live] == 0).all()


def test_swa_write_skips_bad_rows(c2):
    lat = torch.ones(4, D, device="cuda").bfloat16()
    slot = torch.tensor([0, -1, 8, 2], device="cuda")
    pos = torch.tensor([0, 0, 0, -5], device="cuda")
    swa = torch.zeros(8, D, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(8, device="cuda")
    c2.swa_quant_write(lat, slot, swa, scale, pos=pos)
    assert c2.get_device_status() == 0x2
    assert scale[0] > 0 and (scale[1:] == 0).all() and (swa[1:] == 0).all()


def test_swa_write_nonfinite(c2):
    lat = torch.ones(2, D, device="cuda").bfloat16()
    lat[0, 7] = math.nan
    lat[1, 9] = math.inf
    swa = torch.zeros(2, D, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(2, device="cuda")
    c2.swa_quant_write(lat, torch.arange(2, device="cuda"), swa, scale)
    v = swa.view(torch.float8_e4m3fn).float()
    assert torch.isnan(v[0, 7]) and torch.isnan(v[1, 9])
    assert torch.isfinite(torch.cat([v[0, :7], v[0, 8:]])).all()


# ----------------------------------------------------------------- reading
READS = [(1, 1, 1, False), (1, 7, 5, True), (3, 40, 33, True), (2, 100, 100, False), (4, 700, 600, True),
         (1, 5000, 5000, False), (5, 1000, 999, True)]


def read_case(batch, cap, k, listed, seed):
    idx = None
    if listed:
        idx = torch.randint(0, cap, (batch, k), generator=gen(seed), device="cuda", dtype=torch.int32)
        idx[batch - 1, k // 2:] = -1
        idx[0, 0] = idx[0, k - 1] = cap - 1
    at = torch.arange(k, device="cuda").expand(batch, k) if idx is None else idx.clamp_min(0).long()
    return idx, torch.arange(batch, device="cuda")[:, None], at


@pytest.mark.parametrize("batch,cap,k,listed", READS)
def test_kv_read(c2, batch, cap, k, listed):
    kv = entries(c2, batch * cap, cap).view(batch, cap, ENTRY)
    kv[0, 0, 256:] = torch.arange(1, 33, device="cuda", dtype=torch.uint8)   # subnormal and small scales
    idx, b, at = read_case(batch, cap, k, listed, 3)
    out = torch.full((batch, k, D), 9.0, dtype=torch.bfloat16, device="cuda")
    c2.kv_read(kv, out, idx=idx)
    assert c2.get_device_status() == 0
    want = kv64(kv)[b, at]
    if idx is not None:
        want[idx < 0] = 0
    assert torch.equal(out.double(), want)


@pytest.mark.parametrize("batch,cap,k,listed", READS)
def test_swa_read(c2, batch, cap, k, listed):
    swa = torch.randint(0, 256, (batch, cap, D), generator=gen(4), device="cuda").to(torch.uint8)
    swa[(swa & 127) == 127] = 0   # NaN codes have a test of their own
    scale = torch.rand(batch, cap, generator=gen(5), device="cuda")
    idx, b, at = read_case(batch, cap, k, listed, 6)
    out = torch.full((batch, k, D), 9.0, dtype=torch.bfloat16, device="cuda")
    c2.swa_read(swa, scale, out, idx=idx)
    want = (swa.view(torch.float8_e4m3fn).double() * scale.double()[..., None])[b, at]
    if idx is not None:
        want[idx < 0] = 0
    assert ((out.double() - want).abs() <= want.abs() * 2.0 ** -8 * (1 + 2.0 ** -14)).all()


@pytest.mark.parametrize("batch,cap,k,listed", [(1, 4, 1, False), (1, 8, 7, True), (4, 25, 25, False), (2, 302, 301, True),
                                                (1, 9000, 8999, False)])
def test_indexer_k_read(c2, batch, cap, k, listed):
    ik = c2.indexer_k_fp4_cache(batch * cap)
    x = torch.randn(batch * cap, 128, generator=gen(7), device="cuda") * torch.exp2(
        torch.randint(-120, 120, (batch * cap, 1), generator=gen(8), device="cuda").float())
    c2.indexer_k_quant(x.bfloat16(), torch.arange(batch * cap, device="cuda"), ik)
    idx, b, at = read_case(batch, cap, k, listed, 9)
    out = torch.full((batch, k, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    c2.indexer_k_read(ik, out, idx=idx)
    codes, exps = c2.indexer_k_fp4_planes(ik)
    want = (e2m1_64(codes) * torch.exp2(exps.double() - 127).repeat_interleave(32, -1)).view(batch, cap, 128)[b, at]
    if idx is not None:
        want[idx < 0] = 0
    assert torch.equal(out.double(), want)


def test_reads_special_values(c2):
    kv = entries(c2, 4, 1).view(1, 4, ENTRY)
    kv[0, 2, 256 + 3] = 0x7F   # a NaN scale: its 16 channels are NaN, no other
    out = torch.empty(1, 4, D, dtype=torch.bfloat16, device="cuda")
    c2.kv_read(kv, out)
    assert torch.isnan(out[0, 2, 48:64]).all() and int(torch.isnan(out).sum()) == 16
    ik = c2.indexer_k_fp4_cache(4)
    codes, exps = c2.indexer_k_fp4_planes(ik)
    codes.fill_(0x21)   # 0.5, 1
    exps[0, 0], exps[0, 1], exps[1, 0] = 0, 255, 254
    out = torch.empty(1, 4, 128, dtype=torch.bfloat16, device="cuda")
    c2.indexer_k_read(ik, out)
    assert out[0, 0, 0].double() == 2.0 ** -128 and torch.isnan(out[0, 0, 32:64]).all() and out[0, 1, 1].double() == 2.0 ** 127


def test_read_index_past_the_cache(c2):
    kv = entries(c2, 8, 2).view(2, 4, ENTRY)
    out = torch.full((2, 3, D), 9.0, dtype=torch.bfloat16, device="cuda")
    c2.kv_read(kv, out, idx=torch.tensor([[0, 4, 1], [3, 2, -7]], dtype=torch.int32, device="cuda"))
    assert c2.get_device_status() == 0x2
    v = kv64(kv)
    want = torch.stack([v[0, 0], v[0, 0] * 0, v[0, 1], v[1, 3], v[1, 2], v[0, 0] * 0]).view(2, 3, D)
    assert torch.equal(out.double(), want)


# ------------------------------------------------------------------- dense
CROSS = [
    # batch, n_q, cap, lengths
    (1, 1, 1, [1]),
    (1, 1, 300, [300]),
    (1, 2, 256, [256]),
    (2, 3, 600, [257, 600]),
    (3, 5, 1000, [1000, 0, 1]),
    (4, 1, 4096, [4096, 31, 2048, 0]),
    (2, 64, 513, [513, 255]),
    (1, 200, 2000, [1999]),
    (9, 2, 130, [130, 129, 128, 127, 1, 2, 0, 64, 65]),
    (1, 3, 30000, [29999]),
    (2, 100, 8, [8, 7]),
    (80, 2, 6000, [100] * 40 + [6000, 0] + [256] * 38),   # more pairs than workers, one of them shared by many
    (1, 301, 5000, [4321]),
    (700, 1, 300, [(37 * i) % 301 for i in range(700)]),  # many short sequences, some empty
]


def run_cross(c2, q, kv, n_vis, n_max, ws=None, stream=None):
    B, T = q.shape[:2]
    out = torch.full((B, T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, T, H), 7.0, device="cuda")
    if ws is None:
        ws = c2.workspace(c2.OP_CROSS, B * T, n_max, c2.Params.make())
    c2.cross_attn(q, kv, n_vis, n_max, out, ws, lse=lse, stream=stream)
    return out, lse


@pytest.mark.parametrize("batch,n_q,cap,lens", CROSS)
def test_cross_attn(c2, batch, n_q, cap, lens):
    kv = entries(c2, batch * cap, cap).view(batch, cap, ENTRY)
    n_vis = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):
        kv[b, n:] = 0xFF   # never written: every scale a NaN
    q = queries((batch, n_q), n_q)
    out, lse = run_cross(c2, q, kv, n_vis, max(lens))
    assert c2.get_device_status() == 0
    ref = [attend64(q[b].double().view(-1, D), kv64(kv[b, :n])) for b, n in enumerate(lens)]
    check_out(out, lse, torch.stack([r[0] for r in ref]), torch.stack([r[1] for r in ref]))


@pytest.mark.parametrize("order", ["rising", "falling", "one", "spread"])
def test_cross_attn_running_maximum(c2, order):
    """Logits that rise along the cache (every step raises the running maximum),
    fall, hold one key far above the rest, or span +-200."""
    n, T = 1500, 3
    kv = entries(c2, n, 11)
    q = queries((1, T), 12)
    lat = torch.randn(n, D, generator=gen(13), device="cuda")
    lat[:, 0] = 0
    ramp = torch.linspace(-1, 1, n, device="cuda")
    lat[:, 0] = {"rising": 40 * ramp, "falling": -40 * ramp, "one": torch.where(torch.arange(n, device="cuda") == 700, 60.0, 0.0),
                 "spread": 60 * torch.sign(torch.sin(torch.arange(n, device="cuda").float()))}[order]
    q[..., 0] = 80.0
    at = torch.arange(n, device="cuda")
    c2.kv_quant_write(lat.bfloat16(), None, 1, at, at.clone(), kv)
    out, lse = run_cross(c2, q, kv.view(1, n, ENTRY), torch.tensor([n], dtype=torch.int32, device="cuda"), n)
    r, rl = attend64(q[0].double().view(-1, D), kv64(kv))
    check_out(out, lse, r, rl)


def test_cross_attn_without_lse_and_bad_lengths(c2):
    kv = entries(c2, 2 * 100, 14).view(2, 100, ENTRY)
    q = queries((2, 1), 15)
    ws = c2.workspace(c2.OP_CROSS, 2, 100, c2.Params.make())
    out = torch.empty(2, 1, H, D, dtype=torch.bfloat16, device="cuda")
    c2.cross_attn(q, kv, torch.tensor([100, 100], dtype=torch.int32, device="cuda"), 100, out, ws)
    assert c2.get_device_status() == 0
    ref = torch.stack([attend64(q[b, 0].double(), kv64(kv[b]))[0] for b in range(2)])
    check_out(out, torch.zeros(2, H), ref, torch.zeros(2, H).double())
    # a length past n_max or below 0 is flagged and taken as n_max or 0
    c2.cross_attn(q, kv, torch.tensor([101, -1], dtype=torch.int32, device="cuda"), 100, out, ws)
    assert c2.get_device_status() == 0x1
    assert (out[1] == 0).all()


def run_prefix(c2, p, q, pre, kv, idx, swa, sc, sl, ws=None, stream=None):
    B = q.shape[0]
    out = torch.full((B, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, H), 7.0, device="cuda")
    if ws is None:
        ws = c2.workspace(c2.OP_PREFIX, B, pre.shape[0], p)
    c2.prefix_attn(p, q, pre, kv, idx, swa, sc, sl, out, ws, lse=lse, stream=stream)
    return out, lse


def prefix_inputs(c2, batch, n_prefix, K, W, seed, own=None):
    own = own or [(K, W)] * batch
    p = c2.Params.make(index_topk=K, sliding_window=W)
    q = queries((batch,), seed)
    pre = entries(c2, n_prefix, seed + 1)
    cap = K + 50
    kv = entries(c2, batch * cap, seed + 2).view(batch, cap, ENTRY)
    idx = torch.full((batch, K), -1, dtype=torch.int32, device="cuda")
    for b, (k, _) in enumerate(own):
        idx[b, :k] = torch.randperm(cap, generator=gen(seed + b), device="cuda")[:k].sort().values.int()
    swa = torch.zeros(batch, W, D, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(batch, W, device="cuda")
    if W:
        lat = torch.randn(batch * W, D, generator=gen(seed + 3), device="cuda").bfloat16()
        c2.swa_quant_write(lat, torch.arange(batch * W, device="cuda"), swa, sc)
    sl = torch.tensor([w for _, w in own], dtype=torch.int32, device="cuda")
    return p, q, pre, kv, idx, swa, sc, sl


def prefix_ref(q, pre, kv, idx, swa, sc, sl):
    outs, lses = [], []
    for b in range(q.shape[0]):
        i = idx[b][idx[b] >= 0].long()
        n = int(sl[b])
        keys = torch.cat([kv64(pre), kv64(kv[b][i]), swa[b, :n].view(torch.float8_e4m3fn).double() * sc[b, :n].double()[:, None]])
        o, l = attend64(q[b].double(), keys)
        outs.append(o)
        lses.append(l)
    return torch.stack(outs), torch.stack(lses)


@pytest.mark.parametrize("batch,n_prefix,K,W,own", [
    (1, 0, 16, 8, None), (1, 1, 512, 128, None), (1, 5000, 512, 128, None), (2, 257, 37, 0, None),
    (3, 1000, 512, 128, [(512, 128), (0, 0), (5, 1)]), (3, 0, 64, 16, [(64, 16), (0, 0), (0, 16)]),
    (5, 20001, 1, 1, None), (33, 700, 512, 128, None), (200, 300, 16, 8, None)])
def test_prefix_attn(c2, batch, n_prefix, K, W, own):
    args = prefix_inputs(c2, batch, n_prefix, K, W, 20, own)
    out, lse = run_prefix(c2, *args)
    assert c2.get_device_status() == 0
    check_out(out, lse, *prefix_ref(*args[1:]))


def test_prefix_equals_sparse_over_the_union(c2):
    """A prefix of 300 entries and 200 selected ones: the same softmax as
    sparse_attn over one cache that holds both, all 500 selected."""
    p, q, pre, kv, idx, swa, sc, sl = prefix_inputs(c2, 3, 300, 200, 128, 30)
    out, lse = run_prefix(c2, p, q, pre, kv, idx, swa, sc, sl)
    both = torch.stack([torch.cat([pre, kv[b][idx[b].long()]]) for b in range(3)])
    p2 = c2.Params.make(index_topk=500, sliding_window=128)
    o2 = torch.empty(3, H, D, device="cuda")
    l2 = torch.empty(3, H, device="cuda")
    c2.sparse_attn(p2, q, both, torch.arange(500, dtype=torch.int32, device="cuda").repeat(3, 1), swa, sc, sl, o2,
                   c2.workspace(c2.OP_ATTN, 3, 500, p2), lse=l2)
    check_out(out, lse, o2.double(), l2.double())


def test_write_select_read_and_attend_together(c2):
    """The operators as a decode step uses them: window rows written, entries
    written, the shared prefix and the own part attended, the attended rows
    read back and attended again in 64 bits."""
    B, W, K = 4, 128, 64
    p, q, pre, kv, idx, swa, sc, sl = prefix_inputs(c2, B, 900, K, W, 40)
    new = torch.randn(B, D, generator=gen(41), device="cuda").bfloat16()
    slot = torch.arange(B, device="cuda") * W + 5
    c2.swa_quant_write(new, slot, swa, sc, pos=torch.full((B,), 70000, device="cuda"))
    out, lse = run_prefix(c2, p, q, pre, kv, idx, swa, sc, sl)
    sel = torch.empty(B, K, D, dtype=torch.bfloat16, device="cuda")
    win = torch.empty(B, W, D, dtype=torch.bfloat16, device="cuda")
    whole = torch.empty(1, 900, D, dtype=torch.bfloat16, device="cuda")
    c2.kv_read(kv, sel, idx=idx)
    c2.swa_read(swa, sc, win)
    c2.kv_read(pre.view(1, 900, ENTRY), whole)
    assert c2.get_device_status() == 0
    ref = [attend64(q[b].double(), torch.cat([whole[0], sel[b], win[b]]).double()) for b in range(B)]
    r, rl = torch.stack([x[0] for x in ref]), torch.stack([x[1] for x in ref])
    # the window rows read back are rounded to bf16 (2^-8 / sqrt(3) of a value
    # on average): a logit of the sharpest heads moves by 3 x 2^-8 / sqrt(3) =
    # 0.007 on average, the log-sum-exp by less (the window is an eighth of the
    # keys), an output by less than 0.02 of the row's largest
    assert (out.double() - r).abs().max() <= 0.02 * r.abs().max()
    assert (lse.double() - rl).abs().max() <= 1e-2


def test_dense_repeats_and_graph_replays(c2):
    """The same call twice gives the same bits, also from a captured graph
    replayed on new inputs, and with a workspace left full of NaNs."""
    B, T, n = 3, 5, 3000
    kv = entries(c2, B * n, 50).view(B, n, ENTRY)
    nv = torch.tensor([3000, 1, 1700], dtype=torch.int32, device="cuda")
    q = queries((B, T), 51)
    ws = c2.workspace(c2.OP_CROSS, B * T, n, c2.Params.make())
    ws.fill_(0xFF)
    o1, l1 = run_cross(c2, q, kv, nv, n, ws)
    o2, l2 = run_cross(c2, q, kv, nv, n, ws)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    out, lse = torch.empty_like(o1), torch.empty_like(l1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        c2.cross_attn(q, kv, nv, n, out, ws, lse=lse)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            c2.cross_attn(q, kv, nv, n, out, ws, lse=lse)
    q2 = queries((B, T), 52)
    keep = q.clone()
    want = run_cross(c2, q2, kv, torch.tensor([17, 3000, 0], dtype=torch.int32, device="cuda"), n)
    q.copy_(q2)
    nv.copy_(torch.tensor([17, 3000, 0], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    q.copy_(keep)


def test_two_streams_with_their_own_workspaces(c2):
    p, *args = prefix_inputs(c2, 6, 2500, 64, 16, 60)
    want = run_prefix(c2, p, *args)
    torch.cuda.synchronize()
    got = []
    for _ in range(2):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got.append(run_prefix(c2, p, *args))
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


def test_offsets_past_32_bits(c2):
    """A cache of 9 million entries (2.6 GB): the last sequence's rows lie past 2^31 bytes."""
    B, cap = 3, 3_000_000
    kv = torch.zeros(B, cap, ENTRY, dtype=torch.uint8, device="cuda")
    tail = entries(c2, 700, 70)
    kv[2, :700] = tail
    q = queries((B, 1), 71)
    out, lse = run_cross(c2, q, kv, torch.tensor([0, 0, 700], dtype=torch.int32, device="cuda"), 700)
    r, rl = attend64(q[2, 0].double(), kv64(tail))
    check_out(out[2], lse[2], r, rl)
    kv[2, cap - 1] = tail[0]
    back = torch.empty(B, 1, D, dtype=torch.bfloat16, device="cuda")
    c2.kv_read(kv, back, idx=torch.full((B, 1), cap - 1, dtype=torch.int32, device="cuda"))
    assert torch.equal(back[2, 0].double(), kv64(tail[0]))


def test_binding_refusals_on_the_gpu(c2):
    """Tensors of another dtype, shape, layout or device are refused before anything runs."""
    kv = entries(c2, 8, 80).view(1, 8, ENTRY)
    out = torch.empty(1, 4, D, dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    for bad in (dict(kv=kv[:, ::2]), dict(kv=kv.cpu()), dict(kv=kv[..., :256]), dict(out=out.float()), dict(out=out[..., ::2]),
                dict(idx=idx.long()), dict(idx=idx[:, :3]), dict(idx=idx.cpu())):
        a = dict(kv=kv, out=out, idx=idx) | bad
        with pytest.raises(c2.Csa2Error):
            c2.kv_read(a["kv"], a["out"], idx=a["idx"])
    q = queries((1, 2), 81)
    o = torch.empty_like(q)
    nv = torch.tensor([8], dtype=torch.int32, device="cuda")
    ws = c2.workspace(c2.OP_CROSS, 2, 8, c2.Params.make())
    for bad in (dict(q=q.half()), dict(q=q.transpose(0, 1)), dict(nv=nv.long()), dict(n=9), dict(ws=ws[:1024]), dict(ws=ws[16:]),
                dict(o=o[:, :1])):
        a = dict(q=q, nv=nv, n=8, ws=ws, o=o) | bad
        with pytest.raises(c2.Csa2Error):
            c2.cross_attn(a["q"], kv, a["nv"], a["n"], a["o"], a["ws"])
    assert c2.get_device_status() == 0


@pytest.mark.parametrize("batch,n_prefix", [(201, 300), (153, 256), (305, 1)])
def test_prefix_odd_batch_with_whole_pairs(c2, batch, n_prefix):
    """More pairs than workers: most pairs are whole in one range and merged with
    their own part there, the last pair has one token, some own parts are empty."""
    own = [((16, 8), (0, 0), (3, 0), (0, 5))[b % 4] for b in range(batch)]
    args = prefix_inputs(c2, batch, n_prefix, 16, 8, 90, own)
    out, lse = run_prefix(c2, *args)
    assert c2.get_device_status() == 0
    check_out(out, lse, *prefix_ref(*args[1:]))


@pytest.mark.parametrize("batch,n_q,cap,lens", [(3, 3, 700, [257, 0, 700]), (1, 1, 600, [511]), (90, 3, 300, None)])
def test_cross_attn_stays_inside_its_buffers(c2, batch, n_q, cap, lens):
    """A workspace of exactly the size asked for, outputs between guard rows, and
    every byte past a sequence's length 0xFF (scales that are NaN)."""
    lens = lens or [(37 * b) % (cap + 1) for b in range(batch)]
    kv = entries(c2, batch * cap, 95).view(batch, cap, ENTRY)
    for b, n in enumerate(lens):
        kv[b, n:] = 0xFF
    q = queries((batch, n_q), 96)
    rows = batch * n_q
    out = torch.full((rows + 2, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows + 2, H), 7.0, device="cuda")
    size = c2.workspace_bytes(c2.OP_CROSS, rows, cap, c2.Params.make())
    buf = torch.full((size + 512,), 0xAB, dtype=torch.uint8, device="cuda")
    start = -buf.data_ptr() % 256
    ws = buf[start:start + size]
    nv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    c2.cross_attn(q, kv, nv, cap, out[1:-1].view(batch, n_q, H, D), ws, lse=lse[1:-1].view(batch, n_q, H))
    assert c2.get_device_status() == 0
    assert (buf[:start] == 0xAB).all() and (buf[start + size:] == 0xAB).all()
    assert (out[0] == 7).all() and (out[-1] == 7).all() and (lse[0] == 7).all() and (lse[-1] == 7).all()
    for b, n in enumerate(lens):
        o, l = out[1:-1].view(batch, n_q, H, D)[b], lse[1:-1].view(batch, n_q, H)[b]
        if n == 0:
            assert (o == 0).all() and (l == -float("inf")).all()
            continue
        for t in range(n_q):
            ro, rl = attend64(q[b, t].double(), kv64(kv[b, :n]))
            check_out(o[t][None], l[t][None], ro[None], rl[None])
