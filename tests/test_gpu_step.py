"""The slot maps, the windowed attention with sinks and the attention of drafted
trees against plain 64-bit implementations.

Tolerances.  The maps are whole numbers: equal.  A readout rounds each weight to
fp16, independently for each key, so an output of standard deviation s over its
channels is off by 2^-11 / sqrt(3) s, and by five times that at the worst of some
10^5 values; a row's largest of 512 channels is above 2 s, so 2^-9 of it is twice
what five deviations need, which leaves room for fp16 partials (2^-11 of a value).
One key alone is off by 2^-11 of itself, below the same bound.  The output's own
rounding to bf16 adds 2^-8 of each value.  The log-sum-exp is fp32 over fp32
logits: 2e-5 of it (or of 1).
"""
import math
import threading

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


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def queries(shape, seed, sharp=3.0):
    s = torch.linspace(0.5, sharp, H, device="cuda").unsqueeze(-1)
    return (torch.randn(*shape, H, D, generator=gen(seed), device="cuda") * s).bfloat16()


def rows8(shape, seed, std=1.0):
    """E4M3 codes and scales of N(0, std^2) rows."""
    x = torch.randn(*shape, D, generator=gen(seed), device="cuda").double() * std
    s = (x.abs().amax(-1) / 448).float()
    y = x / s.double().clamp_min(1e-300)[..., None]
    return y.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s


def rows64(codes, scale):
    return codes.view(torch.float8_e4m3fn).double() * scale.double()[..., None]


def entries(c2, rows, seed):
    kv = torch.zeros(rows, ENTRY, dtype=torch.uint8, device="cuda")
    at = torch.arange(rows, device="cuda")
    c2.kv_quant_write(torch.randn(rows, D, generator=gen(seed), device="cuda").bfloat16(), None, 1, at, at.clone(), kv)
    return kv


def kv64(kv):
    c = torch.stack([kv[..., :256] & 15, kv[..., :256] >> 4], -1).flatten(-2).long()
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=kv.device)
    return lut[c] * kv[..., 256:].contiguous().view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)


def attend64(q, keys):
    """q [64, 512], keys [n, 512] in 64 bits -> (out, lse)."""
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
    if lse is None:
        return
    l, rl = lse.double().reshape(-1), ref_lse.reshape(-1)
    empty = torch.isinf(rl)
    assert torch.equal(torch.isneginf(l), empty)
    err = (l - rl)[~empty].abs()
    assert (err <= 2e-5 * rl[~empty].abs().clamp_min(1.0)).all(), f"lse off by {err.max().item()}"


# --------------------------------------------------------------- slot maps
def map64(ctx, new, cap, ring, n, e, m):
    tok, pos, swa, epos, slot, cu, ecu = [], [], [], [], [], [0], [0]
    for b, (c, k) in enumerate(zip(ctx, new)):
        for r in range(k):
            p = c + r
            tok.append(b)
            pos.append(p)
            swa.append(b * ring + p % ring if k - r <= ring else -1)
            if p % m == m - 1:
                epos.append(p)
                slot.append(b * cap + p // m if p // m < cap else -1)
        cu.append(len(tok))
        ecu.append(len(epos))

    def fill(x, size):
        return (x + [-1] * size)[:size]

    return (cu, fill(tok, n), fill(pos, n), fill(swa, n), ecu, fill(epos, e), fill(slot, e),
            [min((c + k) // m, cap) for c, k in zip(ctx, new)], [min(c + k, ring) for c, k in zip(ctx, new)])


def lengths(batch, most, seed):
    g = torch.Generator().manual_seed(seed)
    new = torch.randint(0, most + 1, (batch,), generator=g).tolist()
    return torch.randint(0, 5000, (batch,), generator=g).tolist(), new


@pytest.mark.parametrize("batch,most,m,ring,spare", [
    (1, 1, 1, 128, 0), (1, 1, 2, 128, 0), (32, 1, 1, 128, 5), (3, 700, 2, 128, 1), (1, 5000, 1, 1, 0), (31, 33, 2, 200, 300),
    (1000, 7, 1, 135, 0), (1025, 2, 2, 128, 64), (8192, 3, 1, 131, 0), (2, 0, 1, 128, 9), (513, 400, 2, 527, 1000)])
def test_slot_map(c2, batch, most, m, ring, spare):
    ctx, new = lengths(batch, most, batch + most)
    n = sum(new) + spare
    maps = c2.slot_maps(batch, n, m)
    c2.slot_map(ints(ctx), ints(new), 20000, ring, maps, m=m)
    assert c2.last_launch_count() == 1 and c2.get_device_status() == 0
    want = map64(ctx, new, 20000, ring, n, maps.slot.numel(), m)
    for got, ref, name in zip(maps, want, maps._fields):
        assert got.tolist() == ref, name


def test_slot_map_far_positions_and_caps(c2):
    """Slots past 2^32, a position at the largest ctx_len, a sequence past its
    cap, buffers that are too short, lengths below zero."""
    ctx, new = [(1 << 31) - 6, 7, 0, 100], [5, 3, 0, 2]
    maps = c2.slot_maps(4, 12)
    c2.slot_map(ints(ctx), ints(new), 1 << 31, 1 << 31, maps)
    assert c2.get_device_status() == 0
    for got, ref in zip(maps, map64(ctx, new, 1 << 31, 1 << 31, 12, 12, 1)):
        assert got.tolist() == ref
    maps = c2.slot_maps(4, 10)
    c2.slot_map(ints(ctx), ints(new), 101, 128, maps)
    assert c2.get_device_status() == 1
    want = map64(ctx, new, 101, 128, 10, 10, 1)
    assert -1 in want[6]
    for got, ref in zip(maps, want):
        assert got.tolist() == ref
    guard = torch.full((64,), 77, dtype=torch.int64, device="cuda")
    maps = c2.slot_maps(4, 6)._replace(pos=guard[:6], slot=guard[32:38])
    c2.slot_map(ints(ctx), ints(new), 1 << 31, 128, maps)
    assert c2.get_device_status() == 1
    assert guard[:6].tolist() == map64(ctx, new, 1 << 31, 128, 6, 6, 1)[2] and (guard[6:32] == 77).all() and (guard[38:] == 77).all()
    maps = c2.slot_maps(3, 4)
    c2.slot_map(ints([-5, 2, 9]), ints([2, -3, 2]), 100, 128, maps)
    assert c2.get_device_status() == 1
    for got, ref in zip(maps, map64([0, 2, 9], [2, 0, 2], 100, 128, 4, 4, 1)):
        assert got.tolist() == ref
    # sums past 32 bits: nothing is written out of bounds, the sums stay at the largest
    maps = c2.slot_maps(3, 4)
    c2.slot_map(ints([0, 0, 0]), ints([1 << 30] * 3), 1 << 31, 128, maps)
    assert c2.get_device_status() == 1
    assert maps.cu.tolist() == [0, 1 << 30, (1 << 31) - 1, (1 << 31) - 1]
    assert maps.pos.tolist() == [0, 1, 2, 3]


def test_slot_map_graph_and_stream(c2):
    """One captured call, replayed on other lengths; a call on another stream."""
    ctx, new = ints([5, 0, 9]), ints([3, 4, 1])
    maps = c2.slot_maps(3, 12)
    c2.slot_map(ctx, new, 100, 128, maps)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c2.slot_map(ctx, new, 100, 128, maps)
    for c, k in (([5, 0, 9], [3, 4, 1]), ([1, 2, 3], [0, 0, 12]), ([50, 60, 70], [4, 4, 4])):
        ctx.copy_(ints(c))
        new.copy_(ints(k))
        g.replay()
        for got, ref in zip(maps, map64(c, k, 100, 128, 12, 12, 1)):
            assert got.tolist() == ref
    s = torch.cuda.Stream()
    other = c2.slot_maps(3, 12)
    s.wait_stream(torch.cuda.current_stream())
    c2.slot_map(ctx, new, 100, 128, other, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(maps, other))


def test_slot_map_from_two_threads(c2):
    """Calls of two sizes that both need more shared memory than a kernel has by default."""
    sizes, failed = (8192, 4200), []

    def calls(batch, maps, ctx, new, stream):
        try:
            for _ in range(500):
                c2.slot_map(ctx, new, 100, 128, maps, stream=stream)
        except c2.Csa2Error as e:
            failed.append(e)

    given = [(b, c2.slot_maps(b, b), ints(range(b)), ints([1] * b), torch.cuda.Stream()) for b in sizes]
    torch.cuda.synchronize()
    threads = [threading.Thread(target=calls, args=a) for a in given]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    c2.get_device_status()   # (most of the entries lie past the cap of 100)
    for b, maps, *_ in given:
        for got, ref in zip(maps, map64(list(range(b)), [1] * b, 100, 128, b, b, 1)):
            assert got.tolist() == ref


# ------------------------------------------------------------------ window
class Window:
    """A step of a window-only layer: every ring and sink row that no token sees
    holds NaN codes and a NaN scale."""

    def __init__(self, ctx, new, W, S, spare=0, slack=0, seed=0, std=1.0, sharp=3.0):
        self.ctx, self.new, self.W, self.S = ctx, new, W, S
        B, n = len(ctx), sum(new) + spare
        ring = max(1, W - 1 + max(new)) + slack
        self.cu = ints([sum(new[:i]) for i in range(B + 1)])
        self.ctx_t = ints(ctx)
        self.q = queries((n,), seed + 1, sharp)
        swa, scale = rows8((B, ring), seed + 2, std)
        sink, sink_scale = rows8((B, max(S, 1)), seed + 3, std)
        self.swa, self.scale = torch.full_like(swa, 0x7F), torch.full_like(scale, math.nan)
        self.sink, self.sink_scale = torch.full_like(sink, 0x7F), torch.full_like(sink_scale, math.nan)
        for b, (c, k) in enumerate(zip(ctx, new)):
            if k:
                p = torch.arange(max(0, c - W + 1), c + k, device="cuda") % ring
                if W:
                    self.swa[b, p], self.scale[b, p] = swa[b, p], scale[b, p]
                s = max(0, min(S, c + k - W))
                self.sink[b, :s], self.sink_scale[b, :s] = sink[b, :s], sink_scale[b, :s]
        self.sink, self.sink_scale = self.sink[:, :S].contiguous(), self.sink_scale[:, :S].contiguous()
        self.out = torch.full((n, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((n, H), 7.0, device="cuda")

    def call(self, c2, kernel=0, lse=True, **kw):
        c2.window_attn(c2.Params.make(sliding_window=self.W, attn_kernel=kernel), self.q, self.cu, self.ctx_t, self.swa,
                       self.scale, self.out, sink=self.sink if self.S else None,
                       sink_scale=self.sink_scale if self.S else None, lse=self.lse if lse else None, **kw)

    def reference(self):
        ring, i = self.swa.shape[1], 0
        out, lse = self.out.double(), self.lse.double()
        out[:], lse[:] = 7.0, 7.0
        for b, (c, k) in enumerate(zip(self.ctx, self.new)):
            for p in range(c, c + k):
                at = torch.arange(max(0, p - self.W + 1), p + 1, device="cuda")[-self.W:] % ring if self.W else torch.arange(0, device="cuda")
                s = max(0, min(self.S, p - self.W + 1))
                keys = torch.cat([rows64(self.sink[b, :s], self.sink_scale[b, :s]), rows64(self.swa[b, at], self.scale[b, at])])
                out[i], lse[i] = attend64(self.q[i].double(), keys)
                i += 1
        return out, lse, i

    def check(self, lse=True):
        out, ref_lse, n = self.reference()
        check_out(self.out[:n], self.lse[:n] if lse else None, out[:n], ref_lse[:n])
        assert (self.out[n:] == 7.0).all() and (self.lse[n if lse else 0:] == 7.0).all()


WINDOWS = [
    dict(ctx=[0], new=[1], W=128, S=4), dict(ctx=[5000], new=[1], W=128, S=4), dict(ctx=[200, 0, 131], new=[1, 1, 1], W=128, S=0),
    dict(ctx=[10 * i for i in range(40)], new=[1] * 40, W=128, S=8, spare=3),
    dict(ctx=[0, 50, 999, 127], new=[7, 0, 130, 1], W=128, S=4, spare=9), dict(ctx=[120], new=[300], W=128, S=1),
    dict(ctx=[3, 64], new=[65, 40], W=1, S=0), dict(ctx=[3, 0], new=[65, 40], W=1, S=5), dict(ctx=[9, 0], new=[4, 3], W=0, S=6),
    dict(ctx=[9], new=[4], W=0, S=0), dict(ctx=[37, 1], new=[100, 99], W=37, S=3, slack=5), dict(ctx=[90], new=[170], W=100, S=64),
    dict(ctx=[600, 0], new=[20, 40], W=300, S=4), dict(ctx=[1500], new=[3], W=1024, S=64),
    dict(ctx=[0, 0, 0], new=[0, 0, 3], W=128, S=4), dict(ctx=[2 ** 31 - 200], new=[150], W=128, S=4),
    dict(ctx=[20 * i for i in range(150)], new=[3 if i % 7 else 0 for i in range(150)], W=128, S=4, spare=1),
    dict(ctx=[17, 400, 0, 88, 1000], new=[401, 1, 256, 2, 33], W=128, S=15), dict(ctx=[17, 400], new=[33, 260], W=128, S=16),
    dict(ctx=[9, 0], new=[60, 40], W=0, S=6), dict(ctx=[9], new=[100], W=0, S=0), dict(ctx=[0, 700], new=[80, 81], W=128, S=13),
    dict(ctx=[31 * i for i in range(320)], new=[1] * 320, W=128, S=4), dict(ctx=[31 * i for i in range(200)], new=[2 - i % 2 for i in range(200)], W=16, S=1),
    dict(ctx=[100, 5], new=[90, 77], W=1024, S=3), dict(ctx=[31 * i for i in range(100)], new=[4] * 100, W=128, S=2),
    dict(ctx=[2, 0], new=[100, 140], W=0, S=6), dict(ctx=[900], new=[400], W=128, S=13), dict(ctx=[3, 0], new=[121, 90], W=1, S=2),
    dict(ctx=[60 + i for i in range(40)], new=[i % 11 for i in range(40)], W=37, S=3),
]


@pytest.mark.parametrize("kernel", [0, 1, 2])
@pytest.mark.parametrize("case", WINDOWS, ids=[str(i) for i in range(len(WINDOWS))])
def test_window(c2, case, kernel):
    w = Window(**case, seed=11)
    w.call(c2, kernel)
    assert c2.get_device_status() == 0
    w.check()


@pytest.mark.parametrize("W,S", [(0, 64), (1, 63), (1, 64), (77, 64), (78, 64)])
def test_window_as_many_sinks_as_there_can_be(c2, W, S):
    """The most sinks behind windows that leave them room in a tile, and one row more."""
    w = Window([0, 70], [150, 60], W, S, seed=21)
    for kernel in (0, 1, 2):
        w.call(c2, kernel)
        assert c2.get_device_status() == 0
        w.check()


@pytest.mark.parametrize("std", [1e-15, 1e-12, 1e-5, 1e3, 1e12])
@pytest.mark.parametrize("new", [1, 150])
def test_window_rows_of_any_size(c2, std, new):
    """Rows far from 1, some of them zero and some a million times the others."""
    w = Window([200, 100], [new, new], 128, 4, seed=5, std=std)
    if std > 1:   # logits of the same size (queries of 1e-12 are below fp16: every key alike)
        w.q = (w.q.double() / std).bfloat16() if std < 1e4 else torch.zeros_like(w.q)
    w.swa[:, ::7] = 0
    w.scale[:, ::7] = 0
    w.scale[:, 3::11] *= 1e-6
    for kernel in (0, 1, 2):
        w.call(c2, kernel)
        assert c2.get_device_status() == 0
        w.check()


@pytest.mark.parametrize("sharp", [30.0, 120.0])
def test_logits_that_tower(c2, sharp):
    """Logits of a spread of up to 170 powers of two, whose running reference is
    raised again and again: windows, trees with and without entries.  (A logit x is
    off by some 2^-20 of it, so a weight by 1e-4 at most, far below 2^-9.)"""
    for kernel in (0, 1, 2):
        w = Window([300, 20, 0], [90, 150, 64], 128, 4, seed=12, sharp=sharp)
        w.call(c2, kernel)
        assert c2.get_device_status() == 0
        w.check()
        for K in (0, 300):
            t = Tree(c2, 40, 8, K, 128, [9 * i for i in range(40)], cap=310, seed=13)
            t.q = queries((40, 8), 14, sharp)
            t.call(c2, kernel)
            assert c2.get_device_status() == 0
            t.check()


def test_logits_past_two_to_the_29(c2):
    """Queries near fp16's end and rows of 2,000: each head's logit for one key, or
    for two equal ones, is about 2.7e9, the others' far below, and the output is that
    key."""
    sign = torch.where(torch.rand(D, generator=gen(90), device="cuda") < 0.5, -1.0, 1.0)
    tall = (sign * 448).to(torch.float8_e4m3fn).view(torch.uint8)
    for kernel in (0, 1, 2):
        w = Window([400, 10], [100, 80], 128, 4, seed=91, std=20.0)
        w.q = (sign * 60000).bfloat16().expand(180, H, D).contiguous()
        for b, rows in ((0, (350, 420, 421)), (1, (0, 40))):
            r = torch.tensor(rows, device="cuda") % w.swa.shape[1]
            w.swa[b, r], w.scale[b, r] = tall, 2000.0 / 448
        w.call(c2, kernel)
        assert c2.get_device_status() == 0
        w.check()
        t = Tree(c2, 30, 6, 64, 128, [500 + i for i in range(30)], cap=80, seed=92, std=20.0, empty=False)
        t.q = (sign * 60000).bfloat16().expand(30, 6, H, D).contiguous()
        t.swa[:, 7], t.scale[:, 7] = tall, 2000.0 / 448
        t.tree[:, 2], t.tree_scale[:, 2] = tall, 2000.0 / 448
        t.call(c2, kernel)
        assert c2.get_device_status() == 0
        t.check()


def test_window_without_lse_and_scales_of_zero(c2):
    w = Window([300], [64], 128, 4, seed=6)
    w.call(c2, lse=False)
    w.check(lse=False)
    w.scale.zero_()
    w.sink_scale.zero_()
    w.swa.zero_()
    w.sink.zero_()
    w.call(c2)
    w.check()
    # a visible NaN row makes every token that sees it NaN, and no other one
    w = Window([0], [200], 128, 0, seed=7)
    w.swa[0, 60, 5] = 0x7F
    w.call(c2)
    nan = torch.isnan(w.out.float()).flatten(1).any(1)
    assert nan.tolist() == [60 <= p < 188 for p in range(200)]


def test_window_ring_too_short(c2):
    """A ring that has lost rows a token sees: reported, and the other sequences are right."""
    w = Window([500, 40], [30, 4], 128, 4, seed=8)
    short = 130
    cut = w.swa[:, :short].contiguous(), w.scale[:, :short].contiguous().nan_to_num(1.0)
    w.swa, w.scale = cut
    w.call(c2)
    assert c2.get_device_status() == 2
    w.ctx_t[0] = -3
    w.call(c2)
    assert c2.get_device_status() == 2


def test_window_many_empty_sequences(c2):
    """Tokens of the first and the last of a million sequences, and of one among them."""
    B, n, at = 1_000_000, 130, 654_321
    w = Window([300, 200, 5], [n, n, n], 128, 4, seed=9)
    ctx, cu = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    place = torch.tensor([0, at, B - 1], device="cuda")
    ctx[place] = w.ctx_t
    cu[1:at + 1], cu[at + 1:B], cu[B] = n, 2 * n, 3 * n
    # (rings of a million sequences would be 65 GB and more: W = 0, two first tokens each)
    sink, scale = torch.zeros(B, 2, D, dtype=torch.uint8, device="cuda"), torch.ones(B, 2, device="cuda")
    codes, s = rows8((3, 2), 10)
    sink[place], scale[place] = codes, s
    for kernel in (0, 2):
        c2.window_attn(c2.Params.make(sliding_window=0, attn_kernel=kernel), w.q, cu, ctx, None, None, w.out, sink=sink,
                       sink_scale=scale, lse=w.lse)
        assert c2.get_device_status() == 0
        for i in (0, 1, n - 1, n, 2 * n - 1, 2 * n, 3 * n - 1):
            b = i // n
            seen = min(2, w.ctx[b] + i - b * n + 1)
            ref, lse = attend64(w.q[i].double(), rows64(codes[b, :seen], s[b, :seen]))
            check_out(w.out[i], w.lse[i], ref, lse)


@pytest.mark.parametrize("new", [1, 40])
def test_window_graph_stream_and_repeat(c2, new):
    """A captured call replayed on other inputs, beside calls on another stream; the same call twice gives the same bits."""
    case = dict(ctx=[300, 20], new=[new, new], W=128, S=4)
    a, b = Window(**case, seed=21), Window(**case, seed=22)
    a.call(c2)
    first = a.out.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.call(c2)
    a.out.zero_()
    g.replay()
    assert torch.equal(a.out, first)
    for x in ("q", "swa", "scale", "sink", "sink_scale"):
        getattr(a, x).copy_(getattr(b, x))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g.replay()
    b.call(c2, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)
    b.check()


# -------------------------------------------------------------------- tree
class Tree:
    def __init__(self, c2, B, T, K, W, ctx, cap=0, seed=0, std=1.0, slack=0, empty=True):
        self.B, self.T, self.K, self.W, self.ctx = B, T, K, W, ctx
        g = torch.Generator().manual_seed(seed)
        self.q = queries((B, T), seed + 1)
        self.kv = entries(c2, B * cap, seed + 2).view(B, cap, ENTRY) if K else None
        self.idx = None
        if K:
            self.idx = torch.stack([torch.stack([torch.randperm(cap, generator=g)[:K].sort().values for _ in range(T)])
                                    for _ in range(B)]).int().cuda() if K <= cap else None
            self.idx[:, T // 2, K // 2:] = -1
            if empty and T > 2:
                self.idx[0, 1] = -1
        ring = max(1, W) + slack
        self.swa, self.scale = rows8((B, ring), seed + 3, std)
        for b, c in enumerate(ctx):
            if c < ring:
                self.swa[b, c:], self.scale[b, c:] = 0x7F, math.nan
        self.tree, self.tree_scale = rows8((B, T), seed + 4, std)
        self.mask = [[0] * T for _ in range(B)]
        for b in range(B):
            for t in range(T):
                up = int(torch.randint(-1, t, (1,), generator=g)) if t else -1
                self.mask[b][t] = (self.mask[b][up] if up >= 0 else 0) | 1 << t
        if empty and T > 2:
            self.mask[0][1] = 0
        self.put_mask()
        self.out = torch.full((B, T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((B, T, H), 7.0, device="cuda")

    def put_mask(self):
        self.mask_t = torch.tensor([[m - (1 << 64) if m >> 63 else m for m in r] for r in self.mask], dtype=torch.int64, device="cuda")

    def call(self, c2, kernel=0, **kw):
        c2.tree_attn(c2.Params.make(index_topk=max(self.K, 1), sliding_window=self.W, attn_kernel=kernel), self.q, self.kv,
                     self.idx, self.swa, self.scale, ints(self.ctx) if "ctx_t" not in kw else kw.pop("ctx_t"), self.tree,
                     self.tree_scale, self.mask_t, self.out, lse=self.lse, **kw)

    def check(self):
        ring = self.swa.shape[1]
        ref, ref_lse = self.out.double(), self.lse.double()
        for b, c in enumerate(self.ctx):
            for t in range(self.T):
                named = [u for u in range(self.T) if self.mask[b][t] >> u & 1]
                left = max(0, self.W - len(named))
                at = torch.arange(max(0, c - left), c, device="cuda") % ring
                keys = [rows64(self.swa[b, at], self.scale[b, at]), rows64(self.tree[b, named], self.tree_scale[b, named])]
                if self.K:
                    sel = self.idx[b, t]
                    keys.append(kv64(self.kv[b][sel[sel >= 0].long()]))
                ref[b, t], ref_lse[b, t] = attend64(self.q[b, t].double(), torch.cat(keys))
        check_out(self.out, self.lse, ref, ref_lse)


TREES = [
    dict(B=1, T=1, K=512, W=128, cap=600, ctx=[4000]), dict(B=1, T=5, K=512, W=128, cap=1000, ctx=[4000]),
    dict(B=3, T=7, K=37, W=100, cap=50, ctx=[0, 3, 777], slack=9), dict(B=2, T=64, K=16, W=128, cap=300, ctx=[5, 1000]),
    dict(B=2, T=64, K=0, W=128, ctx=[500, 64]), dict(B=2, T=9, K=0, W=0, ctx=[500, 64]), dict(B=2, T=9, K=1, W=0, cap=1, ctx=[0, 64]),
    dict(B=2, T=31, K=0, W=3, ctx=[500, 1]), dict(B=1, T=6, K=2048, W=1024, cap=2100, ctx=[5000]),
    dict(B=40, T=8, K=64, W=128, cap=100, ctx=[31 * i for i in range(40)]), dict(B=64, T=5, K=0, W=128, ctx=[31 * i for i in range(64)]),
    dict(B=64, T=16, K=0, W=128, ctx=[9 * i for i in range(64)]), dict(B=160, T=10, K=0, W=128, ctx=[5 * i for i in range(160)]),
    dict(B=20, T=40, K=0, W=100, ctx=[30 * i for i in range(20)]), dict(B=110, T=3, K=0, W=4, ctx=[i for i in range(110)]),
    dict(B=70, T=9, K=0, W=0, ctx=[7 * i for i in range(70)]),
    dict(B=20, T=9, K=0, W=0, ctx=[7 * i for i in range(20)]), dict(B=10, T=16, K=0, W=128, ctx=[40 * i for i in range(10)]),
    dict(B=30, T=8, K=0, W=3, ctx=[i for i in range(30)]), dict(B=90, T=1, K=0, W=128, ctx=[3 * i for i in range(90)]),
    dict(B=170, T=2, K=1, W=7, cap=3, ctx=[i for i in range(170)]), dict(B=3, T=64, K=130, W=128, cap=200, ctx=[0, 1, 5000]),
    dict(B=5, T=33, K=200, W=37, cap=201, ctx=[2 ** 31 - 1, 0, 36, 37, 38]), dict(B=20, T=16, K=512, W=128, cap=700, ctx=[900] * 20),
]


@pytest.mark.parametrize("kernel", [0, 1, 2])
@pytest.mark.parametrize("case", TREES, ids=[str(i) for i in range(len(TREES))])
def test_tree(c2, case, kernel):
    t = Tree(c2, **case, seed=31)
    t.call(c2, kernel)
    assert c2.get_device_status() == 0
    t.check()


def test_tree_masks(c2):
    """A token that sees nothing, masks of every bit, bits past the tree's size."""
    t = Tree(c2, 2, 6, 8, 0, [50, 60], cap=20, seed=33)
    t.idx[0, 1] = -1
    t.mask[1] = [(1 << 64) - 1, 1, 1 << 5, 0, 1 << 63 | 1 << 6, (1 << 63) - 1]
    t.put_mask()
    t.call(c2)
    assert c2.get_device_status() == 0
    assert (t.out[0, 1] == 0).all() and torch.isneginf(t.lse[0, 1]).all()
    t.check()


@pytest.mark.parametrize("std", [1e-12, 1e-5, 1e3])
def test_tree_rows_of_any_size(c2, std):
    """8-bit rows much smaller or larger than the entries they share a softmax with."""
    for K in (0, 40):
        t = Tree(c2, 2, 9, K, 128, [300, 20], cap=64, seed=35, std=std, empty=False)
        if std > 1:
            t.q = (t.q.double() / std).bfloat16()
        for kernel in (0, 1, 2):
            t.call(c2, kernel)
            assert c2.get_device_status() == 0
            t.check()


def test_rows_aligned_to_16_bytes_only(c2):
    """Caches whose first byte is 16 past a multiple of 32."""
    def shift(t):
        buf = torch.zeros(t.numel() + 48, dtype=torch.uint8, device="cuda")
        off = 16 + (-buf.data_ptr()) % 32
        new = buf[off:off + t.numel()].view(t.shape)
        new.copy_(t)
        return new

    t = Tree(c2, 20, 8, 50, 128, [20 * i for i in range(20)], cap=64, seed=37)
    for name in ("kv", "swa", "tree"):
        setattr(t, name, shift(getattr(t, name)))
        for kernel in (0, 1, 2):
            t.call(c2, kernel)
            assert c2.get_device_status() == 0
            t.check()
    w = Window([300, 20], [100, 90], 128, 4, seed=38)
    w.swa, w.sink = shift(w.swa), shift(w.sink)
    for kernel in (0, 1, 2):
        w.call(c2, kernel)
        assert c2.get_device_status() == 0
        w.check()


@pytest.mark.parametrize("kernel", [0, 1, 2])
def test_tree_an_index_twice(c2, kernel):
    """An entry that a list names twice is two keys."""
    t = Tree(c2, 3, 5, 300, 64, [300, 20, 0], cap=301, seed=51)
    t.idx[:, :, 150:170] = t.idx[:, :, 7:8]
    t.idx[1, 4] = 3
    t.call(c2, kernel)
    assert c2.get_device_status() == 0
    t.check()


def test_two_streams_at_once(c2):
    """Each kernel beside another one on a stream of its own gives what it gives alone."""
    cases = [Window([300, 20], [700, 500], 128, 4, seed=52), Tree(c2, 40, 8, 200, 128, [9 * i for i in range(40)], cap=210, seed=53),
             Tree(c2, 1, 5, 512, 128, [900], cap=600, seed=54), Tree(c2, 64, 5, 0, 128, [9 * i for i in range(64)], seed=55)]
    ctx = [None] + [ints(t.ctx) for t in cases[1:]]
    calls = [lambda **kw: cases[0].call(c2, **kw)] + [
        (lambda t, c: lambda **kw: t.call(c2, ctx_t=c, **kw))(t, c) for t, c in zip(cases[1:], ctx[1:])]
    for call in calls:
        call()
    torch.cuda.synchronize()
    alone = [(t.out.clone(), t.lse.clone()) for t in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for t in cases:
        t.out.zero_()
        t.lse.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for call, s in zip(calls, streams):
            call(stream=s)
    torch.cuda.synchronize()
    assert c2.get_device_status() == 0
    for t, (out, lse) in zip(cases, alone):
        assert torch.equal(t.out, out) and torch.equal(t.lse, lse)


def test_tree_bad_indices(c2):
    """An index past the cache, a length below zero: reported, no access; the tokens without them are right."""
    t = Tree(c2, 2, 4, 16, 128, [300, 20], cap=64, seed=36, empty=False)
    good = t.idx.clone()
    t.idx[1, 3, 5] = 64
    t.call(c2)
    assert c2.get_device_status() == 2
    out = t.out.clone()
    t.idx = good
    t.call(c2)
    assert c2.get_device_status() == 0
    t.check()
    assert torch.equal(out[0], t.out[0]) and torch.equal(out[1, :3], t.out[1, :3])
    t.call(c2, ctx_t=ints([-1, 20]))
    assert c2.get_device_status() == 2


def test_tree_graph_and_stream(c2):
    a = Tree(c2, 3, 5, 64, 128, [300, 20, 0], cap=100, seed=41)
    b = Tree(c2, 3, 5, 64, 128, [300, 20, 0], cap=100, seed=42)
    ctx = ints([300, 20, 0])
    a.call(c2, ctx_t=ctx)
    first = a.out.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.call(c2, ctx_t=ctx)
    a.out.zero_()
    g.replay()
    assert torch.equal(a.out, first)
    for x in ("q", "kv", "idx", "swa", "scale", "tree", "tree_scale", "mask_t"):
        getattr(a, x).copy_(getattr(b, x))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g.replay()
    b.call(c2, ctx_t=ctx, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)
    b.check()


def test_caches_past_32_bits(c2):
    """Entries and ring rows whose byte offsets pass 2^32."""
    cap = 9_000_000                                   # x 2 x 288 B = 5.2 GB
    kv = torch.zeros(2, cap, ENTRY, dtype=torch.uint8, device="cuda")
    t = Tree(c2, 2, 3, 64, 128, [300, 20], cap=64, seed=51, empty=False)
    at = torch.arange(64, device="cuda") * 1000 + cap - 64_001
    kv[:, at] = t.kv
    old = t.idx
    t.idx = torch.where(old >= 0, at.int()[old.clamp(min=0).long()], old)
    t.kv = kv
    t.call(c2)
    assert c2.get_device_status() == 0
    t.check()
    del t, kv
    w = Window([5, 6000], [4, 150], 128, 4, seed=52)
    ring = 4_500_000                                  # x 2 x 512 B = 4.6 GB
    swa = torch.full((2, ring, D), 0x7F, dtype=torch.uint8, device="cuda")
    scale = torch.full((2, ring), math.nan, device="cuda")
    for b, (c, k) in enumerate(zip(w.ctx, w.new)):
        p = torch.arange(max(0, c - 127), c + k, device="cuda")
        far = ring - 200 if b else 0                  # the second sequence's rows go around the ring's end
        swa[b, (p - 5900 + far) % ring if b else p], scale[b, (p - 5900 + far) % ring if b else p] = \
            w.swa[b, p % w.swa.shape[1]], w.scale[b, p % w.swa.shape[1]]
    w.ctx = [5, 6000 - 5900 + ring - 200]
    w.ctx_t = ints(w.ctx)
    w.swa, w.scale = swa, scale
    w.call(c2)
    assert c2.get_device_status() == 0
    w.check()


# ---------------------------------------------------------------- together
def test_step_runs_through(c2):
    """Lengths -> maps -> window rows and entries written through them -> the
    window-only layer and the drafted tree over what was written; each stage
    against the plain one, two steps in a row."""
    B, W, S, cap, ring = 3, 128, 4, 1000, 200
    swa, scale = torch.full((B, ring, D), 0x7F, dtype=torch.uint8, device="cuda"), torch.full((B, ring), math.nan, device="cuda")
    kv = torch.zeros(B, cap, ENTRY, dtype=torch.uint8, device="cuda")
    sink, sink_scale = torch.zeros(B, S, D, dtype=torch.uint8, device="cuda"), torch.zeros(B, S, device="cuda")
    ctx = [0, 0, 0]
    for step, new in enumerate(([50, 7, 70], [1, 66, 73], [33, 2, 5])):
        maps = c2.slot_maps(B, sum(new))
        c2.slot_map(ints(ctx), ints(new), cap, ring, maps)
        lat = torch.randn(sum(new), D, generator=gen(60 + step), device="cuda").bfloat16()
        c2.swa_quant_write(lat, maps.swa_slot, swa, scale, pos=maps.pos)
        c2.kv_quant_write(lat, None, 1, maps.entry_pos, maps.slot, kv)
        if step == 0:   # the first tokens, kept for good
            sink.copy_(swa[:, :S])
            sink_scale.copy_(scale[:, :S])
        w = Window.__new__(Window)
        w.ctx, w.new, w.W, w.S, w.cu, w.ctx_t = ctx, new, W, S, maps.cu, ints(ctx)
        w.swa, w.scale, w.sink, w.sink_scale = swa, scale, sink, sink_scale
        w.q = queries((sum(new),), 70 + step)
        w.out = torch.full((sum(new), H, D), 7.0, dtype=torch.bfloat16, device="cuda")
        w.lse = torch.full((sum(new), H), 7.0, device="cuda")
        w.call(c2)
        assert c2.get_device_status() == 0
        w.check()
        ctx = [c + k for c, k in zip(ctx, new)]
        assert maps.n_vis.tolist() == ctx and maps.swa_len.tolist() == [min(c, ring) for c in ctx]
    # five drafted tokens: their rows, then the readout over entries, window and tree
    T, K = 5, 40
    t = Tree(c2, B, T, K, W, ctx, cap=50, seed=80)
    depth = torch.tensor([[bin(m).count("1") for m in r] for r in t.mask], device="cuda").clamp_min(1) - 1
    pos = (ints(ctx).long()[:, None] + depth).view(-1)
    lat = torch.randn(B * T, D, generator=gen(81), device="cuda").bfloat16()
    c2.swa_quant_write(lat, torch.arange(B * T, device="cuda"), t.tree, t.tree_scale, pos=pos)
    t.kv, t.swa, t.scale = kv, swa, scale
    t.idx = torch.where(t.idx >= 0, t.idx % 35, t.idx)
    t.call(c2)
    assert c2.get_device_status() == 0
    t.check()
