"""Calls of the step operators, and of the readout they share, at the ends of what
the header allows: queries that are no numbers, entries and rows far smaller than
what they share a softmax with, padded steps, outputs changed in place."""
import copy
import math
import pickle

import pytest
import torch

from test_gpu_step import D, ENTRY, H, Tree, Window, attend64, c2, check_out, entries, gen, ints, kv64, queries, rows64, rows8  # noqa: F401

pytestmark = pytest.mark.gpu

BAD_HEADS = {3: math.nan, 16: math.inf, 17: 1e38, 40: -math.inf}   # (1e38 and infinities are beyond the range of q)


def bad_heads(q):
    """q with some heads that are no numbers, the heads that stay, the others."""
    bad = q.clone()
    for h, v in BAD_HEADS.items():
        bad[..., h, :] = v
    bad[..., 40, 1::2] = 1.0
    rest = [h for h in range(H) if h not in BAD_HEADS]
    return bad, rest


@pytest.mark.parametrize("B,kernel", [(3, 0), (60, 0), (60, 1), (60, 2), (170, 0), (3, 2)])
def test_sparse_attn_heads_of_nan(c2, B, kernel):  # noqa: F811
    """Heads whose logits are no numbers leave the other heads alone, in one block of keys and in several."""
    K, W, cap = 512, 128, 600
    kv = entries(c2, B * cap, 1).view(B, cap, ENTRY)
    idx = torch.stack([torch.randperm(cap, generator=gen(b), device="cuda")[:K].sort().values for b in range(B)]).int()
    swa, scale = rows8((B, W), 2)
    q = queries((B,), 3)
    bad, rest = bad_heads(q)
    p = c2.Params.make(attn_kernel=kernel)
    ws = c2.workspace(c2.OP_ATTN, B, cap, p)
    out, lse = [], []
    for x in (q, bad):
        out.append(torch.empty(B, H, D, device="cuda"))
        lse.append(torch.empty(B, H, device="cuda"))
        c2.sparse_attn(p, x, kv, idx, swa, scale, ints([W] * B), out[-1], ws, lse=lse[-1])
        assert c2.get_device_status() == 0
    assert torch.isfinite(out[0]).all()
    assert torch.equal(out[0][:, rest], out[1][:, rest]) and torch.equal(lse[0][:, rest], lse[1][:, rest])
    assert torch.isnan(out[1][:, 3]).all()


@pytest.mark.parametrize("kernel", [0, 1, 2])
def test_step_heads_of_nan(c2, kernel):  # noqa: F811
    """The same of trees and windows."""
    steps = [Tree(c2, 1, 5, 512, 128, [900], cap=600, seed=4), Tree(c2, 12, 9, 300, 128, [70 * i for i in range(12)], cap=310, seed=5),
             Tree(c2, 1, 2, 2048, 1024, [5000], cap=2100, seed=6), Tree(c2, 40, 8, 0, 128, [9 * i for i in range(40)], seed=7),
             Window([700, 0, 40], [120, 60, 3], 128, 4, seed=8), Window([3000], [2], 1024, 64, seed=9)]
    for s in steps:
        s.call(c2, kernel)
        assert c2.get_device_status() == 0
        out, lse = s.out.clone(), s.lse.clone()
        good, (s.q, rest) = s.q, bad_heads(s.q)
        s.call(c2, kernel)
        assert c2.get_device_status() == 0
        assert torch.equal(s.out[..., rest, :], out[..., rest, :]) and torch.equal(s.lse[..., rest], lse[..., rest])
        seen = ~torch.isneginf(lse[..., 3])
        assert torch.isnan(s.out[..., 3, :][seen].float()).all()
        s.q = good
        s.call(c2, kernel)
        s.check()


@pytest.mark.parametrize("kernel", [0, 2])
def test_many_tokens_of_a_single_step(c2, kernel):  # noqa: F811
    """Tokens of at most 64 keys, several for each CTA, beside some of more."""
    t = Tree(c2, 330, 3, 8, 16, [7 * i for i in range(330)], cap=11, seed=15)
    for _ in range(5):
        t.out.fill_(7.0)
        t.call(c2, kernel)
        assert c2.get_device_status() == 0
    t.check()
    w = Window([0, 900, 20], [300, 1, 400], 16, 4, spare=3, seed=16)
    w.call(c2, kernel)
    assert c2.get_device_status() == 0
    w.check()


@pytest.mark.parametrize("kernel", [0, 1, 2])
@pytest.mark.parametrize("B,T,K", [(1, 6, 40), (2, 9, 0), (60, 4, 200), (50, 7, 0)])
def test_padding_tokens_of_nan(c2, kernel, B, T, K):  # noqa: F811
    """Tokens that see nothing give 0 and -inf whatever their queries hold; the others
    are right."""
    t = Tree(c2, B, T, K, 0, [9 * i for i in range(B)], cap=210 if K else 0, seed=17)
    for b in range(B):
        for i in range(1, T, 2):
            t.mask[b][i] = 0
            if K:
                t.idx[b, i] = -1
    t.put_mask()
    good = t.q.clone()
    for i, v in zip(range(1, T, 2), (math.nan, math.inf, -math.inf)):
        t.q[:, i, 5:] = v
    t.call(c2, kernel)
    assert c2.get_device_status() == 0
    assert (t.out[:, 1::2] == 0).all() and torch.isneginf(t.lse[:, 1::2]).all()
    t.q = good
    t.check()


def scaled_entries(c2, rows, seed, std):  # noqa: F811
    kv = torch.zeros(rows, ENTRY, dtype=torch.uint8, device="cuda")
    at = torch.arange(rows, device="cuda")
    lat = (torch.randn(rows, D, generator=gen(seed), device="cuda") * std).bfloat16()
    c2.kv_quant_write(lat, None, 1, at, at.clone(), kv)
    return kv


@pytest.mark.parametrize("kernel", [0, 1, 2])
@pytest.mark.parametrize("row_std", [1.0, 1e-3, 1e-4, 1e-6, 1e-12])
@pytest.mark.parametrize("entry_std", [0.0, 5e-3, 1.0])
def test_entries_smaller_than_fp16_weights(c2, kernel, row_std, entry_std):  # noqa: F811
    """Entries of zeros or of small values beside rows that are smaller still: a key
    counts by its logit, and what it adds is held to its own size."""
    for B, T, K in ((2, 9, 40), (1, 3, 300), (40, 6, 8), (20, 9, 100)):
        t = Tree(c2, B, T, K, 128, [300 + i for i in range(B)], cap=310, seed=18, std=row_std)
        t.kv = scaled_entries(c2, B * 310, 19, entry_std).view(B, 310, ENTRY)
        t.call(c2, kernel)
        assert c2.get_device_status() == 0
        t.check()


@pytest.mark.parametrize("kernel", [0, 1, 2])
@pytest.mark.parametrize("row_std", [1e3, 1e-2, 1e-6])
def test_entries_and_rows_of_every_scale(c2, kernel, row_std):  # noqa: F811
    """Entries whose scales cover E4M3's range, blocks of zeros under large scales and
    all-zero entries among them; rows of zero codes whose scale is 1."""
    for B, T, K in ((2, 9, 40), (1, 3, 300), (40, 6, 8), (20, 9, 100)):
        t = Tree(c2, B, T, K, 128, [300 + i for i in range(B)], cap=310, seed=20, std=row_std)
        n = B * 310
        kv = torch.randint(0, 256, (n, ENTRY), generator=gen(21), device="cuda", dtype=torch.uint8)
        top = torch.randint(1, 127, (n, 1), generator=gen(22), device="cuda")
        kv[:, 256:] = (torch.rand(n, 32, generator=gen(23), device="cuda") * (top + 1)).long().clamp(max=126).to(torch.uint8)
        kv[::5, :128] = 0                     # the first half's codes, whatever its scales are
        kv[::5, 256:272] = 126
        kv[::5, 272:] = (kv[::5, 272:] & 7)   # and the other half subnormal
        kv[3::7, :256] &= 0x88                # zeros and negative zeros
        kv[4::11, 256:] = 0
        t.kv = kv.view(B, 310, ENTRY)
        t.swa[:, ::9] = 0
        t.scale[:, ::9] = 1.0
        t.tree[:, 1::3] = 0x80
        t.tree_scale[:, 1::3] = 1.0
        t.q = (t.q.float() * 2e-4).bfloat16()   # logits of ordinary size under the largest entries
        t.call(c2, kernel)
        assert c2.get_device_status() == 0
        t.check()


def check_close(out, q, keys_of):
    """Outputs [n, 64, 512] within half a step of bf16 of the formula's, and 2^-13 of the sum
    of the weighted magnitudes: weights of 16 bits (2^-15), logits within 2^-16 at the
    sizes here, exponentials and sums in fp32."""
    for i in range(out.shape[0]):
        keys = keys_of(i)
        r, lse = attend64(q[i].double(), keys)
        w = torch.exp(q[i].double() @ keys.T / math.sqrt(D) - lse[:, None])
        err = 2.0 ** -13 * (w @ keys.abs())
        half = torch.exp2(torch.floor(torch.log2(r.abs() + err)) - 8)
        over = (out[i].double() - r).abs() - half - err
        assert (over <= 0).all(), f"token {i}: off by {(over / err).max().item()} allowances too much"


def test_tile_weights_keep_16_bits_without_a_first_reference(c2):  # noqa: F811
    """Trees without a window whose masks leave out the first 16 rows of both halves:
    each half of a row's softmax finds a reference of its own."""
    B, T = 3, 64
    t = Tree(c2, B, T, 0, 0, [5, 60, 700], seed=24, empty=False)
    g = torch.Generator().manual_seed(25)
    for b in range(B):
        for i in range(T):
            bits = torch.randperm(16, generator=g)[:5].tolist()
            t.mask[b][i] = sum(1 << (16 + k) | 1 << (48 + (5 * k + i) % 16) for k in bits)
    t.put_mask()
    t.call(c2)
    assert c2.get_device_status() == 0
    t.check()
    for b in range(B):
        rows = rows64(t.tree[b], t.tree_scale[b])
        check_close(t.out[b], t.q[b], lambda i: rows[[u for u in range(T) if t.mask[b][i] >> u & 1]])


def test_tile_weights_keep_16_bits_when_a_reference_is_raised(c2):  # noqa: F811
    """A window with a row 2^39 and a later one 2^41 above the first ones of a softmax thread."""
    B, T, W = 3, 64, 64
    t = Tree(c2, B, T, 0, W, [64, 64, 64], seed=26, empty=False)
    sign = torch.where(torch.rand(D, generator=gen(27), device="cuda") < 0.5, -1.0, 1.0)
    level = torch.zeros(W, device="cuda")
    level[20], level[40] = 38.4 / 41, 40.6 / 41
    x = level[:, None] * sign + torch.randn(B, W, D, generator=gen(28), device="cuda") * 0.2
    t.scale = x.abs().amax(-1) / 448
    t.swa = (x / t.scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    t.q = (sign * (41 * math.log(2) / math.sqrt(D))).bfloat16().expand(B, T, H, D).contiguous()
    t.mask = [[0] * T for _ in range(B)]
    t.put_mask()
    t.call(c2)
    assert c2.get_device_status() == 0
    t.check()
    for b in range(B):
        rows = rows64(t.swa[b], t.scale[b])   # (position p in row p: rings of W rows, W tokens)
        logit = t.q[b, 0, 0].double() @ rows.T / math.sqrt(D) / math.log(2) + torch.log2(t.scale[b].double())
        first, mid, top = logit[:16].max(), logit[16:32].max(), logit[32:48].max()
        assert mid < first + 40 < top and mid > top - 3.5
        check_close(t.out[b], t.q[b], lambda i: rows)


def test_writers_skip_places_without_a_row(c2):  # noqa: F811
    """Slot -1 is no row and no error, whatever position and values stand beside it;
    slots below it and past the cache are reported."""
    lat = torch.randn(40, D, generator=gen(30), device="cuda").bfloat16()
    pos = torch.arange(40, device="cuda")
    slot = torch.randperm(64, generator=gen(31), device="cuda")[:40]
    use = torch.arange(40, device="cuda") % 3 != 0
    gaps, gap_pos, gap_lat = torch.where(use, slot, -1), torch.where(use, pos, -1), torch.where(use[:, None], lat, math.nan)
    w_ik = torch.randn(128, D, generator=gen(32), device="cuda").bfloat16()
    key = torch.randn(40, 128, generator=gen(33), device="cuda").bfloat16()

    def write(lat, pos, slot, key):
        swa, scale = torch.full((64, D), 9, dtype=torch.uint8, device="cuda"), torch.full((64,), 9.0, device="cuda")
        kv, kv2 = (torch.full((64, ENTRY), 9, dtype=torch.uint8, device="cuda") for _ in range(2))
        k_bf, k_f4 = torch.full((64, 128), 9.0, dtype=torch.bfloat16, device="cuda"), c2.indexer_k_fp4_cache(64)
        bits = []
        for call in (lambda: c2.swa_quant_write(lat, slot, swa, scale, pos=pos), lambda: c2.kv_quant_write(lat, None, 1, pos, slot, kv),
                     lambda: c2.kv_quant_write_ik(lat, None, 1, pos, slot, kv2, w_ik, k_bf), lambda: c2.indexer_k_quant(key, slot, k_f4)):
            call()
            bits.append(c2.get_device_status())
        return (swa, scale, kv, kv2, k_bf, k_f4), bits

    want, bits = write(lat[use], pos[use], slot[use], key[use])
    assert bits == [0] * 4
    got, bits = write(gap_lat, gap_pos, gaps, key)
    assert bits == [0] * 4
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    for bad in (-2, 64, -(1 << 62)):
        got, bits = write(gap_lat, gap_pos, torch.where(pos == 1, bad, gaps), key)
        assert bits == [2] * 4
        rest = torch.ones(64, dtype=torch.bool, device="cuda")
        rest[slot[1]] = False
        assert all(torch.equal(x[rest], y[rest]) for x, y in zip(got[:5], want[:5]))


@pytest.mark.parametrize("m", [1, 2])
def test_padded_steps_leave_the_status_clear(c2, m):  # noqa: F811
    """Maps of more places than tokens, and steps longer than the rings: the writers take
    them as they are, nothing is reported, and the rings hold the last positions."""
    B, W, S, cap, ring, n = 3, 128, 2, 1200, 140, 900
    swa, scale = torch.full((B, ring, D), 0x7F, dtype=torch.uint8, device="cuda"), torch.full((B, ring), math.nan, device="cuda")
    kv = torch.zeros(B, cap, ENTRY, dtype=torch.uint8, device="cuda")
    texts = [torch.randn(1000, D, generator=gen(34 + b), device="cuda").bfloat16() for b in range(B)]
    maps, ctx = c2.slot_maps(B, n, m), [0] * B
    c2.get_device_status()
    for step, new in enumerate(([500, 7, 300], [1, 0, 12], [11, 1, 1])):
        c2.slot_map(ints(ctx), ints(new), cap, ring, maps, m=m)
        lat = torch.full((n, D), math.nan, dtype=torch.bfloat16, device="cuda")
        lat[:sum(new)] = torch.cat([texts[b][c:c + k] for b, (c, k) in enumerate(zip(ctx, new))])
        c2.swa_quant_write(lat, maps.swa_slot, swa, scale, pos=maps.pos)
        e = maps.slot.numel()
        pair = torch.full((e, m, D), math.nan, dtype=torch.bfloat16, device="cuda")
        done = [(b, p) for b, (c, k) in enumerate(zip(ctx, new)) for p in range(c, c + k) if p % m == m - 1]
        pair[:len(done)] = torch.stack([texts[b][p - m + 1:p + 1] for b, p in done])
        c2.kv_quant_write(pair if m == 2 else pair[:, 0].contiguous(), torch.zeros_like(pair) if m == 2 else None, m,
                          maps.entry_pos, maps.slot, kv)
        assert c2.get_device_status() == 0
        before, ctx = ctx, [c + k for c, k in zip(ctx, new)]
        for b in range(B):
            p = torch.arange(max(0, ctx[b] - ring), ctx[b], device="cuda")
            one, one_scale = torch.zeros(len(p), D, dtype=torch.uint8, device="cuda"), torch.zeros(len(p), device="cuda")
            c2.swa_quant_write(texts[b][p], torch.arange(len(p), device="cuda"), one, one_scale, pos=p)
            assert torch.equal(swa[b, p % ring], one) and torch.equal(scale[b, p % ring], one_scale)
            pe = torch.arange(ctx[b] // m, device="cuda")
            src = texts[b][:len(pe) * m].view(-1, m, D)
            whole = torch.zeros(len(pe), ENTRY, dtype=torch.uint8, device="cuda")
            c2.kv_quant_write(src if m == 2 else src[:, 0].contiguous(), torch.zeros_like(src) if m == 2 else None, m, m * pe + m - 1, pe, whole)
            assert torch.equal(kv[b, :len(pe)], whole)
        if step:   # (a ring shorter than its step has lost rows that the first one's tokens see)
            w = Window.__new__(Window)
            w.ctx, w.new, w.W, w.S, w.cu, w.ctx_t = before, new, W, 0, maps.cu, ints(before)
            w.swa, w.scale, w.sink, w.sink_scale = swa, scale, swa[:, :0], scale[:, :0]
            w.q = queries((n,), 40 + step)
            w.out = torch.full((n, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
            w.lse = torch.full((n, H), 7.0, device="cuda")
            w.call(c2)
            assert c2.get_device_status() == 0
            w.check()


def test_slot_map_outputs_changed_in_place(c2):  # noqa: F811
    """An output that is resized, or set to other memory, between two calls is the one that the
    next call checks and writes."""
    ctx, new = ints([5, 0, 9]), ints([3, 4, 1])
    maps = c2.slot_maps(3, 12)
    c2.slot_map(ctx, new, 100, 128, maps)
    assert maps.pos.tolist() == [5, 6, 7, 0, 1, 2, 3, 9] + [-1] * 4
    other = torch.full((40,), 77, dtype=torch.int64, device="cuda")
    maps.pos.set_(other[8:20])
    c2.slot_map(ctx, new + 1, 100, 128, maps)
    want = [5, 6, 7, 8, 0, 1, 2, 3, 4, 9, 10, -1]
    assert maps.pos.tolist() == want and other[8:20].tolist() == want
    assert (other[:8] == 77).all() and (other[20:] == 77).all()
    maps.slot.set_(torch.full((12,), 55, dtype=torch.int64, device="cuda"))
    c2.slot_map(ctx, new, 100, 128, maps)
    assert maps.slot.tolist() == [5, 6, 7, 100, 101, 102, 103, 209] + [-1] * 4
    for name, change in (("swa_slot", lambda t: t.resize_(11)), ("pos", lambda t: t.resize_(400)),
                         ("cu", lambda t: t.set_(torch.zeros(5, dtype=torch.int32, device="cuda"))),
                         ("n_vis", lambda t: setattr(t, "data", torch.zeros(3, dtype=torch.int64, device="cuda"))),
                         ("slot", lambda t: t.set_(torch.zeros(24, dtype=torch.int64, device="cuda")[::2])),
                         ("tok_seq", lambda t: setattr(t, "data", torch.zeros(12, dtype=torch.int32)))):
        maps = c2.slot_maps(3, 12)
        c2.slot_map(ctx, new, 100, 128, maps)
        change(getattr(maps, name))
        with pytest.raises(c2.Csa2Error):
            c2.slot_map(ctx, new, 100, 128, maps)
    with pytest.raises(c2.Csa2Error):   # maps of another batch
        c2.slot_map(ints([1, 2]), ints([1, 1]), 100, 128, c2.slot_maps(3, 12))
    assert c2.get_device_status() == 0


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda m: pickle.loads(pickle.dumps(m))], ids=["copy", "deepcopy", "pickle"])
def test_slot_maps_are_copied_after_a_call(c2, how):  # noqa: F811
    ctx, new = ints([5, 0, 9]), ints([3, 4, 1])
    maps = c2.slot_maps(3, 12)
    c2.slot_map(ctx, new, 100, 128, maps)
    twin = how(maps)
    assert type(twin) is type(maps) and not twin.__dict__ and all(torch.equal(x, y) for x, y in zip(maps, twin))
    kept = [t.clone() for t in maps]
    c2.slot_map(ctx + 1, new, 100, 128, twin)
    assert twin.pos.tolist() == [6, 7, 8, 1, 2, 3, 4, 10] + [-1] * 4
    if how is not copy.copy:   # (a copy of the tuple names the same tensors)
        assert all(torch.equal(x, y) for x, y in zip(maps, kept))


@pytest.mark.parametrize("kernel", [0, 1, 2])
@pytest.mark.parametrize("new", [[30, 4], [100, 90], [170, 60]])
def test_a_short_ring_leaves_the_other_sequences_right(c2, kernel, new):  # noqa: F811
    """A sequence whose ring has lost rows, or whose length is negative, is reported by every
    kernel, and the one beside it comes out as it should."""
    w = Window([500, 40], new, 128, 4, seed=43)
    w.swa, w.scale = w.swa[:, :130].contiguous(), w.scale[:, :130].contiguous()
    ref, ref_lse, n = w.reference()
    for first in (500, -3):
        w.ctx_t = ints([first, 40])
        w.out.fill_(7.0)
        w.call(c2, kernel)
        assert c2.get_device_status() == 2
        check_out(w.out[new[0]:], w.lse[new[0]:], ref[new[0]:], ref_lse[new[0]:])


def test_slot_map_lengths_in_place_are_refused(c2):  # noqa: F811
    """The counts that a step gives do not take the place of its lengths; next to them they may lie."""
    maps = c2.slot_maps(3, 12)
    with pytest.raises(c2.Csa2Error):
        c2.slot_map(maps.n_vis, ints([1, 2, 3]), 100, 128, maps)
    both = torch.zeros(9, dtype=torch.int32, device="cuda")
    ctx, new = both[:3], both[6:]
    ctx += 5
    new += 2
    maps = maps._replace(n_vis=both[3:6])
    c2.slot_map(ctx, new, 100, 128, maps)
    assert both.tolist() == [5] * 3 + [7] * 3 + [2] * 3 and c2.get_device_status() == 0


@pytest.mark.parametrize("kernel", [0, 1, 2])
def test_rows_nobody_names_hold_anything(c2, kernel):  # noqa: F811
    """Rows of a tree, a ring and sinks that no mask or window reaches: NaN codes, scales of
    NaN, infinity and below zero."""
    odd = torch.tensor([math.nan, math.inf, -math.inf, -1.0], device="cuda")
    for B, T, K in ((2, 9, 0), (40, 8, 0), (40, 8, 30), (1, 5, 300)):
        t = Tree(c2, B, T, K, 16, [3 * i for i in range(B)], cap=310 if K else 0, seed=45, slack=4)
        for b in range(B):
            for i in range(T):
                t.mask[b][i] &= ~(1 << (T - 1) | 1 << 2)
        t.put_mask()
        t.tree[:, [2, T - 1]] = 0x7F
        t.tree_scale[:, 2], t.tree_scale[:, T - 1] = odd[torch.arange(B, device="cuda") % 4], odd[torch.arange(B, device="cuda") % 3]
        for b, c in enumerate(t.ctx):
            far = [p % 20 for p in range(c, max(c, 20))] if c < 20 else [p % 20 for p in range(c - 20, c - 16)]
            t.swa[b, far], t.scale[b, far] = 0xFF, odd[b % 4]
        t.call(c2, kernel)
        assert c2.get_device_status() == 0
        t.check()


@pytest.mark.parametrize("kernel", [0, 1, 2])
def test_scales_at_the_ends_of_their_range(c2, kernel):  # noqa: F811
    """Rows whose scales are 2^50, 2^-64, less, and 0, in one softmax (queries of zeros:
    equal weights; then ones under which one row takes all)."""
    for new in (1, 160):
        w = Window([200, 100], [new, new], 128, 4, seed=46)
        for i, s in enumerate((2.0 ** 50, 2.0 ** 49, 1.0, 2.0 ** -64, 2.0 ** -70, 0.0)):
            w.scale[:, i::6] = torch.where(torch.isnan(w.scale[:, i::6]), math.nan, s)
        w.q.zero_()
        w.call(c2, kernel)
        assert c2.get_device_status() == 0
        w.check()
        w.scale[w.scale <= 1.0] = 0.0
        w.q = torch.full_like(w.q, 2.0 ** -24)   # (logits far apart: one key takes all)
        w.call(c2, kernel)
        assert c2.get_device_status() == 0
        w.check()
