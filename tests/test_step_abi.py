"""Host-side checks of the slot maps, the windowed and the tree attention: what
they refuse, and what is a no-op, without a GPU."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def c2():
    import sparse_attention_fp4_csa2_gb300.build as b
    b.build()
    import sparse_attention_fp4_csa2_gb300 as c
    return c


FAKE, ODD = 0x1000, 0x1001   # never dereferenced: the checks fail first
OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.mark.parametrize("change,want", [
    (dict(batch=-1), INVALID), (dict(m=0), INVALID), (dict(m=3), INVALID), (dict(cap=-1), INVALID), (dict(ring=0), INVALID),
    (dict(n=-1), INVALID), (dict(e=-1), INVALID), (dict(ctx=None), INVALID), (dict(new=None), INVALID),
    (dict(cu=None), INVALID), (dict(tok=None), INVALID), (dict(pos=None), INVALID), (dict(swa=None), INVALID),
    (dict(ecu=None), INVALID), (dict(epos=None), INVALID), (dict(slot=None), INVALID), (dict(vis=None), INVALID),
    (dict(len=None), INVALID), (dict(ctx=ODD), INVALID), (dict(tok=ODD), INVALID), (dict(pos=0x1004), INVALID),
    (dict(slot=0x1004), INVALID), (dict(batch=8193), UNSUPPORTED), (dict(n=1 << 31), UNSUPPORTED),
    (dict(e=1 << 31), UNSUPPORTED), (dict(cap=1 << 40), UNSUPPORTED), (dict(ring=1 << 40), UNSUPPORTED),
    (dict(batch=0, ctx=None, new=None, cu=None), OK)])
def test_slot_map_refusals(c2, change, want):
    a = dict(batch=2, ctx=FAKE, new=FAKE, m=1, cap=100, ring=128, n=10, e=10, cu=FAKE, tok=FAKE, pos=FAKE, swa=FAKE,
             ecu=FAKE, epos=FAKE, slot=FAKE, vis=FAKE, len=FAKE) | change
    v = list(a.values())
    out = (ctypes.c_void_p * 9)(*v[8:])
    assert c2.lib().csa2_slot_map(*v[:8], ctypes.addressof(out), None) == want
    assert c2.last_launch_count() == 0


def test_slot_map_without_outputs(c2):
    assert c2.lib().csa2_slot_map(2, FAKE, FAKE, 1, 100, 128, 10, 10, None, None) == INVALID


@pytest.mark.parametrize("change,want", [
    (dict(batch=-1), INVALID), (dict(n=-1), INVALID), (dict(rows=-1), INVALID), (dict(rows=127), INVALID),
    (dict(ns=-1), INVALID), (dict(q=None), INVALID), (dict(q=ODD), INVALID), (dict(cu=None), INVALID),
    (dict(ctx=None), INVALID), (dict(swa=None), INVALID), (dict(swa=ODD), INVALID), (dict(scale=None), INVALID),
    (dict(sink=None), INVALID), (dict(sink=ODD), INVALID), (dict(sink_scale=None), INVALID), (dict(out=None), INVALID),
    (dict(out=ODD), INVALID), (dict(cu=0x1002), INVALID), (dict(scale=0x1002), INVALID), (dict(lse=0x1002), INVALID),
    (dict(n=1 << 25), UNSUPPORTED), (dict(batch=(1 << 24) + 1), UNSUPPORTED),
    (dict(batch=2 ** 31 - 1, params=dict(sliding_window=0), swa=None, scale=None, rows=0), UNSUPPORTED), (dict(ns=65), UNSUPPORTED), (dict(rows=1 << 40), UNSUPPORTED),
    (dict(params=dict(sliding_window=2000)), UNSUPPORTED), (dict(params=dict(attn_kernel=3)), UNSUPPORTED),
    (dict(batch=0, q=None, out=None), OK), (dict(n=0, q=None, out=None), OK)])
def test_window_refusals(c2, change, want):
    a = dict(params={}, batch=2, n=3, q=FAKE, cu=FAKE, ctx=FAKE, swa=FAKE, scale=FAKE, rows=200, sink=FAKE,
             sink_scale=FAKE, ns=4, out=FAKE, lse=None) | change
    p = c2.Params.make(**a.pop("params"))
    assert c2.lib().csa2_window_attn(ctypes.byref(p), *a.values(), None) == want
    assert c2.last_launch_count() == 0


@pytest.mark.parametrize("change,want", [
    (dict(batch=-1), INVALID), (dict(t=-1), INVALID), (dict(cap=-1), INVALID), (dict(cap=0), INVALID),
    (dict(q=None), INVALID), (dict(q=ODD), INVALID), (dict(kv=None), INVALID), (dict(kv=ODD), INVALID),
    (dict(swa=None), INVALID), (dict(swa=ODD), INVALID), (dict(scale=None), INVALID), (dict(rows=127), INVALID),
    (dict(ctx=None), INVALID), (dict(tree=None), INVALID), (dict(tree=ODD), INVALID), (dict(tree_scale=None), INVALID),
    (dict(mask=None), INVALID), (dict(mask=0x1004), INVALID), (dict(out=None), INVALID), (dict(out=ODD), INVALID),
    (dict(idx=0x1002), INVALID), (dict(ctx=0x1002), INVALID), (dict(tree_scale=0x1002), INVALID),
    (dict(t=65), UNSUPPORTED), (dict(batch=1 << 20, t=64), UNSUPPORTED), (dict(cap=1 << 40), UNSUPPORTED),
    (dict(rows=1 << 40), UNSUPPORTED), (dict(params=dict(index_topk=0)), UNSUPPORTED),
    (dict(batch=0, q=None, out=None), OK), (dict(t=0, q=None, out=None), OK)])
def test_tree_refusals(c2, change, want):
    a = dict(params={}, batch=2, t=5, q=FAKE, kv=FAKE, cap=600, idx=FAKE, swa=FAKE, scale=FAKE, rows=128, ctx=FAKE,
             tree=FAKE, tree_scale=FAKE, mask=FAKE, out=FAKE, lse=None) | change
    p = c2.Params.make(**a.pop("params"))
    assert c2.lib().csa2_tree_attn(ctypes.byref(p), *a.values(), None) == want
    assert c2.last_launch_count() == 0


def test_bindings_take_cuda_tensors_only(c2):
    i32 = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 64, 512, dtype=torch.bfloat16)
    p = c2.Params.make()
    with pytest.raises(c2.Csa2Error):
        c2.slot_map(i32, i32, 10, 10, c2.slot_maps(2, 4, device="cpu"))
    with pytest.raises(c2.Csa2Error):
        c2.window_attn(p, q, i32, i32, None, None, q)
    with pytest.raises(c2.Csa2Error):
        c2.tree_attn(p, q[None], None, None, None, None, i32, None, None, None, q[None])
    with pytest.raises(c2.Csa2Error):
        c2.slot_maps(2, 4, m=3, device="cpu")


@pytest.mark.parametrize("batch,n,m,entries", [(3, 7, 1, 7), (3, 7, 2, 5), (1, 1, 2, 1), (4, 0, 2, 2), (0, 0, 1, 0)])
def test_slot_map_buffers(c2, batch, n, m, entries):
    """At m = 2 every sequence may complete one entry more than half its new tokens."""
    s = c2.slot_maps(batch, n, m, device="cpu")
    assert s.pos.numel() == s.swa_slot.numel() == s.tok_seq.numel() == n
    assert s.slot.numel() == s.entry_pos.numel() == entries
    assert s.cu.numel() == s.entry_cu.numel() == batch + 1 and s.n_vis.numel() == s.swa_len.numel() == batch
