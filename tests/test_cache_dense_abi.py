"""Host-side checks of the window writer, the read-backs and the dense
readouts: what they refuse, and what is a no-op, without a GPU."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def c2():
    import sparse_attention_fp4_csa2_gb300.build as b
    b.build()
    import sparse_attention_fp4_csa2_gb300 as c
    return c


FAKE, ODD, WS = 0x1000, 0x1001, 0x1100   # never dereferenced: the checks fail first
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.mark.parametrize("change,want", [
    (dict(n=-1), INVALID), (dict(rows=-1), INVALID), (dict(latent=None), INVALID), (dict(latent=ODD), INVALID),
    (dict(slot=None), INVALID), (dict(swa=None), INVALID), (dict(swa=ODD), INVALID), (dict(scale=None), INVALID),
    (dict(theta=1.0), INVALID), (dict(theta=float("nan")), INVALID), (dict(theta=float("inf")), INVALID),
    (dict(n=1 << 40), UNSUPPORTED), (dict(n=0, latent=None, slot=None, swa=None, scale=None), OK)])
def test_swa_write_refusals(c2, change, want):
    a = dict(latent=FAKE, n=4, pos=FAKE, slot=FAKE, swa=FAKE, scale=FAKE, rows=8, theta=10000.0) | change
    assert c2.lib().csa2_swa_quant_write(a["latent"], a["n"], a["pos"], a["slot"], a["swa"], a["scale"], a["rows"],
                                         a["theta"], None) == want
    assert c2.last_launch_count() == 0


@pytest.mark.parametrize("change,want", [
    (dict(batch=-1), INVALID), (dict(cap=-1), INVALID), (dict(k=-1), INVALID), (dict(cache=None), INVALID),
    (dict(cache=ODD), INVALID), (dict(out=None), INVALID), (dict(out=ODD), INVALID), (dict(idx=None, k=17), INVALID),
    (dict(cap=1 << 40), UNSUPPORTED), (dict(k=1 << 40), UNSUPPORTED), (dict(batch=0, out=None, cache=None), OK),
    (dict(k=0, out=None, cache=None), OK)])
def test_read_refusals(c2, change, want):
    a = dict(cache=FAKE, batch=2, cap=16, idx=FAKE, k=4, out=FAKE) | change
    L = c2.lib()
    assert L.csa2_kv_read(a["cache"], a["batch"], a["cap"], a["idx"], a["k"], a["out"], None) == want
    assert L.csa2_swa_read(a["cache"], FAKE, a["batch"], a["cap"], a["idx"], a["k"], a["out"], None) == want
    assert L.csa2_indexer_k_read(a["cache"], a["batch"], a["cap"], a["idx"], a["k"], a["out"], None) == want
    assert c2.last_launch_count() == 0


def test_read_refusals_of_one_format(c2):
    L = c2.lib()
    assert L.csa2_swa_read(FAKE, None, 2, 16, FAKE, 4, FAKE, None) == INVALID
    assert L.csa2_indexer_k_read(FAKE, 1, 6, FAKE, 4, FAKE, None) == INVALID   # planes of 4 n rows


@pytest.mark.parametrize("change,want", [
    (dict(batch=-1), INVALID), (dict(n_q=-1), INVALID), (dict(n_max=101), INVALID), (dict(n_max=-1), INVALID),
    (dict(q=None), INVALID), (dict(q=ODD), INVALID), (dict(kv=None), INVALID), (dict(kv=ODD), INVALID),
    (dict(n_vis=None), INVALID), (dict(out=None), INVALID), (dict(out=ODD), INVALID), (dict(ws=None), INVALID),
    (dict(ws=0x1010), INVALID), (dict(ws_bytes=1024), WORKSPACE), (dict(batch=1 << 20, n_q=1 << 10), UNSUPPORTED),
    (dict(cap=1 << 40), UNSUPPORTED), (dict(batch=0, q=None, out=None), OK), (dict(n_q=0, q=None, out=None), OK)])
def test_cross_refusals(c2, change, want):
    a = dict(batch=2, n_q=3, q=FAKE, kv=FAKE, cap=100, n_vis=FAKE, n_max=100, out=FAKE, lse=None, ws=WS,
             ws_bytes=1 << 40) | change
    assert c2.lib().csa2_cross_attn(a["batch"], a["n_q"], a["q"], a["kv"], a["cap"], a["n_vis"], a["n_max"], a["out"],
                                    a["lse"], a["ws"], a["ws_bytes"], None) == want
    assert c2.last_launch_count() == 0


@pytest.mark.parametrize("change,want", [
    (dict(batch=0), INVALID), (dict(batch=65536), INVALID), (dict(n_prefix=-1), INVALID), (dict(q=None), INVALID),
    (dict(q=ODD), INVALID), (dict(pre=None), INVALID), (dict(pre=ODD), INVALID), (dict(kv=None), INVALID),
    (dict(kv=ODD), INVALID), (dict(cap=0), INVALID), (dict(idx=None), INVALID), (dict(swa=None), INVALID),
    (dict(out=None), INVALID), (dict(out=ODD), INVALID), (dict(ws=None), INVALID), (dict(ws=0x1010), INVALID),
    (dict(ws_bytes=1 << 19), WORKSPACE), (dict(n_prefix=1 << 40), UNSUPPORTED),
    (dict(params=dict(index_topk=0)), UNSUPPORTED), (dict(params=dict(sliding_window=2000)), UNSUPPORTED)])
def test_prefix_refusals(c2, change, want):
    a = dict(params={}, batch=2, q=FAKE, pre=FAKE, n_prefix=100, kv=FAKE, cap=600, idx=FAKE, swa=FAKE, scale=FAKE,
             len=FAKE, out=FAKE, lse=None, ws=WS, ws_bytes=1 << 40) | change
    p = c2.Params.make(**a["params"])
    assert c2.lib().csa2_prefix_attn(ctypes.byref(p), a["batch"], a["q"], a["pre"], a["n_prefix"], a["kv"], a["cap"],
                                     a["idx"], a["swa"], a["scale"], a["len"], a["out"], a["lse"], a["ws"],
                                     a["ws_bytes"], None) == want
    assert c2.last_launch_count() == 0


def test_workspaces(c2):
    p = c2.Params.make()
    # two partials of two tokens (64 rows of 512 fp16 and a log-sum-exp) and
    # 16 bytes for the combine per worker: one worker at least, one per 256 entries of a token, 76 at most
    unit = 2 * 2 * 64 * (512 * 2 + 4) + 16
    for tokens, n, workers in ((1, 0, 1), (1, 256, 1), (1, 257, 2), (3, 1000, 12), (5000, 1, 76), (1 << 24, 1 << 31, 76)):
        assert c2.workspace_bytes(c2.OP_CROSS, tokens, n, p) == workers * unit
    one, many = (c2.workspace_bytes(c2.OP_PREFIX, b, 1 << 20, p) for b in (1, 65))
    # 64 sequences more: their own part's fp32 rows and log-sum-exps
    assert many - one == 64 * 64 * (512 + 1) * 4
    assert c2.workspace_bytes(c2.OP_PREFIX, 1, 0, c2.Params.make(index_topk=0)) == 0
    assert c2.workspace_bytes(c2.OP_CROSS, 0, 100, p) == 0


def test_binding_refuses_host_tensors(c2):
    z = torch.zeros
    with pytest.raises(c2.Csa2Error):
        c2.swa_quant_write(z(1, 512, dtype=torch.bfloat16), z(1, dtype=torch.int64), z(4, 512, dtype=torch.uint8), z(4))
    with pytest.raises(c2.Csa2Error):   # 3 scales for 4 rows
        c2.swa_quant_write(z(1, 512, dtype=torch.bfloat16), z(1, dtype=torch.int64), z(4, 512, dtype=torch.uint8), z(3))
    with pytest.raises(c2.Csa2Error):
        c2.kv_read(z(1, 4, 288, dtype=torch.uint8), z(1, 4, 512, dtype=torch.bfloat16))
    with pytest.raises(c2.Csa2Error):
        c2.swa_read(z(1, 4, 512, dtype=torch.uint8), z(1, 4), z(1, 4, 512, dtype=torch.bfloat16))
    with pytest.raises(c2.Csa2Error):
        c2.indexer_k_read(z(4 * 68, dtype=torch.uint8), z(1, 4, 128, dtype=torch.bfloat16))
    with pytest.raises(c2.Csa2Error):   # 6 rows are no 4 sequences
        c2.indexer_k_read(z(6 * 68, dtype=torch.uint8), z(4, 1, 128, dtype=torch.bfloat16))
    with pytest.raises(c2.Csa2Error):
        c2.cross_attn(z(1, 1, 64, 512, dtype=torch.bfloat16), z(1, 4, 288, dtype=torch.uint8), z(1, dtype=torch.int32), 4,
                      z(1, 1, 64, 512, dtype=torch.bfloat16), z(1, dtype=torch.uint8))
    with pytest.raises(c2.Csa2Error):
        c2.prefix_attn(c2.Params.make(), z(1, 64, 512, dtype=torch.bfloat16), z(4, 288, dtype=torch.uint8),
                       z(1, 600, 288, dtype=torch.uint8), z(1, 512, dtype=torch.int32), z(1, 128, 512, dtype=torch.uint8),
                       z(1, 128), z(1, dtype=torch.int32), z(1, 64, 512, dtype=torch.bfloat16), z(1, dtype=torch.uint8))
