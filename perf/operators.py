"""Workloads of the quantised-cache and dense-readout operators.

Four operators over the caches of this package (main-KV entries of 288 bytes:
512 E2M1 codes and one E4M3 scale per 16 channels; sliding-window rows of 512
E4M3 codes and one fp32 scale; indexer keys as MXFP4 planes):

* ``write``: sliding-window rows written as FP8 (RoPE on the last 64 channels,
  scale = amax / 448), ``swa_quant_write``;
* ``read``: entries read back as bf16 rows, by a list of positions or in
  order, ``kv_read`` / ``swa_read`` / ``indexer_k_read``;
* ``prefix``: the decode readout of a batch whose sequences share one long
  prefix, with each sequence's selected entries and window, in one softmax,
  ``prefix_attn``;
* ``cross``: queries of one length over every entry of another sequence's
  cache (an encoder's entries, a length per sequence), ``cross_attn``.

``run`` computes them in elementary torch operations, or, with ``own`` set,
through the package's calls.
"""
import math

import torch

own = False

D, H, ROPE = 512, 64, 64
ENTRY = 288


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 32 sequences: each writes its new row into its 128-row window
        {"name": "write_decode_32", "op": "write", "n": 32, "rows": 4096, "rope": True},
        # the window rows of a 2 x 16,384-token prefill chunk with 127 rows before it
        {"name": "write_prefill_2x16k", "op": "write", "n": 32768, "rows": 33022, "rope": True},
        # the entries that 32 sequences' indexers selected (lists of 512, some padded)
        {"name": "read_kv_topk_32x512", "op": "read", "fmt": "kv", "batch": 32, "cap": 16384, "k": 512, "listed": True},
        # a whole 256K-entry cache copy read back in order
        {"name": "read_kv_all_256k", "op": "read", "fmt": "kv", "batch": 1, "cap": 262144, "k": 262144, "listed": False},
        # one sequence's window
        {"name": "read_swa_1x128", "op": "read", "fmt": "swa", "batch": 1, "cap": 128, "k": 128, "listed": False},
        # the smallest shared prompt: one sequence after a short prefix
        {"name": "prefix_1x500", "op": "prefix", "batch": 1, "n_prefix": 500, "k": 512, "window": 128},
        # one sequence on a long prefix: few rows, a long axis
        {"name": "prefix_1x64k", "op": "prefix", "batch": 1, "n_prefix": 65536, "k": 512, "window": 128},
        # a batch of 32 on one 64K prompt, the decode group's shape
        {"name": "prefix_32x64k", "op": "prefix", "batch": 32, "n_prefix": 65536, "k": 512, "window": 128},
        # an odd batch on an odd prefix
        {"name": "prefix_7x10001", "op": "prefix", "batch": 7, "n_prefix": 10001, "k": 512, "window": 128},
        # one new token of each of 4 sequences over an encoder's entries
        {"name": "cross_4x1x4096", "op": "cross", "batch": 4, "n_q": 1, "n_max": 4096, "ragged": True},
        # a prompt of 128 tokens over short encodings of different lengths, one of them empty
        {"name": "cross_8x128x1500", "op": "cross", "batch": 8, "n_q": 128, "n_max": 1500, "ragged": True},
        # the largest: 512 tokens of each of 2 sequences over 16K entries
        {"name": "cross_2x512x16k", "op": "cross", "batch": 2, "n_q": 512, "n_max": 16384, "ragged": False},
    ]


MOST_PAIRS = 2 * 512 * 16384   # (query token, entry) pairs of the largest listed case


def _log(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "prefix", "prefix", "cross", "cross"])
    if op == "write":
        n = _log(rng, 1, 32768)
        return {"op": op, "n": n, "rows": n + _log(rng, 1, 4096), "rope": rng.random() < 0.7}
    if op == "read":
        fmt = rng.choice(["kv", "swa", "ik"])
        batch = _log(rng, 1, 64)
        k = _log(rng, 1, 262144 // batch)
        cap = -(-(k + rng.randrange(0, 1000)) // 4) * 4   # MXFP4 planes hold a multiple of 4 rows
        return {"op": op, "fmt": fmt, "batch": batch, "cap": cap, "k": k, "listed": rng.random() < 0.6}
    if op == "prefix":
        batch = _log(rng, 1, 64)
        return {"op": op, "batch": batch, "n_prefix": _log(rng, 1, min(131072, MOST_PAIRS // batch)),
                "k": rng.choice([1, 37, 256, 512]), "window": rng.choice([0, 1, 100, 128])}
    batch = _log(rng, 1, 16)
    n_q = _log(rng, 1, 512 // batch)
    return {"op": op, "batch": batch, "n_q": n_q, "n_max": _log(rng, 1, min(65536, MOST_PAIRS // (batch * n_q))),
            "ragged": rng.random() < 0.7}


def _lengths(case):
    """Visible entries of each sequence of a cross case: down to half of n_max, the last of a ragged batch empty."""
    b, n = case["batch"], case["n_max"]
    if not case["ragged"]:
        return [n] * b
    return [0 if i and i == b - 1 else n - (i * n) // (2 * b) for i in range(b)]


def _owned(case):
    """(selected entries, window rows) of each sequence of a prefix case: full, but for the second sequence, which has none of its own yet."""
    return [(0, 0) if i == 1 else (case["k"], case["window"]) for i in range(case["batch"])]


# ------------------------------------------------------------------ inputs
def _gen(seed, stream):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000 + stream)
    return g


def _randn(shape, seed, stream):
    return torch.randn(*shape, generator=_gen(seed, stream), device="cuda")


_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _e2m1_codes(y):
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=y.device)
    return torch.bucketize(y.abs(), mids, out_int32=True).to(torch.uint8) | ((y < 0).to(torch.uint8) << 3)


def _kv_entries(rows, seed, stream):
    """Main-KV entries of N(0, 1) latents: uint8 [rows, 288]."""
    x = _randn((rows, 32, 16), seed, stream)
    s = (x.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn)
    c = _e2m1_codes(x.div_(s.float().unsqueeze(-1))).view(rows, 256, 2)
    return torch.cat([c[..., 0] | (c[..., 1] << 4), s.view(torch.uint8)], 1)


def _swa_rows(shape, seed, stream):
    x = _randn((*shape, D), seed, stream)
    s = x.abs().amax(-1) / 448.0
    return (x / s.unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s


def _ik_planes(rows, seed, stream):
    """MXFP4 indexer keys of N(0, 1) rows: codes [rows][64], then exponent bytes [rows][4]."""
    x = _randn((rows, 4, 32), seed, stream)
    e = torch.floor(torch.log2(x.abs().amax(-1))) - 2
    c = _e2m1_codes(x * torch.exp2(-e).unsqueeze(-1)).view(rows, 64, 2)
    return torch.cat([(c[..., 0] | (c[..., 1] << 4)).reshape(-1), (e + 127).to(torch.uint8).reshape(-1)])


def _queries(shape, seed, stream):
    """bf16 queries whose heads are of different sharpness (logits of spread 0.5 to 3)."""
    sharp = torch.linspace(0.5, 3.0, H, device="cuda").unsqueeze(-1)
    return (_randn((*shape, H, D), seed, stream) * sharp).to(torch.bfloat16)


def _positions(batch, cap, k, seed, stream):
    """k distinct positions below cap for each sequence, ascending, int32 [batch, k]."""
    r = torch.rand(batch, cap, generator=_gen(seed, stream), device="cuda")
    return r.topk(k, dim=1, sorted=False).indices.sort(dim=1).values.to(torch.int32)


def prepare(case, seed):
    op, s = case["op"], {"case": case}
    if op == "write":
        n, rows = case["n"], case["rows"]
        s["latent"] = _randn((n, D), seed, 1).to(torch.bfloat16)
        s["slot"] = torch.rand(rows, generator=_gen(seed, 2), device="cuda").argsort()[:n]
        s["pos"] = torch.randint(0, 1 << 20, (n,), generator=_gen(seed, 3), device="cuda") if case["rope"] else None
        s["swa"], s["swa_scale"] = _swa_rows((rows,), seed, 4)
    elif op == "read":
        batch, cap, k = case["batch"], case["cap"], case["k"]
        s["idx"] = None
        if case["listed"]:
            s["idx"] = torch.randint(0, cap, (batch, k), generator=_gen(seed, 5), device="cuda", dtype=torch.int32)
            s["idx"][batch // 2, (k + 1) // 2:] = -1   # a sequence that selected fewer
        if case["fmt"] == "kv":
            s["kv"] = _kv_entries(batch * cap, seed, 100).view(batch, cap, ENTRY)
        elif case["fmt"] == "swa":
            s["swa"], s["swa_scale"] = _swa_rows((batch, cap), seed, 6)
        else:
            s["ik"] = _ik_planes(batch * cap, seed, 7)
        s["out"] = torch.empty(batch, k, 128 if case["fmt"] == "ik" else D, dtype=torch.bfloat16, device="cuda")
    elif op == "prefix":
        batch, k, w = case["batch"], case["k"], case["window"]
        cap = 2 * k
        s["q"] = _queries((batch,), seed, 8)
        s["prefix"] = _kv_entries(case["n_prefix"], seed, 200)
        s["kv"] = _kv_entries(batch * cap, seed, 9).view(batch, cap, ENTRY)
        s["idx"] = _positions(batch, cap, k, seed, 10)
        s["swa"], s["swa_scale"] = _swa_rows((batch, w), seed, 11)
        s["swa_len"] = torch.tensor([x[1] for x in _owned(case)], dtype=torch.int32, device="cuda")
        if batch > 1:
            s["idx"][1] = -1
        s["out"] = torch.empty(batch, H, D, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(batch, H, device="cuda")
        if own:   # the scratch buffer that a caller keeps
            import sparse_attention_fp4_csa2_gb300 as c2
            s["params"] = c2.Params.make(index_topk=k, sliding_window=w)
            s["ws"] = c2.workspace(c2.OP_PREFIX, batch, case["n_prefix"], s["params"])
    else:
        batch, n_q, n = case["batch"], case["n_q"], case["n_max"]
        s["q"] = _queries((batch, n_q), seed, 12)
        s["kv"] = _kv_entries(batch * n, seed, 300).view(batch, n, ENTRY)
        s["n_vis"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
        # rows past a sequence's length were never written: here every byte is a NaN's
        s["kv"][torch.arange(n, device="cuda") >= s["n_vis"].unsqueeze(1)] = 0xFF
        s["out"] = torch.empty(batch, n_q, H, D, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(batch, n_q, H, device="cuda")
        if own:   # the scratch buffer that a caller keeps
            import sparse_attention_fp4_csa2_gb300 as c2
            s["ws"] = c2.workspace(c2.OP_CROSS, batch * n_q, n, c2.Params.make())
    return s


# ------------------------------------------------------------- plain forms
def _rotated(x, pos):
    """RoPE on the last 64 channels as interleaved pairs: angles in 64 bits, rotation in 32."""
    inv = (10000.0 ** (-2.0 * torch.arange(ROPE // 2, dtype=torch.float64, device=x.device) / ROPE)).float()
    ang = pos.double().unsqueeze(-1) * inv.double()
    c, s = ang.cos().float(), ang.sin().float()
    a, b = x[..., D - ROPE::2], x[..., D - ROPE + 1::2]
    return torch.cat([x[..., :D - ROPE], torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)], -1)


def _fp4_values(codes):
    """uint8 [..., n] of two E2M1 codes each -> fp32 [..., 2 n]."""
    lut = torch.tensor(_LEVELS + tuple(-v for v in _LEVELS), device=codes.device)
    return lut[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]


def _kv_values(kv):
    """uint8 [..., 288] -> fp32 [..., 512]."""
    v = _fp4_values(kv[..., :256]).unflatten(-1, (32, 16))
    return (v * kv[..., 256:].contiguous().view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _swa_values(swa, scale):
    return swa.view(torch.float8_e4m3fn).float() * scale.unsqueeze(-1)


def _ik_values(planes, rows):
    v = _fp4_values(planes[:rows * 64].view(rows, 64)).unflatten(-1, (4, 32))
    e = planes[rows * 64:].view(rows, 4).float() - 127.0
    return (v * torch.exp2(e).unsqueeze(-1)).flatten(-2)


def _softmax(logits):
    """(weights, log-sum-exp) over the last axis; -inf is a masked key, a row of them has weights 0."""
    m = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    lse = torch.where(l > 0, m + torch.log(l), torch.full_like(l, -math.inf))
    return torch.where(l > 0, p / l, torch.zeros_like(p)), lse.squeeze(-1)


def _plain_write(s):
    x = s["latent"].float()
    if s["pos"] is not None:
        x = _rotated(x, s["pos"])
    scale = x.abs().amax(-1) / torch.full((), 448.0, device=x.device)
    y = torch.where(scale.unsqueeze(-1) > 0, x / scale.unsqueeze(-1), torch.zeros_like(x))
    s["swa"][s["slot"]] = y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    s["swa_scale"][s["slot"]] = scale
    return s["swa"].view(torch.float8_e4m3fn), s["swa_scale"]


def _plain_read(s):
    case, idx = s["case"], s["idx"]
    batch, cap, k = case["batch"], case["cap"], case["k"]
    at = torch.arange(k, device="cuda").expand(batch, k) if idx is None else idx.clamp(min=0).long()
    b = torch.arange(batch, device="cuda").unsqueeze(1)
    if case["fmt"] == "kv":
        v = _kv_values(s["kv"][b, at])
    elif case["fmt"] == "swa":
        v = _swa_values(s["swa"][b, at], s["swa_scale"][b, at])
    else:
        v = _ik_values(s["ik"], batch * cap).view(batch, cap, 128)[b, at]
    if idx is not None:
        v = torch.where((idx >= 0).unsqueeze(-1), v, torch.zeros_like(v))
    s["out"].copy_(v)
    return s["out"]


def _plain_prefix(s):
    q, idx, w = s["q"].float() * (1.0 / math.sqrt(D)), s["idx"], s["swa"].shape[1]
    batch = q.shape[0]
    pre = _kv_values(s["prefix"])
    sel = _kv_values(s["kv"][torch.arange(batch, device="cuda").unsqueeze(1), idx.clamp(min=0).long()])
    win = _swa_values(s["swa"], s["swa_scale"])
    no_sel, no_win = idx < 0, torch.arange(w, device="cuda") >= s["swa_len"].unsqueeze(1)
    logits = torch.cat([
        (q.view(-1, D) @ pre.T).view(batch, H, -1),
        torch.bmm(q, sel.transpose(1, 2)).masked_fill(no_sel.unsqueeze(1), -math.inf),
        torch.bmm(q, win.transpose(1, 2)).masked_fill(no_win.unsqueeze(1), -math.inf)], -1)
    p, lse = _softmax(logits)
    n, k = pre.shape[0], idx.shape[1]
    out = (p[..., :n].reshape(-1, n) @ pre).view(batch, H, D) + torch.bmm(p[..., n:n + k], sel) + torch.bmm(p[..., n + k:], win)
    return s["out"].copy_(out), s["lse"].copy_(lse)


def _plain_cross(s):
    q, n = s["q"].float() * (1.0 / math.sqrt(D)), s["kv"].shape[1]
    batch, n_q = q.shape[:2]
    past = torch.arange(n, device="cuda") >= s["n_vis"].unsqueeze(1)
    k = _kv_values(s["kv"]).masked_fill(past.unsqueeze(-1), 0.0)
    logits = torch.bmm(q.view(batch, n_q * H, D), k.transpose(1, 2)).masked_fill(past.unsqueeze(1), -math.inf)
    p, lse = _softmax(logits)
    return s["out"].copy_(torch.bmm(p, k).view_as(s["out"])), s["lse"].copy_(lse.view(batch, n_q, H))


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import sparse_attention_fp4_csa2_gb300 as c2
        if op == "write":
            c2.swa_quant_write(s["latent"], s["slot"], s["swa"], s["swa_scale"], pos=s["pos"])
            return s["swa"].view(torch.float8_e4m3fn), s["swa_scale"]
        if op == "read":
            fmt = s["case"]["fmt"]
            if fmt == "kv":
                c2.kv_read(s["kv"], s["out"], idx=s["idx"])
            elif fmt == "swa":
                c2.swa_read(s["swa"], s["swa_scale"], s["out"], idx=s["idx"])
            else:
                c2.indexer_k_read(s["ik"], s["out"], idx=s["idx"])
            return s["out"]
        if op == "prefix":
            c2.prefix_attn(s["params"], s["q"], s["prefix"], s["kv"], s["idx"], s["swa"], s["swa_scale"],
                           s["swa_len"], s["out"], s["ws"], lse=s["lse"])
        else:
            c2.cross_attn(s["q"], s["kv"], s["n_vis"], s["case"]["n_max"], s["out"], s["ws"], lse=s["lse"])
        return s["out"], s["lse"]
    if op == "write":
        return _plain_write(s)
    if op == "read":
        return _plain_read(s)
    if op == "prefix":
        return _plain_prefix(s)
    return _plain_cross(s)


# --------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "write":
        n = case["n"]
        return {"bytes": n * (2 * D + 8 + (8 if case["rope"] else 0) + D + 4), "flops": n * 4 * D}
    if op == "read":
        n = case["batch"] * case["k"]
        row, width = {"kv": (ENTRY, D), "swa": (D + 4, D), "ik": (68, 128)}[case["fmt"]]
        return {"bytes": n * (row + 2 * width + (4 if case["listed"] else 0)), "flops": n * width}
    if op == "prefix":
        n, batch = case["n_prefix"], case["batch"]
        sel, win = (sum(x[i] for x in _owned(case)) for i in (0, 1))
        return {"bytes": n * ENTRY + sel * ENTRY + win * (D + 4) + 4 * batch * (case["k"] + 1) + batch * H * (4 * D + 4),
                "flops": 4 * D * H * (batch * n + sel + win)}
    n, tokens = sum(_lengths(case)), case["batch"] * case["n_q"]
    return {"bytes": n * ENTRY + 4 * case["batch"] + tokens * H * (4 * D + 4), "flops": 4 * D * H * case["n_q"] * n}


# -------------------------------------------------------------------- exact
def _nibbles(b):
    """E2M1 by its bits (sign, two exponent bits of bias 1, one fraction bit), in 64 bits: low nibble first."""
    c = torch.stack([b % 16, b // 16], -1).flatten(-2).to(torch.int64)
    e, f = (c // 2) % 4, (c % 2).double()
    mag = torch.where(e > 0, (1.0 + f / 2) * 2.0 ** (e - 1).double(), f / 2)
    return torch.where(c >= 8, -mag, mag)


def _e4m3(b):
    """E4M3 by its bits (bias 7), in 64 bits; finite codes only."""
    c = b.to(torch.int64)
    e, f = (c // 8) % 16, (c % 8).double()
    mag = torch.where(e > 0, (1.0 + f / 8) * 2.0 ** (e - 7).double(), f / 8 * 2.0 ** -6)
    return torch.where(c >= 128, -mag, mag)


def _entries64(kv):
    return _nibbles(kv[..., :256]) * _e4m3(kv[..., 256:]).repeat_interleave(16, dim=-1)


def _attend64(q, keys, seen):
    """softmax(q . k / sqrt(512)) k over the seen keys, in 64 bits: q [rows, 512], keys [n, 512], seen [n]."""
    keys = keys[seen]
    if not keys.shape[0]:
        return torch.zeros_like(q), torch.full(q.shape[:1], -math.inf, dtype=torch.float64, device=q.device)
    logits = q @ keys.T / math.sqrt(D)
    lse = torch.logsumexp(logits, -1)
    return torch.exp(logits - lse.unsqueeze(-1)) @ keys, lse


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "write":
        x = s["latent"].double()
        if s["pos"] is not None:
            j = torch.arange(ROPE // 2, device="cuda")
            turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                               s["pos"].double()[:, None] * (10000.0 ** (-j.double() / 32)).float().double())
            tail = torch.view_as_complex(x[:, D - ROPE:].reshape(-1, ROPE // 2, 2).contiguous()) * turn
            x = torch.cat([x[:, :D - ROPE], torch.view_as_real(tail).reshape(-1, ROPE)], 1)
        scale = x.abs().max(-1).values / 448
        codes, scales = _e4m3(s["swa"]), s["swa_scale"].double()
        codes[s["slot"]] = x / scale.clamp_min(1e-300)[:, None]
        scales[s["slot"]] = scale
        return codes, scales
    if op == "read":
        batch, cap, k = case["batch"], case["cap"], case["k"]
        rows = torch.arange(batch, device="cuda")[:, None] * cap + (torch.arange(k, device="cuda")[None] if s["idx"] is None else s["idx"].clamp_min(0))
        rows = rows.reshape(-1)
        if case["fmt"] == "kv":
            v = _entries64(s["kv"].view(-1, ENTRY)[rows])
        elif case["fmt"] == "swa":
            v = _e4m3(s["swa"].view(-1, D)[rows]) * s["swa_scale"].view(-1)[rows].double()[:, None]
        else:
            codes, exps = s["ik"][:batch * cap * 64].view(-1, 64)[rows], s["ik"][batch * cap * 64:].view(-1, 4)[rows]
            v = _nibbles(codes) * (2.0 ** (exps.double() - 127)).repeat_interleave(32, dim=-1)
        if s["idx"] is not None:
            v[s["idx"].reshape(-1) < 0] = 0
        return v.view(batch, k, -1)
    outs, lses = [], []
    if op == "prefix":
        pre = _entries64(s["prefix"])
        for b in range(case["batch"]):
            sel, w = s["idx"][b], s["swa_len"][b]
            keys = torch.cat([pre, _entries64(s["kv"][b][sel[sel >= 0].long()]), _e4m3(s["swa"][b, :w]) * s["swa_scale"][b, :w].double()[:, None]])
            o, l = _attend64(s["q"][b].double(), keys, torch.ones(keys.shape[0], dtype=torch.bool, device="cuda"))
            outs.append(o)
            lses.append(l)
    else:
        for b in range(case["batch"]):
            n = int(s["n_vis"][b])
            keys = _entries64(s["kv"][b, :n])
            o, l = _attend64(s["q"][b].double().view(-1, D), keys, torch.ones(n, dtype=torch.bool, device="cuda"))
            outs.append(o.view(case["n_q"], H, D))
            lses.append(l.view(case["n_q"], H))
    return torch.stack(outs), torch.stack(lses)
