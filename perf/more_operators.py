"""Workloads of the step operators: slot maps, windowed attention, drafted trees.

Three operators around one serving step of the cache (main-KV entries of 288
bytes: 512 E2M1 codes and one E4M3 scale per 16 channels; sliding-window rows of
512 E4M3 codes and one fp32 scale, kept in a ring where position p has row p mod
ring):

* ``slots``: from the requests' lengths, the positions and cache rows that the
  writers take, and the visible counts, ``slot_map``;
* ``window``: packed query tokens over their causal sliding window and the first
  few tokens that stay visible (sinks), ``window_attn``;
* ``tree``: drafted tokens over their selected entries, the committed window and
  the drafted tokens that each one descends from, in one softmax, ``tree_attn``.

``run`` computes them in elementary torch operations, or, with ``own`` set,
through the package's calls.
"""
import math

import torch

own = False

D, H = 512, 64
ENTRY = 288


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step of 32 sequences: one new token each
        {"name": "slots_decode_32", "op": "slots", "batch": 32, "new": 1, "ragged": False, "m": 1, "spare": 0},
        # a drafted step of a large odd batch, five tokens each, in buffers sized for more
        {"name": "slots_draft_999x5", "op": "slots", "batch": 999, "new": 5, "ragged": False, "m": 1, "spare": 125},
        # prompts of up to 4,096 tokens (some empty) at two tokens an entry
        {"name": "slots_prefill_64x4k", "op": "slots", "batch": 64, "new": 4096, "ragged": True, "m": 2, "spare": 1000},
        # one token of each of 32 sequences in a window-only layer
        {"name": "window_decode_32", "op": "window", "batch": 32, "new": 1, "ragged": False, "ctx": 5000, "window": 128, "sinks": 4, "spare": 0},
        # prompts of different lengths, the first one fresh and one of them empty, in a buffer with rows to spare
        {"name": "window_ragged_9", "op": "window", "batch": 9, "new": 501, "ragged": True, "ctx": 333, "window": 100, "sinks": 3, "spare": 17},
        # a prefill chunk of two sequences in a window-only layer
        {"name": "window_prefill_2x8k", "op": "window", "batch": 2, "new": 8192, "ragged": False, "ctx": 100000, "window": 128, "sinks": 4, "spare": 0},
        # five drafted tokens of one sequence: the smallest verification
        {"name": "tree_1x5", "op": "tree", "batch": 1, "tree": 5, "k": 512, "cap": 4096, "window": 128, "ctx": 4000},
        # a small odd batch of long drafts at the start of their texts, short lists, a short window
        {"name": "tree_3x31_short", "op": "tree", "batch": 3, "tree": 31, "k": 37, "cap": 1000, "window": 100, "ctx": 50},
        # eight drafted tokens of each of 32 sequences
        {"name": "tree_32x8", "op": "tree", "batch": 32, "tree": 8, "k": 512, "cap": 16384, "window": 128, "ctx": 16000},
        # a draft block of window-only layers: no entries, five tokens of each of 64 sequences
        {"name": "tree_draft_64x5", "op": "tree", "batch": 64, "tree": 5, "k": 0, "cap": 0, "window": 128, "ctx": 9000},
        # the largest: 64 drafted tokens of each of 32 sequences
        {"name": "tree_32x64", "op": "tree", "batch": 32, "tree": 64, "k": 512, "cap": 16384, "window": 128, "ctx": 16000},
    ]


def _log(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["slots", "window", "window", "tree", "tree"])
    if op == "slots":
        batch = _log(rng, 1, 1024)
        return {"op": op, "batch": batch, "new": _log(rng, 1, 262144 // batch), "ragged": rng.random() < 0.6,
                "m": rng.choice([1, 2]), "spare": rng.choice([0, rng.randrange(1, 300)])}
    if op == "window":
        batch = _log(rng, 1, 128)
        return {"op": op, "batch": batch, "new": _log(rng, 1, 16384 // batch), "ragged": rng.random() < 0.6,
                "ctx": rng.choice([0, _log(rng, 1, 1000000)]), "window": rng.choice([1, 37, 100, 128, 128]),
                "sinks": rng.choice([0, 1, 4, 8]), "spare": rng.choice([0, rng.randrange(1, 40)])}
    batch, k = _log(rng, 1, 64), rng.choice([0, 1, 37, 256, 512, 512])
    return {"op": op, "batch": batch, "tree": _log(rng, 1, min(64, 2048 // batch)), "k": k,
            "cap": k and _log(rng, max(k, 64), 16384), "window": rng.choice([0, 1, 37, 100, 128, 128]), "ctx": _log(rng, 1, 1000000)}


def _new(case):
    """New tokens of each sequence: down to half of the most, one sequence of a ragged batch with none."""
    b, n = case["batch"], case["new"]
    if not case["ragged"]:
        return [n] * b
    return [0 if i and i == b // 2 else max(1, n - (i * n) // (2 * b)) for i in range(b)]


def _ctx(case):
    """Tokens before the step, of each sequence; the first one of a ragged batch is fresh."""
    c = case.get("ctx", 20000)
    return [0 if case.get("ragged") and i == 0 else c + (17 * i) % 97 for i in range(case["batch"])]


def _unseen(b, t):
    """Drafted tokens that see nothing at all yet (padding of a fixed-size tree)."""
    return b % 5 == 2 and t % 4 == 3


def _seen(case):
    """(positions seen, entries listed) summed over the tokens of a window or tree case."""
    if case["op"] == "window":
        w, s = case["window"], case["sinks"]
        total = 0
        for c, n in zip(_ctx(case), _new(case)):
            for p in (range(c, c + n) if n < 2048 and c < 4096 else ()):
                total += min(p + 1, w) + min(s, max(0, p + 1 - w))
            if not (n < 2048 and c < 4096):   # beyond the start of a text every token sees the same number (fresh long texts: nearly)
                total += n * (w + s)
        return total, 0
    tokens = case["batch"] * case["tree"] - sum(_unseen(b, t) for b in range(case["batch"]) for t in range(case["tree"]))
    return tokens * min(case["window"], case["ctx"]), tokens * case["k"]


# ------------------------------------------------------------------ inputs
def _gen(seed, stream):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000 + stream)
    return g


def _randn(shape, seed, stream):
    return torch.randn(*shape, generator=_gen(seed, stream), device="cuda")


_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _kv_entries(rows, seed, stream):
    """Main-KV entries of N(0, 1) latents: uint8 [rows, 288]."""
    x = _randn((rows, 32, 16), seed, stream)
    s = (x.abs().amax(-1) / 6.0).to(torch.float8_e4m3fn)
    y = x.div_(s.float().unsqueeze(-1))
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    c = (torch.bucketize(y.abs(), mids, out_int32=True).to(torch.uint8) | ((y < 0).to(torch.uint8) << 3)).view(rows, 256, 2)
    return torch.cat([c[..., 0] | (c[..., 1] << 4), s.view(torch.uint8)], 1)


def _swa_rows(shape, seed, stream):
    x = _randn((*shape, D), seed, stream)
    s = x.abs().amax(-1) / 448.0
    return (x / s.unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s


def _queries(shape, seed, stream):
    """bf16 queries whose heads are of different sharpness (logits of spread 0.5 to 3)."""
    sharp = torch.linspace(0.5, 3.0, H, device="cuda").unsqueeze(-1)
    return _randn((*shape, H, D), seed, stream).mul_(sharp).to(torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _ring_unwritten(s, ring):
    """Ring rows whose position was never written hold NaN codes: a token that reads one shows it."""
    b = s["swa"].shape[0]
    last = s["ctx"].long() + s["new"].long() if "new" in s else s["ctx"].long()
    rows = torch.arange(ring, device="cuda").expand(b, ring)
    unused = rows >= last.unsqueeze(1)   # a text shorter than the ring
    s["swa"][unused] = 0x7F
    s["swa_scale"][unused] = float("nan")


def prepare(case, seed):
    op, s = case["op"], {"case": case}
    batch = case["batch"]
    s["ctx"] = _ints(_ctx(case))
    if op == "slots":
        # the lengths differ from step to step: each request is some way into its text
        s["new"] = _ints(_new(case))
        s["ctx"] = s["ctx"] + torch.randint(0, 4096, (batch,), generator=_gen(seed, 1), device="cuda", dtype=torch.int32)
        n = sum(_new(case)) + case["spare"]
        s["n"], s["n_entries"] = n, n if case["m"] == 1 else (n + batch) // 2
        s["cap"], s["ring"] = 32768 + case["new"], case["new"] + 127
        if own:
            import sparse_attention_fp4_csa2_gb300 as c2
            s["maps"] = c2.slot_maps(batch, n, case["m"])
    elif op == "window":
        new, w, k = _new(case), case["window"], case["sinks"]
        n, ring = sum(new) + case["spare"], w - 1 + max(new)
        s["new"] = _ints(new)
        s["cu"] = _ints([sum(new[:i]) for i in range(batch + 1)])
        s["q"] = _queries((n,), seed, 2)
        s["swa"], s["swa_scale"] = _swa_rows((batch, ring), seed, 3)
        _ring_unwritten(s, ring)
        s["sink"], s["sink_scale"] = _swa_rows((batch, k), seed, 4) if k else (None, None)
        s["out"] = torch.full((n, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.full((n, H), 7.0, device="cuda")
    else:
        t, k, cap, w = case["tree"], case["k"], case["cap"], case["window"]
        ring = max(w, 1) + 5
        s["q"] = _queries((batch, t), seed, 5)
        s["kv"] = _kv_entries(batch * cap, seed, 100).view(batch, cap, ENTRY) if k else None
        s["idx"] = None
        pad = torch.tensor([[_unseen(b, i) for i in range(t)] for b in range(batch)], device="cuda")
        if k:
            r = torch.rand(batch, cap, generator=_gen(seed, 6), device="cuda").argsort(1).to(torch.int32)
            at = torch.randint(0, cap, (batch, t, 1), generator=_gen(seed, 7), device="cuda")
            at = (at + torch.arange(k, device="cuda")) % cap   # a run of a random order: k distinct entries for each token
            s["idx"] = torch.gather(r, 1, at.view(batch, t * k)).view(batch, t, k)
            s["idx"] = s["idx"].sort(-1).values
            s["idx"][:, t // 2, (k + 1) // 2:] = -1            # a token that selected fewer
            s["idx"][pad] = -1
        s["swa"], s["swa_scale"] = _swa_rows((batch, ring), seed, 8)
        _ring_unwritten(s, ring)
        s["tree"], s["tree_scale"] = _swa_rows((batch, t), seed, 9)
        # a random tree: each token hangs on an earlier one or on the text; a token's mask names itself and its ancestors
        mask = torch.zeros(batch, t, dtype=torch.int64, device="cuda")
        u = torch.rand(batch, t, generator=_gen(seed, 10), device="cuda")
        for i in range(t):
            up = (u[:, i] * (i + 1)).long().clamp(max=i) - 1
            above = mask.gather(1, up.clamp(min=0).unsqueeze(1)).squeeze(1) * (up >= 0)
            mask[:, i] = above | torch.full((), 1 << i if i < 63 else -(1 << 63), dtype=torch.int64, device="cuda")
        s["mask"] = mask
        # the padding of a tree: tokens that name no row; with a window they still see the text, without one nothing
        s["mask"][pad] = 0
        s["out"] = torch.empty(batch, t, H, D, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(batch, t, H, device="cuda")
    if own and op != "slots":
        import sparse_attention_fp4_csa2_gb300 as c2
        s["params"] = c2.Params.make(index_topk=max(case.get("k", 1), 1), sliding_window=case["window"])
    return s


# ------------------------------------------------------------- plain forms
def _fp4_values(codes):
    lut = torch.tensor(_LEVELS + tuple(-v for v in _LEVELS), device=codes.device)
    return lut[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]


def _kv_values(kv):
    """uint8 [..., 288] -> fp32 [..., 512]."""
    v = _fp4_values(kv[..., :256]).unflatten(-1, (32, 16))
    return (v * kv[..., 256:].contiguous().view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _swa_values(swa, scale):
    return swa.view(torch.float8_e4m3fn).float() * scale.unsqueeze(-1)


def _softmax(logits):
    """(weights, log-sum-exp) over the last axis; -inf is a masked key, a row of them has weights 0."""
    m = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    lse = torch.where(l > 0, m + torch.log(l), torch.full_like(l, -math.inf))
    return torch.where(l > 0, p / l, torch.zeros_like(p)), lse.squeeze(-1)


def _attend(q, keys, seen):
    """q [n, 64, 512] (bf16), keys [n, k, 512], seen [n, k]: rows and log-sum-exps in 32 bits; unseen keys may hold anything."""
    keys = torch.where(seen.unsqueeze(-1), keys, torch.zeros_like(keys))
    logits = torch.bmm(q.float() * (1.0 / math.sqrt(D)), keys.transpose(1, 2)).masked_fill(~seen.unsqueeze(1), -math.inf)
    p, lse = _softmax(logits)
    return torch.bmm(p, keys), lse


def _plain_slots(s):
    case, ctx, new = s["case"], s["ctx"].long(), s["new"].long()
    batch, m, cap, ring = case["batch"], case["m"], s["cap"], s["ring"]
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")

    def rows(counts, n):
        cu = torch.cat([zero, counts.cumsum(0)])
        i = torch.arange(n, device="cuda")
        b = (torch.searchsorted(cu, i, right=True) - 1).clamp(max=batch - 1)
        return cu, b, i - cu[b], i < cu[-1]

    cu, b, r, live = rows(new, s["n"])
    p = ctx[b] + r
    tok_seq = torch.where(live, b, -1)
    pos = torch.where(live, p, -1)
    swa_slot = torch.where(live & (new[b] - r <= ring), b * ring + p % ring, -1)
    e0, e1 = ctx // m, (ctx + new) // m
    cu_e, b, r, live = rows(e1 - e0, s["n_entries"])
    e = e0[b] + r
    entry_pos = torch.where(live, m * e + m - 1, -1)
    slot = torch.where(live & (e < cap), b * cap + e, -1)
    return (cu.int(), tok_seq.int(), pos, swa_slot, cu_e.int(), entry_pos, slot, e1.clamp(max=cap).int(),
            (ctx + new).clamp(max=ring).int())


def _plain_window(s):
    case, ring, k = s["case"], s["swa"].shape[1], s["case"]["sinks"]
    w, total = case["window"], sum(_new(case))
    i = torch.arange(total, device="cuda")
    b = torch.searchsorted(s["cu"].long(), i, right=True) - 1
    p = s["ctx"].long()[b] + i - s["cu"].long()[b]
    for lo in range(0, total, 1024):
        bb, pp = b[lo:lo + 1024].unsqueeze(1), p[lo:lo + 1024].unsqueeze(1)
        at = pp - (w - 1) + torch.arange(w, device="cuda")
        seen = at >= 0
        row = at.clamp(min=0) % ring
        keys = _swa_values(s["swa"][bb, row], s["swa_scale"][bb, row])
        if k:
            first = torch.arange(k, device="cuda").expand(pp.shape[0], k)
            keys = torch.cat([_swa_values(s["sink"][bb, first], s["sink_scale"][bb, first]), keys], 1)
            seen = torch.cat([first < pp - (w - 1), seen], 1)
        out, lse = _attend(s["q"][lo:lo + 1024][:pp.shape[0]], keys, seen)
        s["out"][lo:lo + pp.shape[0]] = out.to(torch.bfloat16)
        s["lse"][lo:lo + pp.shape[0]] = lse
    return s["out"], s["lse"]


def _plain_tree(s):
    case, mask, idx = s["case"], s["mask"], s["idx"]
    batch, t, w, ring = case["batch"], case["tree"], case["window"], s["swa"].shape[1]
    bits = (mask.unsqueeze(-1) >> torch.arange(t, device="cuda")) & 1 == 1     # [batch, t, t]
    left = (w - bits.sum(-1)).clamp(min=0)                                     # committed rows that the window still holds
    ctx = s["ctx"].long().view(batch, 1, 1)
    at = ctx - w + torch.arange(w, device="cuda").view(1, 1, w)                # [batch, 1, w]
    in_window = (at >= 0) & (at >= ctx - left.unsqueeze(-1))                   # [batch, t, w]
    row = at.clamp(min=0).squeeze(1) % ring
    bb = torch.arange(batch, device="cuda").unsqueeze(1)
    window = _swa_values(s["swa"][bb, row], s["swa_scale"][bb, row])           # [batch, w, 512]
    own_rows = _swa_values(s["tree"], s["tree_scale"])
    step = max(1, 1024 // t)
    for lo in range(0, batch, step):
        hi = min(batch, lo + step)
        n = (hi - lo) * t
        keys = [x[lo:hi].unsqueeze(1).expand(-1, t, -1, -1).reshape(n, -1, D) for x in (window, own_rows)]
        seen = [in_window[lo:hi].reshape(n, w), bits[lo:hi].reshape(n, t)]
        if idx is not None:
            keys.append(_kv_values(s["kv"][bb[lo:hi].unsqueeze(-1), idx[lo:hi].clamp(min=0).long()]).view(n, -1, D))
            seen.append((idx[lo:hi] >= 0).view(n, -1))
        out, lse = _attend(s["q"][lo:hi].reshape(n, H, D), torch.cat(keys, 1), torch.cat(seen, 1))
        s["out"][lo:hi] = out.view(hi - lo, t, H, D).to(torch.bfloat16)
        s["lse"][lo:hi] = lse.view(hi - lo, t, H)
    return s["out"], s["lse"]


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import sparse_attention_fp4_csa2_gb300 as c2
        if op == "slots":
            c2.slot_map(s["ctx"], s["new"], s["cap"], s["ring"], s["maps"], m=s["case"]["m"])
            return tuple(s["maps"])
        if op == "window":
            c2.window_attn(s["params"], s["q"], s["cu"], s["ctx"], s["swa"], s["swa_scale"], s["out"], sink=s["sink"],
                           sink_scale=s["sink_scale"], lse=s["lse"])
        else:
            c2.tree_attn(s["params"], s["q"], s["kv"], s["idx"], s["swa"], s["swa_scale"], s["ctx"], s["tree"],
                         s["tree_scale"], s["mask"], s["out"], lse=s["lse"])
        return s["out"], s["lse"]
    if op == "slots":
        return _plain_slots(s)
    return _plain_window(s) if op == "window" else _plain_tree(s)


# --------------------------------------------------------------------- work
def work(case):
    op, batch = case["op"], case["batch"]
    if op == "slots":
        n = sum(_new(case)) + case["spare"]
        entries = n if case["m"] == 1 else (n + batch) // 2
        return {"bytes": batch * 24 + 8 + n * 20 + entries * 16, "flops": 4 * n + 4 * entries}
    seen, listed_entries = _seen(case)
    if op == "window":
        tokens = sum(_new(case))
        rows = sum(min(c, case["window"] - 1) + n for c, n in zip(_ctx(case), _new(case))) + batch * case["sinks"]
        return {"bytes": rows * (D + 4) + 4 * (2 * batch + 1) + tokens * H * (4 * D + 4), "flops": 4 * D * H * seen}
    tokens = batch * case["tree"]
    rows = batch * (min(case["window"], case["ctx"]) + case["tree"])
    # a sequence's entries are counted once, however many of its tokens list them
    entries = min(listed_entries, batch * case["cap"])
    return {"bytes": entries * ENTRY + 4 * tokens * case["k"] + rows * (D + 4) + 8 * tokens + 4 * batch + tokens * H * (4 * D + 4),
            "flops": 4 * D * H * (seen + listed_entries)}


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


def _rows64(codes, scale):
    return _e4m3(codes) * scale.double()[..., None]


def _readout64(q, keys, seen):
    """softmax(q . k / sqrt(512)) k in 64 bits: q [n, 64, 512], keys [k, 512] of all of them, seen [n, k]."""
    n = q.shape[0]
    logits = (q.reshape(-1, D) @ keys.T).view(n, H, -1) / math.sqrt(D)
    logits = logits + torch.where(seen, 0.0, -math.inf).double()[:, None]
    lse = torch.logsumexp(logits, -1)
    p = torch.exp(logits - torch.where(lse > -math.inf, lse, 0.0)[..., None])
    return (p.view(n * H, -1) @ keys).view(n, H, D), lse


def _exact_slots(s):
    case, out = s["case"], {k: [] for k in ("tok", "pos", "swa", "epos", "slot", "vis", "len")}
    m, cap, ring, cu, cu_e = case["m"], s["cap"], s["ring"], [0], [0]
    for b, (c, n) in enumerate(zip(s["ctx"].tolist(), s["new"].tolist())):
        out["tok"] += [b] * n
        out["pos"] += range(c, c + n)
        out["swa"] += [-1] * max(0, n - ring) + [b * ring + p % ring for p in range(c + max(0, n - ring), c + n)]
        done = [p for p in range(c, c + n) if p % m == m - 1]
        out["epos"] += done
        out["slot"] += [b * cap + p // m if p // m < cap else -1 for p in done]
        out["vis"].append(min((c + n) // m, cap))
        out["len"].append(min(c + n, ring))
        cu.append(cu[-1] + n)
        cu_e.append(cu_e[-1] + len(done))
    def fill(x, n, dtype):
        return torch.tensor(x + [-1] * (n - len(x)), dtype=dtype, device="cuda")
    i32, i64 = torch.int32, torch.int64
    return (_ints(cu), fill(out["tok"], s["n"], i32), fill(out["pos"], s["n"], i64), fill(out["swa"], s["n"], i64),
            _ints(cu_e), fill(out["epos"], s["n_entries"], i64), fill(out["slot"], s["n_entries"], i64),
            _ints(out["vis"]), _ints(out["len"]))


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "slots":
        return _exact_slots(s)
    out, lse = s["out"].double(), s["lse"].double()
    if op == "window":
        w, k, ring, at = case["window"], case["sinks"], s["swa"].shape[1], 0
        for b, (c, n) in enumerate(zip(_ctx(case), _new(case))):
            for lo in range(c, c + n, 256):   # 256 tokens over the positions that any of them sees
                hi = min(lo + 256, c + n)
                first = max(0, lo - w + 1)
                place = torch.arange(first, hi, device="cuda")
                keys, p = _rows64(s["swa"][b, place % ring], s["swa_scale"][b, place % ring]), torch.arange(lo, hi, device="cuda")[:, None]
                seen = (place <= p) & (place > p - w)
                if k:
                    early = torch.arange(k, device="cuda")
                    keys = torch.cat([keys, _rows64(s["sink"][b], s["sink_scale"][b])])
                    seen = torch.cat([seen, (early <= p - w)], 1)
                o, l = _readout64(s["q"][at:at + hi - lo].double(), keys, seen)
                out[at:at + hi - lo], lse[at:at + hi - lo] = o, l
                at += hi - lo
        return out, lse
    t, w, ring = case["tree"], case["window"], s["swa"].shape[1]
    for b in range(case["batch"]):
        c = int(s["ctx"][b])
        place = torch.arange(max(0, c - w), c, device="cuda")
        rows = torch.cat([_rows64(s["swa"][b, place % ring], s["swa_scale"][b, place % ring]), _rows64(s["tree"][b], s["tree_scale"][b])])
        masks = [m % (1 << 64) for m in s["mask"][b].tolist()]
        for i in range(t):
            named = [bool(masks[i] >> j & 1) for j in range(t)]
            seen = torch.cat([place >= c - max(0, w - sum(named)), torch.tensor(named, device="cuda")])
            keys = rows[seen]
            if case["k"]:
                sel = s["idx"][b, i]
                e = s["kv"][b][sel[sel >= 0].long()]
                keys = torch.cat([keys, _nibbles(e[:, :256]) * _e4m3(e[:, 256:]).repeat_interleave(16, dim=-1)])
            if keys.shape[0]:
                o, l = _readout64(s["q"][b, i][None].double(), keys, torch.ones(1, keys.shape[0], dtype=torch.bool, device="cuda"))
                out[b, i], lse[b, i] = o[0], l[0]
            else:
                out[b, i], lse[b, i] = 0.0, -math.inf
    return out, lse
