"""The 16-bit key/value cache's operators as workloads: appending rows of a
batch of sequences (into a ring, where the attention has a window), attention
with a sliding window and a few first positions that stay visible (prompts, and
single tokens and drafts over the cache), and the decode attention of a batch
whose sequences share a long prefix.

Every case is one call as a serving loop makes it.  The plain forms below are
the definitions in elementary torch operations (fp32); exact() states them
again in 64 bits.

The cache: [B][Hkv][T_cap][D] keys and values, bf16 or fp16.  Position t of a
sequence lies in slot t, and from T_cap on, where the attention has a window of
W positions and S first ones, in slot S + (t - S) mod (T_cap - S).  A row at
position p sees the positions t <= p with t > p - W or t < S."""
import math

import torch

own = False

DEV = "cuda"
DT = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}


# ---------------------------------------------------------------- the cases

def _append(name, batch, kv_heads, dim, cap, window, sinks, rows, lo, hi, ragged, dtype, given):
    return {"name": name, "op": "append", "batch": batch, "kv_heads": kv_heads, "dim": dim, "cap": cap, "window": window,
            "sinks": sinks, "rows": rows, "lo": lo, "hi": hi, "ragged": ragged, "dtype": dtype, "given": given}


def _prompt(name, batch, q_heads, kv_heads, dim, rows, start, window, sinks, ragged, dtype):
    return {"name": name, "op": "prompt", "batch": batch, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "rows": rows,
            "start": start, "window": window, "sinks": sinks, "ragged": ragged, "dtype": dtype}


def _token(name, batch, q_heads, kv_heads, dim, cap, window, sinks, rows, lo, hi, ragged, dtype):
    return {"name": name, "op": "token", "batch": batch, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "cap": cap,
            "window": window, "sinks": sinks, "rows": rows, "lo": lo, "hi": hi, "ragged": ragged, "dtype": dtype}


def _prefix(name, batch, q_heads, kv_heads, dim, prefix, cap, rows, lo, hi, ragged, dtype):
    return {"name": name, "op": "prefix", "batch": batch, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
            "prefix": prefix, "cap": cap, "rows": rows, "lo": lo, "hi": hi, "ragged": ragged, "dtype": dtype}


def listed():
    """lo .. hi: the sequences' lengths before the call's rows (one at each
    end, the others spread between)."""
    return [
        # a served batch: each sequence's next token joins its ring
        _append("append_token", 48, 8, 128, 4224, 4096, 4, 1, 5, 30011, False, "float16", "float16"),
        # two prompts of unequal length, longer than the window, as a projection in fp32 gives them
        _append("append_prompts", 2, 2, 256, 4224, 4096, 16, 16411, 0, 70, True, "bfloat16", "float32"),
        # three short questions, padded to the longest: latency
        _prompt("prompt_short", 3, 16, 2, 256, 77, 0, 4096, 4, True, "bfloat16"),
        # a prompt eight times as long as the window
        _prompt("prompt_window", 1, 32, 8, 128, 8195, 0, 1024, 4, False, "bfloat16"),
        # a prompt's next piece, behind what came before
        _prompt("prompt_piece", 2, 32, 8, 64, 2048, 6001, 2048, 16, False, "float16"),
        # a long prompt of the 16/2/256 attention
        _prompt("prompt_long", 1, 16, 2, 256, 32768, 0, 4096, 4, False, "bfloat16"),
        # one token early in a conversation: latency
        _token("token_short", 1, 16, 2, 256, 4224, 4096, 4, 1, 517, 517, False, "bfloat16"),
        # a token and three draft rows of eight conversations that have outgrown the ring
        _token("token_drafts", 8, 16, 2, 256, 8224, 8192, 4, 4, 9001, 100003, True, "bfloat16"),
        # a served batch of unequal lengths, one slot of it idle
        _token("token_batch", 48, 32, 8, 128, 4224, 4096, 4, 1, 1, 30011, True, "float16"),
        # four questions about one document
        _prefix("prefix_few", 4, 16, 2, 256, 8197, 512, 1, 0, 201, False, "bfloat16"),
        # a served batch behind one long set of instructions
        _prefix("prefix_batch", 64, 32, 8, 128, 16411, 1024, 1, 3, 1000, True, "float16"),
        # many answers, each with three draft rows, to one long document
        _prefix("prefix_largest", 128, 16, 2, 256, 131071, 2048, 4, 100, 2001, True, "bfloat16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    case = _drawn(rng, rng.choice(["append", "prompt", "prompt", "token", "token", "prefix", "prefix"]))
    del case["name"]
    return case


def _drawn(rng, op):
    dim = rng.choice([64, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 4, 5, 8])
    dtype = rng.choice(["bfloat16", "bfloat16", "float16"])
    batch = _log(rng, 1, 64)
    window, sinks = _log(rng, 16, 8192), rng.choice([0, 1, 4, rng.randint(5, 64)])
    ragged = rng.random() < 0.5
    if op == "append":
        # at most 2^26 values of keys in the call, 2^28 in the cache
        rows = min(rng.choice([1, _log(rng, 2, 16), _log(rng, 16, 16384)]), (1 << 26) // (batch * kv * dim))
        cap = min(sinks + window + rng.randint(7, 300), (1 << 28) // (batch * kv * dim))
        window = min(window, cap - sinks - 7)
        hi = _log(rng, 1, 100000) - 1
        return _append(None, batch, kv, dim, cap, window, sinks, rows, rng.randint(0, hi), hi, ragged, dtype,
                       rng.choice([dtype, dtype, "float32"]))
    if op == "prompt":
        # at most 2^30 scores, as the longest listed one has within its window
        batch = min(batch, 8)
        rows, start = _log(rng, 1, 16384), rng.choice([0, 0, _log(rng, 1, 16384)])
        rows = max(1, min(rows, (1 << 30) // (batch * heads * min(window + sinks, start + rows))))
        return _prompt(None, batch, heads, kv, dim, rows, start, window, sinks, ragged, dtype)
    if op == "token":
        rows = rng.choice([1, 1, 1, rng.randint(2, 8)])
        cap = min(sinks + window + rng.randint(7, 300), (1 << 28) // (batch * kv * dim))
        window = min(window, cap - sinks - 7)
        hi = _log(rng, 1, 100000) - 1
        return _token(None, batch, heads, kv, dim, cap, window, sinks, rows, rng.randint(0, hi), hi, ragged, dtype)
    rows = rng.choice([1, 1, 1, rng.randint(2, 8)])
    prefix = min(_log(rng, 1, 131071), (1 << 30) // (batch * rows * heads))
    hi = _log(rng, 1, 2000) - 1
    return _prefix(None, batch, heads, kv, dim, prefix, hi + rows + rng.randint(0, 200), rows, rng.randint(0, hi), hi, ragged,
                   dtype)


# ------------------------------------------------------------- their inputs

def _int(gen, lo, hi):
    return int(torch.randint(lo, hi + 1, (1,), generator=gen).item())


def _lengths(case, gen):
    n = [case["hi"], case["lo"]] + [_int(gen, case["lo"], case["hi"]) for _ in range(case["batch"])]
    return n[:case["batch"]]


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _keys(shape, gen, dtype):
    """Normal values with a few strong channels, as rotated keys have."""
    x = torch.randn(shape, device=DEV, generator=gen)
    x[..., torch.randint(0, shape[-1], (4,), device=DEV, generator=gen)] *= 4.0
    return x.to(dtype)


def _values(shape, gen, dtype):
    return (torch.randn(shape, device=DEV, generator=gen) * 0.7).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    c = case
    b, g, d, rows, dt = c["batch"], c["kv_heads"], c["dim"], c["rows"], DT[c["dtype"]]
    s = {"case": dict(c)}
    counts = [rows] + [_int(host, 1, rows) for _ in range(b)] if c["ragged"] else [rows] * b
    s["counts"] = _ints(counts[:b]) if c["ragged"] and rows > 1 else None
    if c["op"] == "prompt":
        total = c["start"] + rows
        s["q"] = (torch.randn((b, rows, c["q_heads"], d), device=DEV, generator=gen) * 1.25).to(dt)
        kv = torch.empty((b, total, 2 * g, d), dtype=dt, device=DEV)     # one projection's output
        s["k"], s["v"] = kv[:, :, :g], kv[:, :, g:]
        s["k"].copy_(_keys((b, total, g, d), gen, dt))
        s["v"].copy_(_values((b, total, g, d), gen, dt))
        s["pos"] = _ints([c["start"]] * b)
        return s
    s["k"] = _keys((b, g, c["cap"], d), gen, dt)
    s["v"] = _values((b, g, c["cap"], d), gen, dt)
    n = _lengths(c, host)
    if c["op"] != "append" and c["ragged"] and b > 2:
        n[2] = -1  # an idle slot of the batch: no row of it sees anything
    s["pos"] = _ints(n)
    if c["op"] == "append":
        shape = (b, rows, g, d)
        s["k_new"], s["v_new"] = _keys(shape, gen, DT[c["given"]]), _values(shape, gen, DT[c["given"]])
    else:
        s["q"] = (torch.randn((b, rows, c["q_heads"], d), device=DEV, generator=gen) * 1.25).to(dt)
    if c["op"] == "prefix":
        s["pk"], s["pv"] = _keys((c["prefix"], g, d), gen, dt), _values((c["prefix"], g, d), gen, dt)
    if own:
        import quantized_moe_decode_layer_gb300 as moe
        s["cache"] = moe.KVCache(c["cap"], batch=b, q_heads=c.get("q_heads", g), kv_heads=g, head_dim=d, dtype=dt,
                                 window=c.get("window"), sinks=c.get("sinks", 0), max_rows=min(rows, 8),
                                 max_prefix=c.get("prefix", 0), buffers=(s["k"], s["v"]))
    return s


# ------------------------------------------------------------ one pass of it

def run(s):
    c = s["case"]
    if c["op"] == "append":
        if own:
            s["cache"].append(s["k_new"], s["v_new"], s["pos"], counts=s["counts"])
        else:
            _plain_append(s)
        return {"k": s["k"], "v": s["v"]}
    if not own:
        return {"o": {"prompt": _plain_prompt, "token": _plain_token, "prefix": _plain_prefix}[c["op"]](s)}
    if c["op"] == "prompt":
        import quantized_moe_decode_layer_gb300 as moe
        o, _ = moe.window_attention(s["q"], s["k"], s["v"], c["window"], sinks=c["sinks"], pos=s["pos"], counts=s["counts"])
    elif c["op"] == "token":
        o, _ = s["cache"].attend(s["q"], s["pos"], counts=s["counts"])
    else:
        o, _ = s["cache"].attend(s["q"], s["pos"], counts=s["counts"], prefix=(s["pk"], s["pv"]))
    return {"o": o}


def _ends(s):
    """One past the last position of each sequence's rows (idle ones: none)."""
    rows = s["case"]["rows"] if s["counts"] is None else s["counts"]
    return torch.where(s["pos"] < 0, s["pos"], s["pos"] + rows).long()


def _slots(t, sinks, cap):
    return torch.where(t < sinks, t, sinks + (t - sinks) % (cap - sinks))


def _plain_append(s):
    """The last T_cap - S rows at their slots, and rows at the first S
    positions; slots that no row falls on are written as they were."""
    c = s["case"]
    sinks, cap = c["sinks"], c["cap"]
    pos, end = s["pos"].long()[:, None], _ends(s)[:, None]
    bi = torch.arange(c["batch"], device=DEV)[:, None]
    ring = end - 1 - torch.arange(min(c["rows"], cap - sinks), device=DEV)
    first = torch.arange(sinks, device=DEV).expand(c["batch"], sinks)
    for_ring = (ring >= pos) & (ring >= sinks)
    for_first = (first >= pos) & (first < end)
    at_ring = sinks + (ring - sinks) % (cap - sinks)
    _plain_write(s["k"], s["k_new"], bi, ring - pos, at_ring, for_ring)
    _plain_write(s["v"], s["v_new"], bi, ring - pos, at_ring, for_ring)
    if sinks:
        _plain_write(s["k"], s["k_new"], bi, first - pos, first, for_first)
        _plain_write(s["v"], s["v_new"], bi, first - pos, first, for_first)


def _plain_write(cache, new, bi, row, slot, within):
    x = new[bi, row.clamp(0, new.shape[1] - 1)].to(cache.dtype)
    cache[bi, :, slot] = torch.where(within[:, :, None, None], x, cache[bi, :, slot])


def _softmax(sc):
    """Over the last axis; rows that are all -inf get zeros."""
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(top == -math.inf, 0.0, top))
    return p / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _plain_prompt(s):
    """Rows in blocks as long as the window; a block sees the two windows of
    keys that end with it, and the first positions."""
    c = s["case"]
    b, m, hq, d = s["q"].shape
    g, w, sinks, total = c["kv_heads"], c["window"], c["sinks"], s["k"].shape[1]
    blk = min(w, m)
    nb, band = -(-m // blk), min(blk + w - 1, total)
    nf = min(sinks, total)
    pos = s["pos"].long()
    row = torch.arange(nb * blk, device=DEV).view(nb, blk)
    p = pos[:, None, None] + row                                                       # [b, nb, blk]
    last = (pos[:, None] + row[:, -1]).clamp(max=total - 1)                            # [b, nb]
    t = last[:, :, None] - (band - 1) + torch.arange(band, device=DEV)                 # [b, nb, band]
    live = row < (m if s["counts"] is None else s["counts"][:, None, None])            # [b or 1, nb, blk]
    near = (t[:, :, None] >= 0) & (t[:, :, None] <= p[..., None]) & (t[:, :, None] > p[..., None] - w) & live[..., None]
    f = torch.arange(nf, device=DEV)
    far = (f <= p[..., None] - w) & live[..., None]                                    # [b, nb, blk, nf]: not in the window
    bi = torch.arange(b, device=DEV)[:, None, None]
    kb, vb = (s[x][bi, t.clamp(min=0)].float() for x in ("k", "v"))                    # [b, nb, band, g, d]
    kb, vb = kb.permute(0, 3, 1, 4, 2), vb.permute(0, 3, 1, 2, 4)
    kf, vf = (s[x][:, :nf].float().transpose(1, 2)[:, :, None] for x in ("k", "v"))    # [b, g, 1, nf, d]
    q = torch.nn.functional.pad(s["q"].float(), (0, 0, 0, 0, 0, nb * blk - m))
    q = q.view(b, nb, blk, g, hq // g, d).permute(0, 3, 1, 4, 2, 5).reshape(b, g, nb, -1, d)
    sc = torch.cat([q @ kb, q @ kf.transpose(3, 4)], -1).view(b, g, nb, hq // g, blk, band + nf)
    sc *= d ** -0.5
    sc.masked_fill_(~torch.cat([near, far], -1)[:, None, :, None], -math.inf)
    pr = _softmax(sc).view(b, g, nb, -1, band + nf)
    del sc
    o = pr[..., :band] @ vb + pr[..., band:] @ vf
    o = o.view(b, g, nb, hq // g, blk, d).permute(0, 2, 4, 1, 3, 5).reshape(b, nb * blk, hq, d)
    return o[:, :m].to(s["q"].dtype)


def _grouped(q, g):
    """[b, m, hq, d] as [b, g, m * hq / g, d] in fp32."""
    b, m, hq, d = q.shape
    return q.float().view(b, m, g, hq // g, d).permute(0, 2, 1, 3, 4).reshape(b, g, -1, d)


def _ungrouped(o, like):
    b, m, hq, d = like.shape
    g = o.shape[1]
    return o.view(b, g, m, hq // g, d).permute(0, 2, 1, 3, 4).reshape(b, m, hq, d).to(like.dtype)


def _plain_token(s):
    c = s["case"]
    b, m, hq, d = s["q"].shape
    g, w, sinks, cap = c["kv_heads"], c["window"], c["sinks"], c["cap"]
    pos, end = s["pos"].long(), _ends(s)
    n = min(w + m - 1, cap - sinks)
    first = (pos[:, None] - w + 1).clamp(min=sinks) + torch.arange(n, device=DEV)
    t = torch.cat([torch.arange(sinks, device=DEV).expand(b, sinks), first], 1)        # [b, sinks + n]
    p = pos[:, None] + torch.arange(m, device=DEV)                                     # [b, m]
    sees = (t[:, None] <= p[..., None]) & ((t[:, None] > p[..., None] - w) | (t[:, None] < sinks))
    sees &= ((p < end[:, None]) & (pos[:, None] >= 0))[..., None]                      # [b, m, n]
    bi = torch.arange(b, device=DEV)[:, None]
    k, v = (s[x][bi, :, _slots(t, sinks, cap)].float().transpose(1, 2) for x in ("k", "v"))
    sc = _grouped(s["q"], g) @ k.transpose(2, 3) * d ** -0.5                           # [b, g, m * hq / g, n]
    sc.view(b, g, m, hq // g, -1).masked_fill_(~sees[:, None, :, None], -math.inf)
    return _ungrouped(_softmax(sc) @ v, s["q"])


def _plain_prefix(s):
    c = s["case"]
    b, m, hq, d = s["q"].shape
    g, n = c["kv_heads"], c["prefix"]
    q = _grouped(s["q"], g) * d ** -0.5
    pk, pv = s["pk"].float().transpose(0, 1), s["pv"].float().transpose(0, 1)          # [g, n, d]
    shared = (q.transpose(0, 1).reshape(g, -1, d) @ pk.transpose(1, 2)).view(g, b, -1, n).transpose(0, 1)
    alone = q @ s["k"].float().transpose(2, 3)
    p, end = s["pos"].long()[:, None] + torch.arange(m, device=DEV), _ends(s)[:, None]
    live = (p < end) & (s["pos"][:, None] >= 0)                                        # [b, m]
    sees = (torch.arange(c["cap"], device=DEV) <= p[..., None]) & live[..., None]
    alone.view(b, g, m, hq // g, -1).masked_fill_(~sees[:, None, :, None], -math.inf)
    pr = _softmax(torch.cat([shared, alone], -1))
    del shared, alone
    o = (pr[..., :n].transpose(0, 1).reshape(g, -1, n) @ pv).view(g, b, -1, d).transpose(0, 1)
    o = _ungrouped(o + pr[..., n:] @ s["v"].float(), s["q"])
    return o * live[:, :, None, None]


# ------------------------------------------------------------------ its work

def _seen(case):
    """About how many (row, position) pairs the case's rows see, and how many
    positions any row does, over the batch."""
    c, pairs, keys = case, 0, 0
    m, w, sinks = c["rows"], c.get("window") or 1 << 40, c.get("sinks", 0)
    if c["op"] == "prompt":
        a, z = c["start"], c["start"] + m
        full = max(0, min(z, w) - a)                       # rows that see all positions up to theirs
        pairs = full * (a + (full + 1) / 2) + (m - full) * min(w + sinks, z)
        keys = min(z, m + w - 1 + sinks)
        return c["batch"] * pairs, c["batch"] * keys
    for i in range(c["batch"]):
        n = c["hi"] if i == 0 else c["lo"] if i == 1 else (c["hi"] + c["lo"]) // 2
        if c["ragged"] and c["batch"] > 2 and i == 2:
            continue
        seen = min(n + 1, w + sinks)
        pairs += m * seen
        keys += min(n + m, w + m - 1 + sinks)
    return pairs, keys


def work(case):
    c = case
    size = {"bfloat16": 2, "float16": 2, "float32": 4}
    g, d, m, b, e = c["kv_heads"], c["dim"], c["rows"], c["batch"], 2
    if c["op"] == "append":
        kept = min(m, c["cap"]) * b * g * d * 2
        return {"bytes": kept * (size[c["given"]] + e), "flops": 0}
    pairs, keys = _seen(c)
    rows = b * m * c["q_heads"] * d
    if c["op"] == "prefix":
        pairs += b * m * c["prefix"]
        keys += c["prefix"]
    return {"bytes": keys * g * d * 2 * e + rows * 2 * e, "flops": 4 * pairs * c["q_heads"] * d}


# ------------------------------------------------------ the same in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c = case
    pos = s["pos"].tolist()
    counts = [c["rows"]] * c["batch"] if s["counts"] is None else s["counts"].tolist()
    if c["op"] == "append":
        k, v = s["k"].double(), s["v"].double()
        for i in range(c["batch"]):
            for lo, hi in ((0, c["sinks"]), (max(c["sinks"], pos[i] + counts[i] - (c["cap"] - c["sinks"])), 1 << 62)):
                t = torch.arange(max(lo, pos[i]), max(lo, pos[i], min(hi, pos[i] + counts[i])), device=DEV)
                at = _at(t, c)
                for to, new in ((k, s["k_new"]), (v, s["v_new"])):
                    to[i][:, at] = new[i, t - pos[i]].to(DT[c["dtype"]]).double().transpose(0, 1)
        return {"k": k, "v": v}
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    w, sinks = c.get("window") or 1 << 40, c.get("sinks", 0)
    step = max(1, min(1024, (1 << 27) // (c["q_heads"] * (c.get("prefix", 0) + 8192))))
    for i in range(c["batch"]):
        if pos[i] < 0:
            continue
        for r0 in range(0, counts[i], step):
            r1 = min(counts[i], r0 + step)
            p = torch.arange(pos[i] + r0, pos[i] + r1, device=DEV)
            lo, hi = max(0, pos[i] + r0 - w + 1), pos[i] + r1
            t = torch.cat([torch.arange(min(sinks, lo), device=DEV), torch.arange(lo, hi, device=DEV)])
            hide = (t > p[:, None]) | ((t <= p[:, None] - w) & (t >= sinks))             # [rows, keys]
            if c["op"] == "prompt":
                k, v = s["k"][i, t].double(), s["v"][i, t].double()                      # [keys, g, d]
            else:
                k, v = (s[x][i][:, _at(t, c)].double().transpose(0, 1) for x in ("k", "v"))
            if c["op"] == "prefix":
                k, v = torch.cat([s["pk"].double(), k]), torch.cat([s["pv"].double(), v])
                hide = torch.cat([torch.zeros((r1 - r0, c["prefix"]), dtype=torch.bool, device=DEV), hide], 1)
            for h in range(c["q_heads"]):
                a = h // (c["q_heads"] // c["kv_heads"])
                z = s["q"][i, r0:r1, h].double() @ k[:, a].t() / math.sqrt(c["dim"])
                z[hide] = -math.inf
                z = torch.exp(z - z.max(1, keepdim=True).values)
                o[i, r0:r1, h] = z @ v[:, a] / z.sum(1, keepdim=True)
    return {"o": o}


def _at(t, c):
    """The slots of positions t."""
    s = c.get("sinks", 0)
    return torch.where(t < s, t, (t - s) % (c["cap"] - s) + s)
