"""The 8-bit key/value cache's operators as workloads: appending rows, decode
attention (with the attention weight each position received), eviction by that
weight, and reading values back.

Every case is one call as a decode loop makes it.  The plain forms below are
the definitions in elementary torch operations (fp32); exact() states them
again in 64 bits.

The cache: codes [B][Hkv][T_cap][D], 8 bits (int8 or e4m3), and one fp32
scale, a power of two, per block of `block` positions of a head, for keys and
for values; value = code * scale."""
import math

import torch

own = False

DEV = "cuda"
FMT = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
DT = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}
MIN_E = -126


# ---------------------------------------------------------------- the cases

def _append(name, batch, kv_heads, dim, cap, block, fmt, rows, lo, hi, ragged, dtype):
    return {"name": name, "op": "append", "batch": batch, "kv_heads": kv_heads, "dim": dim, "cap": cap, "block": block,
            "fmt": fmt, "rows": rows, "lo": lo, "hi": hi, "ragged": ragged, "dtype": dtype}


def _attend(name, batch, q_heads, kv_heads, dim, cap, block, fmt, rows, lo, hi, ragged, dtype, weights):
    return {"name": name, "op": "attend", "batch": batch, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "cap": cap,
            "block": block, "fmt": fmt, "rows": rows, "lo": lo, "hi": hi, "ragged": ragged, "dtype": dtype,
            "weights": weights}


def _evict(name, batch, kv_heads, dim, cap, block, fmt, lo, hi, budget, sinks, recent):
    return {"name": name, "op": "evict", "batch": batch, "kv_heads": kv_heads, "dim": dim, "cap": cap, "block": block,
            "fmt": fmt, "lo": lo, "hi": hi, "budget": budget, "sinks": sinks, "recent": recent}


def listed():
    """lo .. hi: the sequences' lengths before the call's rows (one at each
    end, the others spread between)."""
    return [
        # one token of one sequence joins the cache of the 16/2/256 attention
        _append("append_token", 1, 2, 256, 4096, 64, "int8", 1, 1003, 1003, False, "bfloat16"),
        # a served batch: each sequence's token and three draft rows, at odd places in their blocks
        _append("append_drafts", 48, 8, 128, 4096, 32, "e4m3", 4, 5, 4001, False, "bfloat16"),
        # two prompts of unequal length, padded to the longer one
        _append("append_prompts", 2, 2, 256, 32768, 64, "int8", 16411, 0, 70, True, "bfloat16"),
        # one token early in a conversation: latency
        _attend("attend_short", 1, 16, 2, 256, 4096, 64, "int8", 1, 517, 517, False, "bfloat16", False),
        # a token and three draft rows verified against 32K positions
        _attend("attend_verify", 1, 16, 2, 256, 40960, 64, "int8", 4, 32771, 32771, False, "bfloat16", False),
        # one token at 128K positions
        _attend("attend_long", 1, 16, 2, 256, 135168, 64, "int8", 1, 131071, 131071, False, "bfloat16", False),
        # a served batch of unequal lengths, one slot of it idle
        _attend("attend_batch", 32, 32, 8, 128, 16384, 32, "e4m3", 1, 1, 16000, True, "float16", False),
        # a decode step that also counts what weight each position received
        _attend("attend_weights", 8, 32, 8, 64, 24576, 32, "int8", 2, 9001, 20011, True, "bfloat16", True),
        # eight long conversations at once: the cache is a gigabyte
        _attend("attend_largest", 8, 16, 2, 256, 131072, 64, "int8", 1, 100003, 131071, False, "bfloat16", False),
        # steady state of a bounded cache: one block over its budget
        _evict("evict_step", 4, 2, 256, 2176, 64, "int8", 2112, 2112, 2048, 4, 256),
        # a prompt's cache cut to an eighth before decoding
        _evict("evict_prompt", 1, 8, 128, 32768, 32, "e4m3", 32749, 32749, 4096, 16, 128),
        # long conversations cut down
        _evict("evict_long", 4, 2, 256, 131072, 64, "int8", 90001, 131072, 16384, 4, 1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    case = _drawn(rng, rng.choice(["append", "attend", "attend", "evict"]))
    del case["name"]
    return case


def _drawn(rng, op):
    dim = rng.choice([64, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    block = rng.choice([16, 32, 64, 128])
    fmt = rng.choice(["int8", "e4m3"])
    batch = _log(rng, 1, 48)
    # positions: at most what the largest case holds, 8 * 2 * 256 * 131072 values
    most = min(131072, (1 << 28) // (batch * kv * dim))
    hi = _log(rng, 2, most) - 1
    lo = rng.randint(0, hi)
    if op == "append":
        rows = min(rng.choice([1, _log(rng, 2, 16), _log(rng, 16, 8192)]), most, (1 << 24) // (batch * kv * dim))
        cap = -(-(hi + rows) // block) * block
        return _append(None, batch, kv, dim, cap, block, fmt, rows, lo, hi, rng.random() < 0.5,
                       rng.choice(["bfloat16", "float16", "float32"]))
    if op == "attend":
        rows = rng.choice([1, 1, 1, rng.randint(2, 8)])
        cap = -(-(hi + rows) // block) * block
        return _attend(None, batch, kv * rng.choice([1, 2, 4, 5, 8]), kv, dim, cap, block, fmt, rows, lo, hi,
                       rng.random() < 0.5, rng.choice(["bfloat16", "bfloat16", "float16"]), rng.random() < 0.3)
    hi = max(hi, 64)
    budget = _log(rng, 16, max(17, hi))
    sinks = rng.randint(0, min(16, budget // 4))
    return _evict(None, batch, kv, dim, -(-hi // block) * block, block, fmt, min(lo, hi), hi, budget, sinks,
                  rng.randint(0, budget // 2))


# ------------------------------------------------------------- their inputs

def _lengths(case, rng):
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    n = [hi, lo] + [rng_int(rng, lo, hi) for _ in range(b)]
    return n[:b]


def rng_int(gen, lo, hi):
    return int(torch.randint(lo, hi + 1, (1,), generator=gen).item())


def _steps(amax, fmt):
    """The exponent of a block's step, from its largest magnitude."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 255 / 256, x - 7, x - 6) if fmt == "int8" else torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e.clamp(min=MIN_E), MIN_E)


def _codes(y, fmt):
    """Values in units of the step, rounded to the codes' values (fp32)."""
    if fmt == "int8":
        return y.round().clamp(-127, 127)
    return y.to(torch.float8_e4m3fn).float()


def _pow2(e):
    """2^e in fp32 from its bits, -126 <= e <= 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _filled(case, gen):
    """A cache full of normal values: a few strong channels in the keys, as
    rotated keys have, and blocks of differing size in the values."""
    b, g, t, d, blk, fmt = (case[k] for k in ("batch", "kv_heads", "cap", "dim", "block", "fmt"))
    out = []
    for which in range(2):
        codes = torch.empty((b, g, t, d), dtype=FMT[fmt], device=DEV)
        scale = torch.empty((b, g, t // blk), device=DEV)
        boost = torch.ones(d, device=DEV)
        if which == 0:
            boost[torch.randint(0, d, (4,), device=DEV, generator=gen)] = 4.0
        for i in range(b):
            x = torch.randn((g, t // blk, blk, d), device=DEV, generator=gen)
            x *= boost if which == 0 else 0.25 + torch.rand((g, t // blk, 1, 1), device=DEV, generator=gen)
            e = _steps(x.abs().amax((2, 3)), fmt)
            codes[i] = _codes(x * _pow2(-e)[:, :, None, None], fmt).to(FMT[fmt]).view(g, t, d)
            scale[i] = _pow2(e)
        out += [codes, scale]
    return out


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    c = case
    s = {"case": dict(c)}
    s["k"], s["k_scale"], s["v"], s["v_scale"] = _filled(c, gen)
    n = _lengths(c, host)
    b = c["batch"]
    if c["op"] == "append":
        dt = DT[c["dtype"]]
        shape = (b, c["rows"], c["kv_heads"], c["dim"])
        s["k_new"] = torch.randn(shape, device=DEV, generator=gen).to(dt)
        s["v_new"] = (torch.randn(shape, device=DEV, generator=gen) * 0.7).to(dt)
        s["pos"] = torch.tensor(n, dtype=torch.int32, device=DEV)
        counts = [c["rows"]] + [rng_int(host, 1, c["rows"]) for _ in range(b)] if c["ragged"] else [c["rows"]] * b
        s["counts"] = torch.tensor(counts[:b], dtype=torch.int32, device=DEV) if c["ragged"] else None
        s["start"] = s["pos"] // c["block"] * c["block"]
        s["lens"] = s["pos"] + torch.tensor(counts[:b], dtype=torch.int32, device=DEV)
    elif c["op"] == "attend":
        if c["ragged"] and b > 2:
            n[2] = -1  # an idle slot of the batch: no row of it sees anything
        s["q"] = (torch.randn((b, c["rows"], c["q_heads"], c["dim"]), device=DEV, generator=gen) * 1.25).to(DT[c["dtype"]])
        s["pos"] = torch.tensor(n, dtype=torch.int32, device=DEV)
        rows = [c["rows"]] + [rng_int(host, 1, c["rows"]) for _ in range(b)]
        s["counts"] = torch.tensor(rows[:b], dtype=torch.int32, device=DEV) if c["ragged"] and c["rows"] > 1 else None
        if c["weights"]:
            s["acc_in"] = torch.rand((b, c["kv_heads"], c["cap"]), device=DEV, generator=gen)
            s["acc"] = torch.zeros((b, c["kv_heads"], c["cap"]), device=DEV)
    else:
        s["lens"] = torch.tensor(n, dtype=torch.int32, device=DEV)
        # accumulated weights: a long tail, as attention leaves them
        s["acc"] = torch.randn((b, c["kv_heads"], c["cap"]), device=DEV, generator=gen).mul_(1.5).exp_()
        cap = -(-c["budget"] // c["block"]) * c["block"]
        shape = (b, c["kv_heads"], cap, c["dim"])
        s["to"] = {"k": torch.zeros(shape, dtype=FMT[c["fmt"]], device=DEV), "v": torch.zeros(shape, dtype=FMT[c["fmt"]], device=DEV),
                   "k_scale": torch.zeros(shape[:2] + (cap // c["block"],), device=DEV),
                   "v_scale": torch.zeros(shape[:2] + (cap // c["block"],), device=DEV),
                   "acc": torch.zeros(shape[:3], device=DEV)}
    if own:
        import quantized_moe_decode_layer_gb300 as moe
        q_heads = c.get("q_heads", c["kv_heads"])

        def handle(t, cap):
            return moe.KV8Cache(cap, batch=b, q_heads=q_heads, kv_heads=c["kv_heads"], head_dim=c["dim"], block=c["block"],
                                fmt=c["fmt"], max_rows=min(c.get("rows", 1), 8), weights=c.get("weights", False),
                                buffers=(t["k"], t["v"], t["k_scale"], t["v_scale"]))
        s["cache"] = handle(s, c["cap"])
        if c["op"] == "evict":
            s["to_cache"] = handle(s["to"], cap)
    return s


# ------------------------------------------------------------ one pass of it

def run(s):
    op = s["case"]["op"]
    if op == "append":
        return _run_append(s)
    return _run_attend(s) if op == "attend" else _run_evict(s)


def _window(c):
    """Positions that an append can change: its rows' blocks."""
    return min(((c["rows"] - 1) // c["block"] + 2) * c["block"], c["cap"])


def _run_append(s):
    c = s["case"]
    if own:
        s["cache"].append(s["k_new"], s["v_new"], s["pos"], counts=s["counts"])
        k, v = s["cache"].read(s["start"], _window(c), lens=s["lens"])
        return {"k": k, "v": v, "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    _plain_append(s["k"], s["k_scale"], s["k_new"], s["pos"], s["lens"], c["fmt"])
    _plain_append(s["v"], s["v_scale"], s["v_new"], s["pos"], s["lens"], c["fmt"])
    return {"k": _plain_read(s["k"], s["k_scale"], s["start"], _window(c), s["lens"]),
            "v": _plain_read(s["v"], s["v_scale"], s["start"], _window(c), s["lens"]),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_append(codes, scale, new, pos, lens, fmt):
    """New rows at positions pos .. lens - 1; a block with earlier rows keeps
    the larger of its step and theirs, its codes rounded again where it grew."""
    b, g, cap, d = codes.shape
    blk = cap // scale.shape[2]
    nb = min((new.shape[1] - 1) // blk + 2, scale.shape[2])
    first = (pos // blk).clamp(max=scale.shape[2] - nb).long()
    at = first[:, None] + torch.arange(nb, device=codes.device)                            # [b, nb] blocks
    t = at[:, :, None] * blk + torch.arange(blk, device=codes.device)                      # [b, nb, blk] positions
    bi = torch.arange(b, device=codes.device)[:, None, None]
    is_new = (t >= pos[:, None, None]) & (t < lens[:, None, None])
    is_old = t < pos[:, None, None]
    row = (t - pos[:, None, None]).clamp(0, new.shape[1] - 1)
    x = new[bi, row].float() * is_new[..., None, None]                                     # [b, nb, blk, g, d]
    e = _steps(x.abs().amax((2, 4)), fmt)                                                  # [b, nb, g]
    was = torch.frexp(scale[bi[:, :, 0], :, at])[1] - 1                                    # [b, nb, g]
    e = torch.where(is_old.any(2)[..., None], torch.maximum(e, was), e)
    e = torch.where(is_new.any(2)[..., None], e, was)                                      # blocks without new rows stay
    down = _pow2((was - e).clamp(min=MIN_E, max=0))[:, :, None, :, None]
    raw = codes.view(torch.int8)
    old = raw[bi, :, t].view(codes.dtype).float()                                          # [b, nb, blk, g, d]
    y = torch.where(is_new[..., None, None], _codes(x * _pow2(-e)[:, :, None, :, None], fmt),
                    torch.where(is_old[..., None, None], _codes(old * down, fmt), old))
    scale[bi[:, :, 0], :, at] = _pow2(e)
    raw[bi, :, t] = y.to(codes.dtype).view(torch.int8)


def _plain_read(codes, scale, start, n, lens):
    """bf16 values [b, n, g, d] of positions start .. start + n - 1; zero from lens on."""
    b, g, cap, d = codes.shape
    blk = cap // scale.shape[2]
    t = start[:, None].long() + torch.arange(n, device=codes.device)
    seen = (t >= 0) & (t < lens[:, None]) & (t < cap)
    t = t.clamp(0, cap - 1)
    bi = torch.arange(b, device=codes.device)[:, None]
    x = codes.view(torch.int8)[bi, :, t].view(codes.dtype).float() * scale[bi, :, t // blk][..., None]
    return (x * seen[:, :, None, None]).to(torch.bfloat16)


def _run_attend(s):
    c = s["case"]
    if own:
        if c["weights"]:
            o, _ = s["cache"].attend(s["q"], s["pos"], counts=s["counts"], acc=s["acc"], acc_in=s["acc_in"], decay=0.875,
                                     out_dtype=s["q"].dtype)
            return {"o": o, "acc": s["acc"]}
        o, _ = s["cache"].attend(s["q"], s["pos"], counts=s["counts"], out_dtype=s["q"].dtype)
        return {"o": o}
    b, m, hq, d = s["q"].shape
    g, cap, blk = c["kv_heads"], c["cap"], c["block"]
    k = (s["k"].float().view(b, g, cap // blk, blk, d) * s["k_scale"][..., None, None]).view(b, g, cap, d)
    q = s["q"].float().view(b, m, g, hq // g, d).permute(0, 2, 1, 3, 4).reshape(b, g, m * (hq // g), d)
    sc = q @ k.transpose(2, 3) * d ** -0.5                                                 # [b, g, m * hq / g, cap]
    del k
    row = torch.arange(m, device=DEV)
    seen = s["pos"][:, None] + row + 1                                                     # [b, m]
    seen = torch.where(s["pos"][:, None] >= 0, seen, 0)
    if s["counts"] is not None:
        seen = torch.where(row < s["counts"][:, None], seen, 0)
    hide = torch.arange(cap, device=DEV) >= seen[:, :, None]                               # [b, m, cap]
    hide = hide[:, None, :, None, :].expand(b, g, m, hq // g, cap).reshape(sc.shape)
    sc.masked_fill_(hide, -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(top == -math.inf, 0.0, top))
    del sc, hide
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    v = (s["v"].float().view(b, g, cap // blk, blk, d) * s["v_scale"][..., None, None]).view(b, g, cap, d)
    o = (p @ v).view(b, g, m, hq // g, d).permute(0, 2, 1, 3, 4).reshape(b, m, hq, d).to(s["q"].dtype)
    if not c["weights"]:
        return {"o": o}
    t = torch.arange(cap, device=DEV)
    was = torch.where(t < s["pos"][:, None], 0.875, 0.0)[:, None] * s["acc_in"]
    within = t < seen.amax(1)[:, None]
    s["acc"].copy_(torch.where(within[:, None], was + p.sum(2), s["acc"]))
    return {"o": o, "acc": s["acc"]}


def _run_evict(s):
    c = s["case"]
    if own:
        idx, lens = s["cache"].evict_into(s["to_cache"], s["lens"], s["acc"], c["budget"], sinks=c["sinks"],
                                          recent=c["recent"], dst_acc=s["to"]["acc"])
        k, v = s["to_cache"].read(None, c["budget"], lens=lens)
        return {"idx": idx, "lens": lens, "k": k, "v": v, "acc": s["to"]["acc"]}
    b, g, cap, d = s["k"].shape
    blk, budget, fmt, to = c["block"], c["budget"], c["fmt"], s["to"]
    n = s["lens"].long()[:, None, None]
    t = torch.arange(cap, device=DEV).expand(b, g, cap)
    rank = torch.where((t < c["sinks"]) | (t >= n - c["recent"]), math.inf, s["acc"])
    rank = torch.where(t < n, rank, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True)[1][..., :budget]
    if order.shape[-1] < budget:
        order = torch.nn.functional.pad(order, (0, budget - order.shape[-1]), value=cap)
    kept = torch.sort(torch.where(order < n, order, cap), dim=-1)[0]                       # [b, g, budget]
    there = kept < n
    at = kept.clamp(max=cap - 1)
    pad = to["k"].shape[2] - budget
    lens = s["lens"].clamp(0, budget)
    for codes, scale, dst, dst_scale in ((s["k"], s["k_scale"], to["k"], to["k_scale"]), (s["v"], s["v_scale"], to["v"], to["v_scale"])):
        x = torch.gather(codes.view(torch.int8), 2, at[..., None].expand(b, g, budget, d)).view(codes.dtype).float()
        x = x * torch.gather(scale, 2, at // blk)[..., None] * there[..., None]
        x = torch.nn.functional.pad(x, (0, 0, 0, pad)).view(b, g, -1, blk, d)
        e = _steps(x.abs().amax((3, 4)), fmt)
        used = torch.arange(e.shape[2], device=DEV) * blk < lens[:, None, None]
        dst_scale.copy_(torch.where(used, _pow2(e), dst_scale))
        y = _codes(x * _pow2(-e)[..., None, None], fmt).view(dst.shape)
        live = (torch.arange(dst.shape[2], device=DEV) < lens[:, None, None])[..., None]
        dst.copy_(torch.where(live, y, dst.float()).to(dst.dtype))
    live = torch.arange(to["acc"].shape[2], device=DEV) < lens[:, None, None]
    acc = torch.nn.functional.pad(torch.gather(s["acc"], 2, at), (0, pad))
    to["acc"].copy_(torch.where(live, acc, to["acc"]))
    start = torch.zeros_like(lens)
    return {"idx": torch.where(there, kept, -1).int(), "lens": lens,
            "k": _plain_read(to["k"], to["k_scale"], start, budget, lens),
            "v": _plain_read(to["v"], to["v_scale"], start, budget, lens), "acc": to["acc"]}


# ----------------------------------------------------------------- its work

def _total(case):
    """Positions that the sequences of a case hold, about (the lengths between
    the two ends are drawn evenly)."""
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    return hi + (lo if b > 1 else 0) + max(0, b - 2) * (lo + hi) / 2


def work(case):
    c = case
    b, g, d, blk = c["batch"], c["kv_heads"], c["dim"], c["block"]
    if c["op"] == "append":
        rows = c["rows"] * (1 + (b - 1) * (0.5 if c["ragged"] else 1.0))
        size = 4 if c["dtype"] == "float32" else 2
        # new rows in, codes and scales out, the values read back
        return {"bytes": 2 * g * (rows * d * (size + 1) + rows / blk * 4 + b * _window(c) * d * 2),
                "flops": 2 * g * rows * d * 3}
    if c["op"] == "attend":
        n = _total(c) + b * c["rows"]
        io = 2 * b * c["rows"] * c["q_heads"] * d * 2
        return {"bytes": n * g * (2 * d + 8 / blk + (8 if c["weights"] else 0)) + io,
                "flops": 4 * n * c["rows"] * c["q_heads"] * d}
    kept = min(c["budget"], c["hi"]) * b
    # the weights, the kept codes in and out, indices and weights out, the values read back
    return {"bytes": g * (4 * _total(c) + kept * (2 * 2 * d + 8 + 2 * 2 * d)), "flops": g * (_total(c) * 4 + kept * 4 * d)}


# ------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "append":
        return _exact_append(s, c)
    return _exact_attend(s, c) if c["op"] == "attend" else _exact_evict(s, c)


def _exact_step(largest, fmt):
    """The smallest power of two (from 2^-126 up) in whose units `largest`
    rounds to a code: 127.5 or less for int8, 448 or less for e4m3."""
    limit = 127.5 if fmt == "int8" else 448.0
    ok = largest > 0
    guess = torch.floor(torch.log2(torch.where(ok, largest, 1.0) / limit)) - 1
    for _ in range(3):
        guess = torch.where(torch.where(ok, largest, 0.0) > limit * _two(guess), guess + 1, guess)
    return torch.where(ok, guess, MIN_E).clamp(min=MIN_E)


def _two(e):
    """2^e in 64 bits, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _log_of(scale):
    """The exponents of powers of two."""
    return torch.round(torch.log2(scale.double()))


def _exact_round(y, fmt):
    """64-bit values, in units of the step, to the nearest code (ties to even)."""
    if fmt == "int8":
        low = torch.floor(y)
        part = y - low
        up = (part > 0.5) | ((part == 0.5) & (low % 2 != 0))
        return torch.clamp(low + up, -127, 127)
    # e4m3: three fraction bits, exponents from -6 up
    e = torch.floor(torch.log2(torch.where(y == 0, 1.0, y.abs()))).clamp(min=-6)
    ulp = _two(e - 3)
    z = y / ulp
    low = torch.floor(z)
    part = z - low
    up = (part > 0.5) | ((part == 0.5) & (low % 2 != 0))
    return (low + up) * ulp


def _exact_append(s, c):
    blk, fmt, n = c["block"], c["fmt"], _window(c)
    out = {"k": [], "v": [], "k_scale": s["k_scale"].double(), "v_scale": s["v_scale"].double()}
    pos, lens, start = s["pos"].tolist(), s["lens"].tolist(), s["start"].tolist()
    for key in ("k", "v"):
        scale = out[key + "_scale"]
        for b in range(c["batch"]):
            vals = torch.zeros((n, c["kv_heads"], c["dim"]), dtype=torch.float64, device=DEV)
            for t0 in range(start[b], lens[b], blk):
                t1 = min(t0 + blk, lens[b])
                first = max(t0, pos[b])
                new = s[key + "_new"][b, first - pos[b]:t1 - pos[b]].double()             # [rows, g, d]
                e = _exact_step(new.abs().amax((0, 2)), fmt)
                if first > t0:
                    was = _log_of(scale[b, :, t0 // blk])
                    e = torch.maximum(e, was)
                    old = s[key][b, :, t0:first].double() * _two(was)[:, None, None]
                    old = _exact_round(old * _two(-e)[:, None, None], fmt) * _two(e)[:, None, None]
                    vals[t0 - start[b]:first - start[b]] = old.transpose(0, 1)
                scale[b, :, t0 // blk] = _two(e)
                new = _exact_round(new * _two(-e)[None, :, None], fmt) * _two(e)[None, :, None]
                vals[first - start[b]:t1 - start[b]] = new
            out[key].append(vals)
        out[key] = torch.stack(out[key])
    return out


def _exact_attend(s, c):
    b, m, hq, d = s["q"].shape
    g, blk = c["kv_heads"], c["block"]
    o = torch.zeros((b, m, hq, d), dtype=torch.float64, device=DEV)
    acc = s["acc"].double() if c["weights"] else None
    pos = s["pos"].tolist()
    rows = s["counts"].tolist() if s["counts"] is not None else [m] * b
    for i in range(b):
        end = pos[i] + rows[i] if pos[i] >= 0 else 0
        if c["weights"] and end:
            acc[i, :, :end] = 0.0
            acc[i, :, :pos[i]] = 0.875 * s["acc_in"][i, :, :pos[i]].double()
        for h in range(g):
            if not end:
                continue
            k = s["k"][i, h, :end].double() * s["k_scale"][i, h].double().repeat_interleave(blk)[:end, None]
            v = s["v"][i, h, :end].double() * s["v_scale"][i, h].double().repeat_interleave(blk)[:end, None]
            for r in range(rows[i]):
                see = pos[i] + r + 1
                q = s["q"][i, r, h * (hq // g):(h + 1) * (hq // g)].double()
                z = torch.matmul(k[:see], q.t()) / math.sqrt(d)                            # [see, heads]
                w = torch.exp(z - z.max(0, keepdim=True)[0])
                w = w / w.sum(0, keepdim=True)
                o[i, r, h * (hq // g):(h + 1) * (hq // g)] = torch.matmul(w.t(), v[:see])
                if c["weights"]:
                    acc[i, h, :see] += w.sum(1)
    return {"o": o, "acc": acc} if c["weights"] else {"o": o}


def _exact_evict(s, c):
    b, g, cap, d = s["k"].shape
    blk, budget, fmt = c["block"], c["budget"], c["fmt"]
    idx = torch.full((b, g, budget), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(b, dtype=torch.int32, device=DEV)
    acc = s["to"]["acc"].double()
    out = {key: torch.zeros((b, budget, g, d), dtype=torch.float64, device=DEV) for key in ("k", "v")}
    for i, n in enumerate(s["lens"].tolist()):
        lens[i] = min(n, budget)
        for h in range(g):
            if n <= budget:
                keep = torch.arange(n, device=DEV)
            else:
                forced = torch.cat([torch.arange(c["sinks"], device=DEV), torch.arange(n - c["recent"], n, device=DEV)]).unique()
                free = torch.ones(n, dtype=torch.bool, device=DEV)
                free[forced] = False
                free = free.nonzero()[:, 0]
                # largest first, then lowest index
                by = torch.sort(-s["acc"][i, h, free].double(), stable=True)[1][:budget - forced.numel()]
                keep = torch.cat([forced, free[by]]).sort()[0]
            m = keep.numel()
            idx[i, h, :m] = keep.int()
            acc[i, h, :m] = s["acc"][i, h, keep].double()
            for key in ("k", "v"):
                x = s[key].view(torch.int8)[i, h, keep].view(s[key].dtype).double()
                x = x * s[key + "_scale"][i, h, keep // blk].double()[:, None]
                full = torch.zeros((-(-m // blk) * blk, d), dtype=torch.float64, device=DEV)
                full[:m] = x
                full = full.view(-1, blk, d)
                e = _two(_exact_step(full.abs().amax((1, 2)), fmt))[:, None, None]
                out[key][i, :m, h] = (_exact_round(full / e, fmt) * e).view(-1, d)[:m]
    return {"idx": idx, "lens": lens, "k": out["k"], "v": out["v"], "acc": acc}
