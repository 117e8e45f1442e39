"""GPU parity of the 8-bit key/value cache (moe_kv8_*) with its definition in
64 bits (kv8_ref.py).

Steps and codes are defined exactly, so appending, reading back and eviction
must agree bit for bit.

Attention's tolerance, from its arithmetic.  A score is an fp32 sum of D exact
products (a tensor core may truncate: a step of 2^-23 each), scaled by two
more factors: |e| <= (D + 4) 2^-23 smax with smax the largest scale * sum |q_d
k_d|; the exponential adds a few 2^-23 of itself and of |s| <= smax.  A relative
error e of every weight moves the weighted mean by at most 2 e sum_t w_t |v_t|
(oabs).  The sums over positions add at most one 2^-23 per addition in a row;
a chunk has at most 1024 additions in a row, and a row's chunks are joined one by one:
(1024 + chunks) 2^-23 oabs, for numerator and denominator.  A weight may
be split into two halves of 11 bits: 2^-22.  An output in bf16 (fp16) is off
by 2^-8 (2^-11) of itself more; fp16's smallest step is 2^-24."""
import numpy as np
import pytest
import torch

import kv8_ref
import quantized_moe_decode_layer_gb300 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
E23 = 2.0 ** -23
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def rows(gen, *shape, dtype=torch.bfloat16, size=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * size).to(dtype)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def same_state(cache, ref, lens):
    """Codes and steps of every sequence's first lens[b] positions."""
    for which, (c, s) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
        got, step = c.cpu().float().double(), s.cpu().double()
        for b, n in enumerate(lens):
            nb = -(-n // cache.block)
            assert torch.equal(step[b, :, :nb], torch.ldexp(torch.ones(1, dtype=torch.float64), ref.exp[which, b, :, :nb]))
            assert torch.equal(got[b, :, :n], ref.codes[which, b, :, :n])


def err_of(cache):
    v = int(cache.err.item())
    cache.err.zero_()
    return v


# ------------------------------------------------------------ append, read

@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D,block,dtype", [(64, 16, torch.bfloat16), (128, 32, torch.float16), (256, 64, torch.float32),
                                           (64, 128, torch.float32), (256, 16, torch.bfloat16), (128, 128, torch.bfloat16)])
def test_append_and_read(fmt, D, block, dtype):
    """Prompts of unequal length, then single tokens and drafts at odd places
    of their blocks, magnitudes that grow (codes are rounded again) and shrink."""
    B, G, T = 3, 2, 4 * block
    cache = moe.KV8Cache(T, batch=B, q_heads=4, kv_heads=G, head_dim=D, block=block, fmt=fmt)
    ref = kv8_ref.Ref(B, G, D, T, block, fmt)
    r, pos = gen(5), [0, 0, 3]
    for M, counts, size in ((block + 7, [block + 7, 1, block // 2], 1.0), (1, None, 3.0), (1, None, 0.01), (4, [4, 0, 3], 40.0),
                            (block // 2 + 1, None, 700.0), (2, None, 2.0 ** -10)):
        k, v = rows(r, B, M, G, D, dtype=dtype, size=size), rows(r, B, M, G, D, dtype=dtype, size=0.3 * size)
        for _ in range(2):                       # again: nothing changes
            cache.append(k, v, i32(pos), counts=None if counts is None else i32(counts))
        ref.append(k, v, pos, counts)
        pos = [p + (M if counts is None else n) for p, n in zip(pos, counts or pos)]
        same_state(cache, ref, [0 if b == 2 else p for b, p in enumerate(pos)])
        assert err_of(cache) == 0
    start = [0, 2, -1]
    n = max(pos)
    k, v = cache.read(i32(start), n, lens=i32(pos))
    for which, got in enumerate((k, v)):
        want = torch.zeros((B, n, G, D), dtype=torch.float64)
        for b in range(2):
            for g in range(G):
                x = ref.values(which, b, g, pos[b])[start[b]:]
                want[b, :len(x), g] = x
        assert torch.equal(got[:2].cpu().double(), want[:2])
        assert not got[2, 0].any() and torch.isfinite(got[2].float()).all()


def test_append_takes_views_of_a_wider_projection():
    """k and v as slices of rows [B, M, n]: with aligned strides, and with odd
    ones (element loads), and a batch that shares one row (stride 0)."""
    B, M, G, D = 2, 3, 2, 64
    for pad, off in ((0, 0), (8, 8), (1, 0), (0, 1)):
        wide = rows(gen(7), B, M, 2 * G * D + pad + off)
        k = wide[:, :, off:off + G * D].unflatten(2, (G, D))
        v = wide[:, :, off + G * D:off + 2 * G * D].unflatten(2, (G, D))
        cache, ref = moe.KV8Cache(32, batch=B, q_heads=2, kv_heads=G, head_dim=D, block=16), kv8_ref.Ref(B, G, D, 32, 16, "int8")
        cache.append(k, v, i32([15, 0]))
        ref.append(k, v, [15, 0])
        same_state(cache, ref, [0, 3])
        assert torch.equal(cache.k[0, :, 15:18].cpu().double(), ref.codes[0, 0, :, 15:18])
    one = rows(gen(8), 1, M, G, D).expand(B, M, G, D)
    cache.append(one, one, i32([0, 0]))
    assert torch.equal(cache.k[0, :, :M], cache.k[1, :, :M])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_append_extremes(fmt, dtype):
    """The limits of a step (127.5 and 448 steps, one value beyond), ties, the
    smallest and largest numbers of the type, zeros, infinities and NaN."""
    D, fi = 64, torch.finfo(dtype)
    x = torch.zeros((1, 16 * 8, 1, D), dtype=torch.float64)
    blocks = x.view(8, 16, D)
    blocks[0, 0, :4] = torch.tensor([127.5, 0.5, 1.5, -2.5])
    blocks[1, 0, :4] = torch.tensor([128.0, -127.0, 126.5, 0.25])
    blocks[2, 0, :4] = torch.tensor([448.0, 17.0, -19.0, 2.0 ** -9])
    blocks[3, 0, :4] = torch.tensor([449.0 if dtype != torch.bfloat16 else 452.0, 3.0, -1.0, 2.0 ** -8])
    blocks[4, 3, :3] = torch.tensor([fi.tiny, -fi.smallest_normal, fi.smallest_normal / 2 if dtype != torch.float32 else 0.0])
    blocks[5, 15, :3] = torch.tensor([fi.max, -fi.max, 1.0])
    blocks[7, 1, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 1.0])
    x = x.to(dtype).to(DEV)
    cache, ref = moe.KV8Cache(128, q_heads=1, kv_heads=1, head_dim=D, block=16, fmt=fmt), kv8_ref.Ref(1, 1, D, 128, 16, fmt)
    cache.append(x[:, :112], x[:, :112], i32([0]))
    assert err_of(cache) == 0
    cache.append(x[:, 112:], x[:, 112:], i32([112]))
    assert err_of(cache) == moe.KV8Cache.ERR_NONFINITE
    ref.append(x, x, [0])
    same_state(cache, ref, [128])


def test_append_idle_and_out_of_range():
    """Idle sequences and rows past the cache write nothing; the error word
    says when a row was left out."""
    cache = moe.KV8Cache(64, batch=4, q_heads=2, kv_heads=2, head_dim=64, block=16)
    k = rows(gen(9), 4, 5, 2, 64)
    cache.append(k, k, i32([-1, 3, -2 ** 31, 59]))
    assert err_of(cache) == 0
    assert not cache.k[0].any() and not cache.k[2].any() and not cache.k[1, :, :3].any() and not cache.k[1, :, 8:].any()
    before = cache.k.clone()
    cache.append(k, k, i32([-1, 2 ** 31 - 1, 64, 62]))
    assert err_of(cache) == moe.KV8Cache.ERR_RANGE
    assert torch.equal(cache.k[:, :, :62], before[:, :, :62]) and torch.equal(cache.k[1], before[1])
    cache.append(k, k, i32([0, -1, -1, -1]), counts=i32([9, 9, -4, 0]))
    assert err_of(cache) == moe.KV8Cache.ERR_RANGE
    assert cache.k[0, :, :5].any() and not cache.k[0, :, 5:].any()
    cache.append(k, k, i32([-1, 10, -1, 64]), counts=i32([1, 0, 1, 0]))
    assert err_of(cache) == 0


def test_rewound_draft_keeps_its_block_readable():
    """Appending at an earlier position (rejected drafts) keeps the block's
    step; a block whose first position is rewritten starts anew."""
    cache, ref = moe.KV8Cache(64, q_heads=1, kv_heads=1, head_dim=64, block=16), kv8_ref.Ref(1, 1, 64, 64, 16, "int8")
    r = gen(10)
    for pos, M, size in ((0, 10, 1.0), (10, 4, 90.0), (11, 2, 0.1), (16, 3, 50.0), (16, 2, 0.01)):
        k = rows(r, 1, M, 1, 64, size=size)
        cache.append(k, -k, i32([pos]))
        ref.append(k, -k, [pos])
    same_state(cache, ref, [18])
    assert float(cache.k_scale[0, 0, 1]) < 2.0 ** -9


# ---------------------------------------------------------------- attention

def filled(B, Hq, G, D, T, block, fmt, lens, seed, size=1.0, rows_max=8, weights=False, dtype=torch.bfloat16):
    """A cache whose sequences hold lens[b] positions, everything else the
    bytes and steps that would show (NaN codes of e4m3, NaN steps)."""
    cache = moe.KV8Cache(T, batch=B, q_heads=Hq, kv_heads=G, head_dim=D, block=block, fmt=fmt, max_rows=rows_max, weights=weights)
    cache.k.view(torch.uint8).fill_(0x7F)
    cache.v.view(torch.uint8).fill_(0xFF)
    cache.k_scale.fill_(float("nan"))
    cache.v_scale.fill_(float("nan"))
    cache.ws.fill_(0xFF)
    r, M = gen(seed), max(max(lens), 1)
    k, v = rows(r, B, M, G, D, dtype=dtype, size=size), rows(r, B, M, G, D, dtype=dtype, size=size)
    cache.append(k, v, i32([0 if n > 0 else -1 for n in lens]), counts=i32([max(n, 0) for n in lens]))
    assert err_of(cache) == 0
    return cache, r


def check(cache, q, pos, counts=None, scale=None, out_dtype=torch.float32, acc=None, acc_in=None, decay=1.0):
    ref = kv8_ref.of_cache(cache)
    o, oabs, smax, w = ref.attend(q, pos, counts, scale)
    before = None if acc is None else acc.clone()
    was = None if acc is None else (before if acc_in is None else acc_in).clone()
    got, err = cache.attend(q, i32(pos), counts=None if counts is None else i32(counts), scale=scale, acc=acc, acc_in=acc_in,
                            decay=decay, out_dtype=out_dtype)
    assert err is cache.err and err_of(cache) == 0
    assert got.dtype == out_dtype and got.shape == q.shape
    D, chunks = cache.head_dim, cache.T_cap // 128 + 1
    ew = (D + 12) * E23 * smax + 8 * E23 + 2.0 ** -22            # of a weight, relative
    tol = 2 * (ew + (1024 + chunks) * E23) * oabs + HALF[out_dtype] * o.abs() + (2.0 ** -24 if out_dtype == torch.float16 else 1e-30)
    d = (got.double().cpu() - o).abs()
    assert torch.isfinite(got.float()).all()
    assert (d <= tol).all(), f"worst {float((d / tol).max()):.3g} tolerances at {np.unravel_index(int((d / tol).argmax()), d.shape)}"
    if acc is not None:
        B, M, Hq, T = w.shape
        G = cache.kv_heads
        want, tol = torch.zeros((B, G, T), dtype=torch.float64), torch.zeros((B, G, T), dtype=torch.float64)
        ew = 2 * (ew + (1024 + chunks) * E23)
        for b in range(B):
            rows_b = M if counts is None else min(max(counts[b], 0), M)
            n = 0 if pos[b] < 0 or rows_b == 0 else min(T, pos[b] + rows_b)      # no rows: left alone
            want[b, :, n:] = before[b, :, n:].cpu()
            p = max(0, min(pos[b], n))
            if n:
                want[b, :, :p] = decay * was[b, :, :p].cpu().double()
                want[b, :, :n] += w[b, :, :, :n].sum(0).view(G, Hq // G, n).sum(1)
                tol[b, :, :n] = (ew[b] * w[b, :, :, :n]).sum(0).view(G, Hq // G, n).sum(1) + (Hq // G * M + 2) * E23 * want[b, :, :n]
        d = (acc.double().cpu() - want).abs()
        d[want.isnan() & acc.cpu().isnan()] = 0.0                    # left alone: as they were
        assert (d <= tol + 1e-30).all(), f"weights: worst {float((d / (tol + 1e-30)).max()):.3g} tolerances"
    return got


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D,Hq,G,block,M", [(256, 16, 2, 64, 1), (256, 16, 2, 64, 3), (128, 32, 8, 32, 1), (64, 6, 6, 16, 2),
                                            (128, 10, 2, 128, 1), (64, 64, 1, 16, 1), (256, 5, 1, 32, 8), (128, 16, 1, 64, 8),
                                            (64, 24, 2, 128, 4)])
def test_attention_matches_definition(fmt, D, Hq, G, block, M):
    """Lengths of one to a few chunks, ends inside and at tiles, blocks and
    chunks, an idle sequence, one without any earlier position."""
    lens = [M, M + 15, M + 16, M + 31, 255, 257, 700, 1024, -1]
    cache, r = filled(len(lens), Hq, G, D, 1024, block, fmt, lens, 11)
    q = rows(r, len(lens), M, Hq, D, size=1.5)
    o = check(cache, q, [n - M if n > 0 else -1 for n in lens])
    assert not o[-1].any()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype,out_dtype", [(torch.float16, torch.float16), (torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32)])
def test_attention_types_counts_and_strides(fmt, dtype, out_dtype):
    """Padded rows, q as a slice of a wider projection, an explicit scale."""
    lens = [40, 130, 5]
    cache, r = filled(3, 8, 2, 128, 160, 32, fmt, lens, 12)
    q = rows(r, 3, 4, 9 * 128 + 3, dtype=dtype)[:, :, 3:3 + 8 * 128].unflatten(2, (8, 128))
    assert not q.is_contiguous()
    o = check(cache, q, [36, 126, 1], counts=[4, 1, 0], scale=0.2, out_dtype=out_dtype)
    assert not o[1, 1:].any() and not o[2].any()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_attention_over_unequal_blocks(fmt):
    """Blocks whose steps differ by many powers of two: one of keys that takes
    all the weight, values that are tiny where the weight is."""
    B, Hq, G, D, T, block = 1, 8, 1, 128, 512, 16
    for case in range(4):
        cache = moe.KV8Cache(T, batch=B, q_heads=Hq, kv_heads=G, head_dim=D, block=block, fmt=fmt)
        r = gen(13 + case)
        k, v = rows(r, B, T, G, D, dtype=torch.float32), rows(r, B, T, G, D, dtype=torch.float32)
        s = torch.ones(T, device=DEV)
        if case == 0:
            s = torch.exp2(torch.randint(-8, 8, (T // block,), device=DEV, generator=r).float()).repeat_interleave(block)
        if case == 1:
            s[:256] = 2.0 ** -30                      # a chunk of tiny values beside normal ones
        if case == 2:
            s[::1] = 2.0 ** -100
        if case == 3:
            s[:] = 2.0 ** 100
        v = v * s[:, None, None]
        k[:, 300:302] *= 4.0
        if case == 0:
            k = k * s.flip(0)[:, None, None].clamp(max=4)
        cache.append(k, v, i32([0]))
        check(cache, rows(r, B, 1, Hq, D), [T - 1])


def test_attention_large_scores():
    """Scores of hundreds: one position takes everything."""
    cache, r = filled(1, 16, 2, 256, 512, 64, "int8", [500], 14, size=8.0)
    o = check(cache, rows(r, 1, 1, 16, 256, size=30.0), [499])
    assert float(o.abs().max()) > 4.0
    tiny = check(cache, rows(r, 1, 1, 16, 256, size=1e-30), [499])    # every weight the same
    assert torch.isfinite(tiny).all()
    check(cache, torch.zeros((1, 2, 16, 256), dtype=torch.bfloat16, device=DEV), [498])


def test_attention_nan_query_stays_in_its_row():
    cache, r = filled(1, 16, 2, 256, 512, 64, "int8", [500], 15)
    q = rows(r, 1, 2, 16, 256)
    clean, _ = cache.attend(q, i32([498]))
    q[0, 1, 3, 7] = float("nan")
    q[0, 0, 9, 0] = float("inf")
    o, _ = cache.attend(q, i32([498]))
    assert o[0, 1, 3].isnan().all() and o[0, 0, 9].isnan().all()
    o[0, 1, 3], o[0, 0, 9] = clean[0, 1, 3], clean[0, 0, 9]
    assert torch.equal(o, clean)


@pytest.mark.parametrize("fmt,D,Hq,G,T", [("int8", 256, 16, 2, 2048), ("e4m3", 128, 32, 8, 1024), ("int8", 64, 4, 4, 12288)])
def test_rows_and_sequences_do_not_interact(fmt, D, Hq, G, T):
    """Row m of a call of 8 rows is bitwise the one-row call at its position,
    and a sequence's rows are bitwise the same in another batch."""
    lens = [T - 3, 900]
    cache, r = filled(2, Hq, G, D, T, 64, fmt, lens, 16)
    q = rows(r, 2, 8, Hq, D)
    pos = [n - 8 for n in lens]
    all_rows, _ = cache.attend(q, i32(pos))
    for m in (0, 3, 7):
        one, _ = cache.attend(q[:, m:m + 1], i32([p + m for p in pos]))
        assert torch.equal(one[:, 0], all_rows[:, m])
    alone, _ = cache.attend(q, i32([pos[0], -1]))
    assert torch.equal(alone[0], all_rows[0]) and not alone[1].any()
    fewer, _ = cache.attend(q, i32(pos), counts=i32([8, 2]))
    assert torch.equal(fewer[0], all_rows[0]) and torch.equal(fewer[1, :2], all_rows[1, :2]) and not fewer[1, 2:].any()
    again, _ = cache.attend(q, i32(pos))
    assert torch.equal(again, all_rows)


def test_attention_out_of_range():
    cache, r = filled(3, 2, 1, 64, 64, 16, "int8", [64, 64, 64], 17)
    q = rows(r, 3, 3, 2, 64)
    want, _ = cache.attend(q, i32([61, 61, 61]))
    o, _ = cache.attend(q, i32([62, 2 ** 31 - 1, 61]), counts=i32([3, 1, 3]))
    assert err_of(cache) == moe.KV8Cache.ERR_RANGE
    assert torch.equal(o[2], want[2]) and not o[1].any() and not o[0, 2].any() and o[0, :2].any()


@pytest.mark.parametrize("D,Hq,G,M,T,lens", [(256, 16, 2, 1, 1024, [1000, 1, -1, 513]), (64, 32, 8, 2, 512, [2, 300, 17, 512]),
                                             (128, 20, 1, 7, 512, [511, 7, 300, 128])])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_position_weights(fmt, D, Hq, G, M, T, lens):
    """acc in place, from another tensor, with decay, and with none before."""
    cache, r = filled(4, Hq, G, D, T, 64, fmt, lens, 18, weights=True)
    q = rows(r, 4, M, Hq, D, size=2.0)
    pos = [n - M if n > 0 else -1 for n in lens]
    acc = torch.rand((4, G, T), generator=r, device=DEV)
    check(cache, q, pos, acc=acc)
    check(cache, q, pos, acc=acc, acc_in=torch.rand((4, G, T), generator=r, device=DEV), decay=0.5)
    check(cache, q, pos, acc=acc, acc_in=torch.zeros_like(acc), counts=[M, max(M - 1, 0), 1, 0])
    plain, _ = cache.attend(q, i32(pos))
    withw, _ = cache.attend(q, i32(pos), acc=acc)
    assert torch.equal(plain, withw)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_long_cache(fmt):
    """Tens of thousands of positions: many chunks per row."""
    cache, r = filled(2, 16, 2, 256, 40960, 64, fmt, [40000, 32769], 19, rows_max=4, weights=True)
    acc = torch.zeros((2, 2, 40960), device=DEV)
    check(cache, rows(r, 2, 4, 16, 256), [39996, 32765], acc=acc)


def test_offsets_past_32_bits():
    """The last sequence of a cache of more than 2^32 codes gives what a small cache gives."""
    T, G, D = 1 << 20, 8, 256
    big = moe.KV8Cache(T, batch=3, q_heads=8, kv_heads=G, head_dim=D, block=128, max_rows=1, weights=False,
                       buffers=tuple(torch.empty((3, G, T, D), dtype=torch.int8, device=DEV) for _ in range(2)) +
                       tuple(torch.empty((3, G, T // 128), device=DEV) for _ in range(2)))
    small = moe.KV8Cache(1024, batch=1, q_heads=8, kv_heads=G, head_dim=D, block=128, max_rows=1)
    r = gen(20)
    k, v, q = rows(r, 3, 200, G, D), rows(r, 3, 200, G, D), rows(r, 3, 1, 8, D)
    big.append(k, v, i32([-1, -1, 0]))
    small.append(k[2:], v[2:], i32([0]))
    assert torch.equal(big.k[2, :, :200], small.k[0, :, :200])
    o, _ = big.attend(q, i32([-1, -1, 199]))
    want, _ = small.attend(q[2:], i32([199]))
    assert float((o[2] - want[0]).abs().max()) <= 1e-5 and not o[:2].any()
    got, _ = big.read(i32([0, 0, 0]), 200, lens=i32([0, 0, 200]))
    assert torch.equal(got[2], small.read(None, 200)[0][0])
    idx, n = big.evict_into(moe.KV8Cache(128, batch=3, q_heads=8, kv_heads=G, head_dim=D, block=128, max_rows=1),
                            i32([0, 0, 200]), torch.ones((3, G, T), device=DEV), 128, sinks=0)
    assert n.tolist() == [0, 0, 128] and idx[2, 7].tolist() == list(range(128)) and (idx[:2] == -1).all()


# ------------------------------------------------------------------ eviction

def check_evict(cache, lens, acc, budget, sinks, recent, dT=None):
    dT = dT or -(-budget // cache.block) * cache.block
    dst = moe.KV8Cache(dT, batch=cache.batch, q_heads=cache.q_heads, kv_heads=cache.kv_heads, head_dim=cache.head_dim,
                       block=cache.block, fmt=cache.fmt)
    dst.k.view(torch.uint8).fill_(0x55)
    dst.k_scale.fill_(-1.0)
    dacc = torch.full((cache.batch, cache.kv_heads, dT), -7.0, device=DEV)
    ref, want = kv8_ref.of_cache(cache), kv8_ref.Ref(cache.batch, cache.kv_heads, cache.head_dim, dT, cache.block, cache.fmt)
    keep = ref.evict(want, lens, acc.cpu(), budget, sinks, recent)
    idx, n = cache.evict_into(dst, i32(lens), acc, budget, sinks=sinks, recent=recent, dst_acc=dacc)
    assert err_of(cache) == 0
    kept = [min(max(x, 0), budget) for x in lens]
    assert n.tolist() == kept
    for b in range(cache.batch):
        for g in range(cache.kv_heads):
            assert idx[b, g].tolist() == keep[b][g] + [-1] * (budget - kept[b])
            a = acc[b, g, torch.tensor(keep[b][g], dtype=torch.long, device=DEV)]
            assert torch.equal(dacc[b, g, :kept[b]].view(torch.int32), a.view(torch.int32))
            assert (dacc[b, g, kept[b]:] == -7.0).all()
        assert (dst.k.view(torch.uint8)[b, :, kept[b]:] == 0x55).all()
        assert (dst.k_scale[b, :, -(-kept[b] // cache.block):] == -1.0).all()
    same_state(dst, want, kept)
    return dst, n, dacc


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D,G,block,T,lens,budget,sinks,recent", [
    (64, 2, 16, 256, [256, 100, 33, 32, 31, 0, -1], 32, 4, 8), (256, 2, 64, 640, [640, 321], 320, 0, 0),
    (128, 3, 32, 512, [512, 500], 77, 5, 72), (128, 1, 128, 2048, [2047, 1500], 1, 0, 0), (64, 1, 16, 4096, [4096, 1025], 1024, 16, 1),
    (64, 1, 64, 64, [64, 5], 64, 3, 3)])
def test_evict(fmt, D, G, block, T, lens, budget, sinks, recent):
    """More and fewer positions than the budget, one more and as many, all of
    them forced, a budget of one, odd sizes; blocks of differing steps."""
    B = len(lens)
    cache, r = filled(B, 2 * G, G, D, T, block, fmt, lens, 21)
    cache.append(rows(r, B, 9, G, D, size=25.0), rows(r, B, 9, G, D, size=0.01), i32([max(n // 2 - 9, 0) if n > 20 else -1 for n in lens]))
    acc = torch.randn((B, G, T), generator=r, device=DEV).exp()
    check_evict(cache, lens, acc, budget, sinks, recent)


@pytest.mark.parametrize("kind", ["ties", "zeros", "nan", "inf", "close", "negative"])
def test_evict_ranks(kind):
    """Equal weights go to the lower position, NaN last, -0 as 0, neighbours
    one bit apart."""
    B, G, T = 2, 2, 2992
    lens = [T, T - 5]
    cache, r = filled(B, G, G, 64, T, 16, "int8", lens, 22)
    acc = torch.randn((B, G, T), generator=r, device=DEV).abs()
    u = torch.rand((B, G, T), generator=r, device=DEV)
    if kind == "ties":
        acc = (acc * 2).round()
    elif kind == "zeros":
        acc = torch.where(u < 0.9, torch.where(u < 0.4, -0.0, 0.0), acc)
    elif kind == "nan":
        acc = torch.where(u < 0.95, float("nan"), -acc)
    elif kind == "inf":
        acc = torch.where(u < 0.3, float("inf"), torch.where(u > 0.5, -float("inf"), acc))
    elif kind == "close":
        acc = (torch.ones_like(acc).view(torch.int32) + (u * 40).int()).view(torch.float32)
    else:
        acc = -acc
    check_evict(cache, lens, acc, 1000, 4, 16)


def test_evict_long():
    """More positions than one CTA's share, several blocks of the selection."""
    cache, r = filled(2, 2, 2, 64, 131072, 128, "int8", [131072, 99999], 23)
    acc = torch.randn((2, 2, 131072), generator=r, device=DEV).exp()
    acc[0, 0, 5000:120000] = 0.5
    ref = kv8_ref.Ref(1, 1, 64, 128, 128, "int8")
    dst = moe.KV8Cache(16384, batch=2, q_heads=2, kv_heads=2, head_dim=64, block=128)
    idx, n = cache.evict_into(dst, i32([131072, 99999]), acc, 16301, sinks=7, recent=1000)
    assert n.tolist() == [16301, 16301]
    for b, ln in enumerate((131072, 99999)):
        for g in range(2):
            want = ref.kept(ln, acc[b, g].tolist(), 16301, 7, 1000)
            assert idx[b, g].tolist() == want
            at = torch.tensor(want, device=DEV)
            s = cache.v_scale[b, g, at // 128]
            got = dst.v[b, g, :16301].double() * dst.v_scale[b, g].repeat_interleave(128)[:16301, None].double()
            # one rounding to a step that is no smaller
            assert ((got - cache.v[b, g, at].double() * s[:, None].double()).abs().amax(1) <= dst.v_scale[b, g].repeat_interleave(128)[:16301].double() / 2).all()


def test_evict_length_past_the_cache():
    cache, r = filled(1, 1, 1, 64, 64, 16, "int8", [64], 24)
    dst = moe.KV8Cache(64, q_heads=1, kv_heads=1, head_dim=64, block=16)
    idx, n = cache.evict_into(dst, i32([65]), torch.ones((1, 1, 64), device=DEV), 64)
    assert err_of(cache) == moe.KV8Cache.ERR_RANGE and n.item() == 64 and idx.view(-1).tolist() == list(range(64))


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_decode_with_a_bounded_cache(fmt):
    """Prompt, tokens, weights, eviction to a smaller cache, more tokens, and
    the other cache again: at every step the state is the definition's bit
    for bit and the attention within its bound."""
    B, Hq, G, D, block = 2, 8, 2, 128, 16
    a = moe.KV8Cache(96, batch=B, q_heads=Hq, kv_heads=G, head_dim=D, block=block, fmt=fmt, weights=True)
    c = moe.KV8Cache(96, batch=B, q_heads=Hq, kv_heads=G, head_dim=D, block=block, fmt=fmt, weights=True)
    acc, acc2 = torch.zeros((B, G, 96), device=DEV), torch.full((B, G, 96), float("nan"), device=DEV)
    r, lens = gen(25), [0, 0]
    ref = kv8_ref.Ref(B, G, D, 96, block, fmt)
    k, v = rows(r, B, 50, G, D), rows(r, B, 50, G, D)
    a.append(k, v, i32(lens), counts=i32([50, 37]))
    ref.append(k, v, lens, [50, 37])
    lens = [50, 37]
    for step in range(60):
        M = 1 + step % 3
        k, v, q = rows(r, B, M, G, D, size=1 + step % 5), rows(r, B, M, G, D), rows(r, B, M, Hq, D)
        a.append(k, v, i32(lens))
        ref.append(k, v, lens)
        same_state(a, ref, [n + M for n in lens])
        check(a, q, lens, acc=acc, decay=0.9)
        lens = [n + M for n in lens]
        if max(lens) > 90:
            nxt = kv8_ref.Ref(B, G, D, 96, block, fmt)
            keep = ref.evict(nxt, lens, acc.cpu(), 64, 4, 8)
            idx, n = a.evict_into(c, i32(lens), acc, 64, sinks=4, recent=8, dst_acc=acc2)
            assert [[x for x in h if x >= 0] for s in idx.tolist() for h in s] == [h for s in keep for h in s]
            a, c, acc, acc2, ref, lens = c, a, acc2, acc, nxt, n.tolist()
            same_state(a, ref, lens)


def test_captured_decode_step():
    """A graph of append, attention with weights and eviction replays with the
    lengths and rows of the moment, as eager calls on another stream do."""
    B, Hq, G, D, T = 3, 8, 2, 64, 512
    r = gen(26)
    cache, other = filled(B, Hq, G, D, T, 32, "int8", [300, 64, 1], 27, weights=True)[0], None
    other = moe.KV8Cache(T, batch=B, q_heads=Hq, kv_heads=G, head_dim=D, block=32, weights=True,
                         buffers=tuple(t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)))
    pos, acc, acc_o = i32([300, 64, 1]), torch.zeros((B, G, T), device=DEV), torch.zeros((B, G, T), device=DEV)
    k, v, q = rows(r, B, 1, G, D), rows(r, B, 1, G, D), rows(r, B, 1, Hq, D)
    dst = moe.KV8Cache(64, batch=B, q_heads=Hq, kv_heads=G, head_dim=D, block=32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step(c, acc):
        c.append(k, v, pos)
        o, _ = c.attend(q, pos, acc=acc)
        idx, n = c.evict_into(dst, pos + 1, acc, 64, sinks=2, recent=4)
        return o, idx, n
    with torch.cuda.stream(side):
        step(cache, acc.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, idx, n = step(cache, acc)
    for i in range(5):
        if i:
            pos.add_(1)
            for t in (k, v, q):
                t.copy_(torch.randn(t.shape, generator=r, device=DEV))
        graph.replay()
        got = [t.clone() for t in (o, idx, n, acc, dst.k)]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            eo, ei, en = step(other, acc_o)
        torch.cuda.synchronize()
        for x, y in zip(got, (eo, ei, en, acc_o, dst.k)):
            assert torch.equal(x, y)
        assert torch.equal(cache.k, other.k) and torch.equal(cache.v_scale.view(torch.int32), other.v_scale.view(torch.int32))
    assert err_of(cache) == 0


def test_binding_refusals():
    cache = moe.KV8Cache(64, batch=2, q_heads=4, kv_heads=2, head_dim=64, block=16, max_rows=2)
    k, q, p = torch.zeros((2, 1, 2, 64), dtype=torch.bfloat16, device=DEV), torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16, device=DEV), i32([0, 0])
    acc = torch.zeros((2, 2, 64), device=DEV)
    dst = moe.KV8Cache(64, batch=2, q_heads=4, kv_heads=2, head_dim=64, block=16)
    for bad in (lambda: cache.append(k[:1], k[:1], p), lambda: cache.append(k, k.half(), p), lambda: cache.append(k, k.cpu(), p),
                lambda: cache.append(k.long(), k.long(), p), lambda: cache.append(k, k, p.long()), lambda: cache.append(k, k, p[:1]),
                lambda: cache.append(k, k, None), lambda: cache.append(k.transpose(1, 3), k.transpose(1, 3), p),
                lambda: cache.append(k[..., ::2], k[..., ::2], p), lambda: cache.append(k, k, p.cpu()),
                lambda: cache.attend(k, p), lambda: cache.attend(q.float(), p), lambda: cache.attend(q, p, acc_in=acc),
                lambda: cache.attend(q, p, acc=acc[:, :1]), lambda: cache.attend(q, p, out=torch.zeros((2, 1, 4, 32), device=DEV)),
                lambda: cache.attend(q, p, out_dtype=torch.float64), lambda: cache.read(p[:1], 4),
                lambda: cache.evict_into(cache.k, p, acc, 8), lambda: cache.evict_into(dst, p, acc, 0),
                lambda: cache.evict_into(dst, p, acc.half(), 8), lambda: cache.attend(q.repeat(1, 3, 1, 1), p),
                lambda: cache.attend(q, p, acc=acc)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: cache.read(None, 65), lambda: cache.evict_into(dst, p, acc, 65),
                lambda: cache.evict_into(dst, p, acc, 8, sinks=6, recent=3), lambda: cache.evict_into(cache, p, acc, 8),
                lambda: cache.append(k.repeat(1, 65, 1, 1), k.repeat(1, 65, 1, 1), p)):
        with pytest.raises(moe.MoeError):
            bad()
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_evict_far_apart_steps_and_zeros(fmt):
    """Blocks whose steps are as far apart as fp32 allows, rows of zeros under a
    large step beside small values, the smallest codes alone in a block."""
    cache, r = filled(1, 2, 2, 64, 256, 16, fmt, [256], 28)
    k = torch.zeros((1, 256, 2, 64), device=DEV)
    k[0, :16] = rows(r, 16, 2, 64, dtype=torch.float32) * 2.0 ** 110
    k[0, 3:16:2] = 0.0
    k[0, 16:32] = rows(r, 16, 2, 64, dtype=torch.float32) * 2.0 ** -119
    k[0, 32] = 1.0
    k[0, 33:48, :, ::7] = 1.0 / 512
    k[0, 48:64] = rows(r, 16, 2, 64, dtype=torch.float32) * 1e-3
    k[0, 64:] = rows(r, 192, 2, 64, dtype=torch.float32)
    cache.append(k, k * 2.0 ** -3, i32([0]))
    acc = torch.rand((1, 2, 256), generator=r, device=DEV)
    acc[0, 0, 3:16:2] += 2.0
    acc[0, 0, 16:32] += 1.0
    acc[0, 1, 33:64] += 2.0
    check_evict(cache, [256], acc, 40, 0, 0)
    check_evict(cache, [256], 3 - acc, 100, 2, 5)


@pytest.mark.parametrize("T,lens", [(512, [300, 64, 1]), (40960, [30000, 12, 40900])])
def test_calls_in_a_row_equal_calls_waited_for(T, lens):
    """Steps enqueued without a wait, each reading what the ones before wrote (rows,
    lengths, weights in place, kept positions), give the bits of the same steps
    with the device waited for after every call."""
    B, Hq, G, D = 3, 8, 2, 128
    out = []
    for wait in (True, False):
        cache, r = filled(B, Hq, G, D, T, 32, "int8", lens, 29, weights=True)
        dst = moe.KV8Cache(256, batch=B, q_heads=Hq, kv_heads=G, head_dim=D, block=32)
        pos, acc, dacc = i32(lens), torch.zeros((B, G, T), device=DEV), torch.zeros((B, G, 256), device=DEV)
        steps = [(rows(r, B, 1, G, D), rows(r, B, 1, G, D), rows(r, B, 1, Hq, D, size=2.0)) for _ in range(25)]
        torch.cuda.synchronize()
        got = []

        def done():
            if wait:
                torch.cuda.synchronize()
        for k, v, q in steps:
            cache.append(k, v, pos)
            done()
            o, _ = cache.attend(q, pos, acc=acc, decay=0.97)
            done()
            pos.add_(1)
            done()
            idx, n = cache.evict_into(dst, pos, acc, 200, sinks=2, recent=5, dst_acc=dacc)
            done()
            kv = dst.read(None, 200, lens=n)
            done()
            got += [o, idx, *kv]
        torch.cuda.synchronize()
        assert err_of(cache) == 0
        out.append(got + [acc, dacc])
    for x, y in zip(*out):
        assert torch.equal(x, y)


@pytest.mark.parametrize("D,Hq,G", [(64, 4, 2), (128, 8, 2), (256, 8, 1)])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_rows_do_not_feel_later_rows_steps(fmt, D, Hq, G):
    """A call whose last rows' values lie in a block of a far larger step gives its
    first rows the bits of one-row calls, whose positions end before that block."""
    T, n = 512, 328                                   # rows 328 .. 335 | 336 ..: blocks of 16, tiles of up to 64
    cache, r = filled(1, Hq, G, D, T, 16, fmt, [n], 30)
    k, v = rows(r, 1, 16, G, D), rows(r, 1, 16, G, D)
    v[:, 8:] *= 3000.0
    cache.append(k, v, i32([n]))
    q = rows(r, 1, 8, Hq, D, size=3.0)
    for first in (n, n + 4, n + 7):
        all_rows, _ = cache.attend(q, i32([first]))
        for m in range(8):
            one, _ = cache.attend(q[:, m:m + 1], i32([first + m]))
            assert torch.equal(one[:, 0], all_rows[:, m]), (first, m)


def test_many_sequences():
    """More sequences than threads of a CTA and more chunks than CTAs: every
    sequence's rows against a batched 64-bit softmax."""
    B, Hq, G, D, T = 700, 8, 4, 64, 128
    r = gen(31)
    lens = torch.randint(0, T - 1, (B,), generator=r, device=DEV, dtype=torch.int32)
    lens[::7] = -1
    lens[5] = T - 2
    cache = moe.KV8Cache(T, batch=B, q_heads=Hq, kv_heads=G, head_dim=D, block=16, fmt="int8", max_rows=2, weights=True)
    cache.append(rows(r, B, T, G, D), rows(r, B, T, G, D), torch.zeros_like(lens))
    q = rows(r, B, 2, Hq, D, size=1.5)
    acc = torch.full((B, G, T), -3.0, device=DEV)
    o, _ = cache.attend(q, lens, acc=acc, acc_in=torch.zeros_like(acc))
    assert err_of(cache) == 0
    k, v = (t.double().transpose(1, 2) for t in cache.read(None, T))                 # [B, G, T, D]
    s = torch.einsum("bmghd,bgtd->bgmht", q.double().view(B, 2, G, Hq // G, D), k) * D ** -0.5
    see = torch.where(lens[:, None] >= 0, lens[:, None] + 1 + torch.arange(2, device=DEV), 0)
    s = s.masked_fill((torch.arange(T, device=DEV) >= see[:, :, None])[:, None, :, None], -float("inf"))
    w = torch.softmax(s, -1).nan_to_num(0.0)
    want = torch.einsum("bgmht,bgtd->bmghd", w, v).reshape(B, 2, Hq, D)
    wabs = torch.einsum("bgmht,bgtd->bmghd", w, v.abs()).reshape(B, 2, Hq, D)
    smax = 1.5 * 6 * D ** 0.5 * 4 * D ** -0.5 * D ** 0.5                             # above any scale * sum |q k| here
    assert ((o.double() - want).abs() <= 2 * ((D + 12) * E23 * smax + 2.0 ** -12) * wabs + 1e-30).all()
    total = w.sum((2, 3))
    seen = torch.arange(T, device=DEV) < see[:, 1][:, None, None]
    assert ((acc.double() - torch.where(seen, total, -3.0)).abs() <= 2 * ((D + 12) * E23 * smax + 2.0 ** -12) * total).all()


def test_more_chunks_than_three_waves():
    """2048 heads: CTAs take their chunks from the counter, call after call."""
    B, Hq, G, D, T = 256, 8, 8, 64, 512
    r = gen(32)
    cache = moe.KV8Cache(T, batch=B, q_heads=Hq, kv_heads=G, head_dim=D, block=32, fmt="e4m3", max_rows=1)
    cache.append(rows(r, B, T, G, D), rows(r, B, T, G, D), torch.zeros(B, dtype=torch.int32, device=DEV))
    q = rows(r, B, 1, Hq, D)
    pos = torch.randint(0, T, (B,), generator=r, device=DEV, dtype=torch.int32)
    k, v = (t.double().transpose(1, 2) for t in cache.read(None, T))
    s = torch.einsum("bhd,bhtd->bht", q[:, 0].double(), k) * D ** -0.5
    w = torch.softmax(s.masked_fill((torch.arange(T, device=DEV) > pos[:, None])[:, None], -float("inf")), -1)
    want, wabs = torch.einsum("bht,bhtd->bhd", w, v), torch.einsum("bht,bhtd->bhd", w, v.abs())
    first = None
    for _ in range(4):
        cache.ws.fill_(0xFF)
        o, _ = cache.attend(q, pos)
        assert ((o[:, 0].double() - want).abs() <= 2 * (76 * E23 * 24 * 4 + 2.0 ** -12) * wabs).all()
        first = o if first is None else first
        assert torch.equal(o, first)


@pytest.mark.parametrize("D,Hq,G,M,T,lens", [(64, 64, 1, 8, 64, [64, 30]), (128, 64, 1, 8, 64, [64, 9]), (256, 64, 1, 8, 64, [63, 64]),
                                             (64, 5, 1, 3, 96, [96, 17]), (256, 3, 3, 5, 16, [16, 5]), (128, 7, 1, 1, 32, [32, 1])])
def test_column_counts(D, Hq, G, M, T, lens):
    """512 columns, odd numbers of them, the smallest cache; with weights."""
    cache, r = filled(2, Hq, G, D, T, 16, "int8", lens, 33, weights=True)
    acc = torch.rand((2, G, T), generator=r, device=DEV)
    check(cache, rows(r, 2, M, Hq, D), [n - M for n in lens], acc=acc, decay=0.5)


def test_evict_into_a_larger_cache():
    cache, r = filled(2, 2, 2, 128, 256, 32, "int8", [256, 90], 34)
    check_evict(cache, [256, 90], torch.rand((2, 2, 256), generator=r, device=DEV), 100, 3, 10, dT=1024)


def test_a_stream_of_ones_own():
    """Calls on an explicit stream, with the inputs made on another."""
    cache, r = filled(1, 4, 2, 64, 64, 16, "int8", [40], 35)
    q, k, pos = rows(r, 1, 1, 4, 64), rows(r, 1, 1, 2, 64), i32([40])
    cache.append(k, k, pos)
    want, _ = cache.attend(q, pos)
    kv = cache.read(None, 41)
    other = moe.KV8Cache(64, batch=1, q_heads=4, kv_heads=2, head_dim=64, block=16,
                         buffers=tuple(t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other.append(k, k, pos, stream=st)
    o, _ = other.attend(q, pos, stream=st)
    kv2 = other.read(None, 41, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(o, want) and torch.equal(kv[0], kv2[0]) and torch.equal(kv[1], kv2[1])


def test_results_lie_in_the_writing_streams_memory():
    """A result for an explicit stream does not reuse memory that the current
    stream has freed and may still be reading."""
    cache, r = filled(1, 4, 2, 64, 64, 16, "int8", [40], 36)
    q, pos, lens, acc = rows(r, 1, 1, 4, 64), i32([39]), i32([40]), torch.zeros((1, 2, 64), device=DEV)
    dst = moe.KV8Cache(64, batch=1, q_heads=4, kv_heads=2, head_dim=64, block=16)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for make, call in ((lambda: torch.empty((1, 33, 2, 64), dtype=torch.bfloat16, device=DEV), lambda: cache.read(None, 33, stream=st)),
                       (lambda: torch.empty((1, 1, 4, 64), device=DEV), lambda: cache.attend(q, pos, stream=st)[:1]),
                       (lambda: torch.empty((1, 2, 17), dtype=torch.int32, device=DEV),
                        lambda: cache.evict_into(dst, lens, acc, 17, stream=st))):
        old = [make() for _ in range(4)]
        freed = {t.data_ptr() for t in old}
        del old
        got = call()
        assert not freed & {t.data_ptr() for t in got}
    torch.cuda.synchronize()


def test_numbers_past_31_bits_are_refused():
    cache = moe.KV8Cache(64, batch=1, q_heads=2, kv_heads=1, head_dim=64, block=16)
    dst = moe.KV8Cache(64, batch=1, q_heads=2, kv_heads=1, head_dim=64, block=16)
    lens, acc = i32([40]), torch.zeros((1, 1, 64), device=DEV)
    k = torch.zeros((1, 1, 1, 64), device=DEV).expand(1, 2 ** 32 + 1, 1, 64)
    for bad in (lambda: cache.evict_into(dst, lens, acc, 2 ** 32 + 8), lambda: cache.evict_into(dst, lens, acc, 8, sinks=2 ** 32),
                lambda: cache.evict_into(dst, lens, acc, 8, sinks=0, recent=2 ** 32 + 1), lambda: cache.append(k, k, lens)):
        with pytest.raises(ValueError):
            bad()


def test_rows_of_a_long_cache_do_not_interact():
    """As above where one row and eight are joined by different forms of the merge."""
    cache, r = filled(1, 16, 2, 256, 65536, 64, "int8", [65000], 37)
    q = rows(r, 1, 8, 16, 256)
    all_rows, _ = cache.attend(q, i32([64992]))
    for m in (0, 5, 7):
        one, _ = cache.attend(q[:, m:m + 1], i32([64992 + m]))
        assert torch.equal(one[:, 0].view(torch.int32), all_rows[:, m].view(torch.int32))
