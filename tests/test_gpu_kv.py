"""GPU parity of the 16-bit key/value cache (moe_kv_*) and of attention over
prompts (moe_window_attn) with their definitions in 64 bits (kv_ref.py, which
derives the tolerances)."""
import pytest
import torch

import kv_ref
import quantized_moe_decode_layer_gb300 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float16


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rows(r, *shape, dtype=BF, size=1.0):
    return (torch.randn(shape, generator=r, device=DEV) * size).to(dtype)


def err_of(t):
    v = int(t.item())
    t.zero_()
    return v


def filled(r, T, lens, G, D, dtype, Hq=None, window=None, sinks=0, **kw):
    """A cache whose sequence b has lens[b] positions (their keys and values as
    [B, n, G, D] too), and NaN everywhere else."""
    B, n = len(lens), max(max(lens), 1)
    cache = moe.KVCache(T, batch=B, q_heads=Hq or G, kv_heads=G, head_dim=D, dtype=dtype, window=window, sinks=sinks, **kw)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    k, v = rows(r, B, n, G, D, dtype=dtype), rows(r, B, n, G, D, dtype=dtype)
    cache.append(k, v, i32([0 if x > 0 else -1 for x in lens]), counts=i32([max(x, 0) for x in lens]))
    assert err_of(cache.err) == 0
    return cache, k, v


def check_cache(cache, k, v, q, pos, counts=None, prefix=None, scale=None):
    o, err = cache.attend(q, i32(pos), counts=None if counts is None else i32(counts), prefix=prefix, scale=scale)
    assert err_of(err) == 0
    M = q.shape[1]

    def of(x, i):
        def get(b, m):
            t = kv_ref.seen(pos[b] + m, cache.window, cache.sinks).to(DEV)
            own = x[b, t]
            return own if prefix is None else torch.cat([prefix[i], own])
        return get
    kv_ref.check_rows(o, q, of(k, 0), of(v, 1), lambda b, m: pos[b] >= 0 and m < (M if counts is None else counts[b]),
                      cache.head_dim ** -0.5 if scale is None else scale)
    return o


# ------------------------------------------------------------------- append

@pytest.mark.parametrize("window,sinks,T", [(None, 0, 90), (16, 4, 40), (16, 0, 23), (1, 2, 10)])
@pytest.mark.parametrize("dtype,given", [(BF, torch.float32), (FP, torch.float32), (BF, BF), (FP, FP), (FP, BF), (BF, FP)])
def test_append(window, sinks, T, dtype, given):
    """Prompts, tokens and drafts into linear caches and rings: every position
    that the ring holds has its last row's value, rounded; the rest is left alone."""
    r, B, G, D = gen(1), 3, 2, 64
    cache = moe.KVCache(T, batch=B, q_heads=4, kv_heads=G, head_dim=D, dtype=dtype, window=window, sinks=sinks, max_rows=1)
    cache.k.fill_(-7.0)
    cache.v.fill_(-9.0)
    want_k, want_v = cache.k.clone(), cache.v.clone()
    pos = [0, 2, -1]
    for M, counts in ((37, [37, 1, 5]), (1, None), (4, [4, 0, 4]), (8, None), (30, [30, 29, 1])):
        k, v = rows(r, B, M, G, D, dtype=given), rows(r, B, M, G, D, dtype=given, size=3.0)
        cache.append(k, v, i32(pos), counts=None if counts is None else i32(counts))
        for b in range(B):
            n = M if counts is None else counts[b]
            for m in range(n if pos[b] >= 0 else 0):
                s = int(kv_ref.slots(torch.tensor(pos[b] + m), window, sinks, T))
                want_k[b, :, s], want_v[b, :, s] = k[b, m].to(dtype), v[b, m].to(dtype)
            if pos[b] >= 0:
                pos[b] += n
        assert err_of(cache.err) == 0
        assert torch.equal(cache.k, want_k) and torch.equal(cache.v, want_v)


def test_append_strided_and_unaligned():
    r, B, M, G, D = gen(2), 2, 5, 3, 128
    cache = moe.KVCache(16, batch=B, q_heads=3, kv_heads=G, head_dim=D)
    wide = rows(r, B, M, 2 * G * D + 3, dtype=torch.float32)
    k, v = wide[:, :, 3:3 + G * D].unflatten(2, (G, D)), wide[:, :, 3 + G * D:].unflatten(2, (G, D))
    cache.append(k, v, i32([1, 7]))
    for b, p in enumerate((1, 7)):
        assert torch.equal(cache.k[b, :, p:p + M], k[b].to(BF).transpose(0, 1))
        assert torch.equal(cache.v[b, :, p:p + M], v[b].to(BF).transpose(0, 1))
    one = rows(r, 1, 1, G, D).expand(B, M, G, D)            # strides of 0
    cache.append(one, one, i32([0, 0]))
    assert torch.equal(cache.k[1, :, 0], one[0, 0]) and torch.equal(cache.k[0, :, 4], one[0, 0])


def test_out_of_range():
    """Rows behind the cache's end, bad counts: left out, zeros, reported."""
    r, T = gen(3), 20
    cache, k, v = filled(r, T, [20, 20, 20], 2, 64, BF, Hq=4)
    kn = rows(r, 3, 4, 2, 64)
    before = cache.k.clone()
    cache.append(kn, kn, i32([18, 2 ** 31 - 1, 4]), counts=i32([4, 4, -1]))
    assert err_of(cache.err) == moe.KVCache.ERR_RANGE
    assert torch.equal(cache.k[0, :, 18:], kn[0, :2].transpose(0, 1)) and torch.equal(cache.k[1:], before[1:])
    q = rows(r, 3, 4, 4, 64)
    o, err = cache.attend(q, i32([18, 2 ** 31 - 1, 4]), counts=i32([4, 4, 5]))
    assert err_of(err) == moe.KVCache.ERR_RANGE
    assert o[0, :2].any() and not o[0, 2:].any() and not o[1].any() and o[2].isfinite().all()
    q, kv = rows(r, 1, 70, 4, 64), rows(r, 1, 100, 2, 64)
    for p, c, n in ((50, 70, 50), (100, 70, 0), (31, 71, 69)):
        err = i32([0])
        o, _ = moe.window_attention(q, kv, kv, 8, pos=i32([p]), counts=i32([c]), err=err)
        assert err_of(err) == 1 and not o[0, n:].any() and (n == 0 or o[0, :n].any(-1).any(-1).all())


# ------------------------------------------------- tokens and drafts, windows

@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D,Hq,G,M", [(64, 4, 2, 1), (128, 32, 8, 1), (256, 16, 2, 1), (256, 16, 2, 2), (64, 5, 1, 3), (128, 1, 1, 8),
                                      (256, 16, 2, 4), (64, 64, 1, 1), (128, 64, 1, 3), (128, 10, 2, 5), (64, 64, 1, 8), (256, 40, 1, 8)])
def test_tokens_in_a_ring(dtype, D, Hq, G, M):
    """Lengths before, at and far behind the ring's end, windows that end inside and
    at tiles, an idle sequence; what was never written is NaN."""
    W, S = 200, 4
    T = S + W + M - 1 + (3 if D == 64 else 0)
    lens = [M, M + 1, 63 + M, 64 + M, T - 1 + M, T, T + 1, T + 130, 3 * T + 5, 0]
    cache, k, v = filled(gen(4), T, [max(n, 0) for n in lens], G, D, dtype, Hq=Hq, window=W, sinks=S, max_rows=M)
    q = rows(gen(5), len(lens), M, Hq, D, dtype=dtype, size=1.5)
    check_cache(cache, k, v, q, [n - M if n >= M else -1 for n in lens])


@pytest.mark.parametrize("W,S,T", [(1, 0, 8), (1, 3, 12), (7, 0, 15), (64, 64, 140), (128, 1, 137), (130, 300, 437), (5, 130, 142), (1000, 0, 1007)])
@pytest.mark.parametrize("Hq,M", [(2, 1), (2, 8), (32, 8)])
def test_windows(W, S, T, Hq, M):
    lens = [M, 9 + M, 64 + M, 128 + M, 129 + M, 450 + M, 2 * T + 3 + M]
    cache, k, v = filled(gen(6), T, lens, 1, 64, BF, Hq=Hq, window=W, sinks=S, max_rows=M)
    q = rows(gen(7), len(lens), M, Hq, 64, size=2.0)
    check_cache(cache, k, v, q, [n - M for n in lens])


@pytest.mark.parametrize("Hq,M", [(8, 4), (16, 8)])
def test_counts_scale_and_strides(Hq, M):
    """Padded rows with NaN in them, q as a slice of a wider projection, an explicit scale."""
    G, D = 2, 128
    lens = [40, 130, 5, 70]
    cache, k, v = filled(gen(8), 160, lens, G, D, FP, Hq=Hq)
    q = rows(gen(9), 4, M, (Hq + 2) * D, dtype=FP)[:, :, D:(Hq + 1) * D].unflatten(2, (Hq, D))
    counts = [M, 1, 0, 2]
    for b, c in enumerate(counts):
        q[b, c:] = float("nan")
    o = check_cache(cache, k, v, q, [n - M for n in lens], counts=counts, scale=0.2)
    assert not o[2].any() and not o[1, 1:].any()


def test_many_sequences_of_all_lengths():
    """More sequences than a CTA's threads, most of them idle or short."""
    B, T = 300, 257
    lens = [(7 * b) % 258 if b % 3 else 0 for b in range(B)]
    cache, k, v = filled(gen(10), T, lens, 1, 64, BF, Hq=2)
    check_cache(cache, k, v, rows(gen(11), B, 1, 2, 64), [n - 1 for n in lens])


@pytest.mark.parametrize("D,Hq,M", [(64, 8, 1), (128, 32, 4), (256, 16, 2), (256, 16, 8)])
def test_rising_scores(D, Hq, M):
    """Keys whose scores rise along the sequence, over the reference again and
    again, then fall far below it; and scores of hundreds."""
    G, T = Hq // 8, 900
    cache, k, v = filled(gen(12), T, [T, T], G, D, BF, Hq=Hq)
    q = rows(gen(13), 2, M, Hq, D)
    q[..., 0] = 2.0
    ramp = torch.cat([torch.linspace(-60, 90, 600), torch.linspace(90, -200, 300)]).to(DEV)
    k[0, :, :, 0] = (ramp * D ** 0.5 / 2).to(BF)[:, None]
    k[1] *= 12.0
    cache.append(k, v, i32([0, 0]))
    check_cache(cache, k, v, q, [T - M, T - M])


def test_one_visible_position_is_its_value():
    """A window of 1 without first positions: the weight is 1, exactly."""
    for Hq, M in ((4, 1), (16, 4)):
        cache, k, v = filled(gen(14), 40, [90, 3], 2, 128, BF, Hq=Hq, window=1, max_rows=M)
        q = rows(gen(15), 2, M, Hq, 128, size=30.0)
        o, _ = cache.attend(q, i32([90 - M, -1]))
        want = v[0, 90 - M:90].repeat_interleave(Hq // 2, 1)
        assert torch.equal(o[0], want) and not o[1].any()
    k = rows(gen(16), 1, 300, 2, 64)
    o, _ = moe.window_attention(rows(gen(17), 1, 300, 8, 64, size=9.0), k, k, 1)
    assert torch.equal(o[0], k[0].repeat_interleave(4, 1))


@pytest.mark.parametrize("Hq,M", [(2, 2), (16, 4)])
def test_nan_and_infinity_stay_in_their_rows(Hq, M):
    """A query with NaN or infinity: its own row.  A key with one: the rows that see it."""
    cache, k, v = filled(gen(18), 300, [200], 2, 128, BF, Hq=Hq)
    q = rows(gen(19), 1, M, Hq, 128)
    clean, _ = cache.attend(q, i32([200 - M]))
    bad = q.clone()
    bad[0, 1, 1, 7], bad[0, 0, Hq - 1, 0] = float("nan"), float("inf")
    o, _ = cache.attend(bad, i32([200 - M]))
    assert o[0, 1, 1].isnan().all() and o[0, 0, Hq - 1].isnan().all()
    o[0, 1, 1], o[0, 0, Hq - 1] = clean[0, 1, 1], clean[0, 0, Hq - 1]
    assert torch.equal(o, clean)
    cache.k[0, :, 199, 3] = float("nan")              # the last row's own key
    o, _ = cache.attend(q, i32([200 - M]))
    assert torch.equal(o[0, :-1], clean[0, :-1]) and o[0, -1].isnan().all()


# ------------------------------------------------------------------- prompts

def check_prompt(q, k, v, window, sinks, pos=None, counts=None, scale=None, some=None, **kw):
    """Against the definition, all rows or every `some`-th and the last ones."""
    B, M = q.shape[:2]
    T, D = k.shape[1], q.shape[3]
    o, err = moe.window_attention(q, k, v, window, sinks=sinks, pos=None if pos is None else i32(pos),
                                  counts=None if counts is None else i32(counts), scale=scale, **kw)
    assert err_of(err) == 0 and o.is_contiguous()
    p = [T - M] * B if pos is None else pos
    for b in range(B):
        n = 0 if p[b] < 0 else M if counts is None else counts[b]
        assert not o[b, n:].any()
        for m in [m for m in range(n) if some is None or m % some == 0 or m > n - 4]:
            t = kv_ref.seen(p[b] + m, window, sinks).to(DEV)
            want, tol = kv_ref.row(q[b, m], k[b, t], v[b, t], D ** -0.5 if scale is None else scale)
            kv_ref.close(o[b, m], want, tol, f"row {b}, {m}")
    return o


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D,Hq,G", [(64, 4, 2), (64, 10, 2), (128, 32, 8), (128, 5, 1), (256, 16, 2), (256, 3, 1), (64, 64, 1), (256, 64, 1)])
def test_prompts(dtype, D, Hq, G):
    """Prompts of unequal length behind NaN padding, with a window and first positions."""
    r, M = gen(20), 333
    counts = [333, 1, 128, 0, 257]
    q, k, v = rows(r, 5, M, Hq, D, dtype=dtype, size=1.3), rows(r, 5, M, G, D, dtype=dtype), rows(r, 5, M, G, D, dtype=dtype)
    for b, c in enumerate(counts):
        q[b, c:], k[b, c:], v[b, c:] = float("nan"), float("nan"), float("nan")
    check_prompt(q, k, v, 100, 3, pos=[0] * 5, counts=counts, some=7)
    check_prompt(q, k, v, None, 0, pos=[0, 0, -1, 0, 0], counts=counts, some=11)


@pytest.mark.parametrize("M", [1, 2, 3, 15, 16, 17, 31, 32, 33, 64, 65, 127, 128, 129, 256, 257, 600])
@pytest.mark.parametrize("D,Hq", [(64, 2), (128, 4), (256, 8)])
def test_prompt_lengths(M, D, Hq):
    r = gen(21)
    k, v = rows(r, 1, M + 70, 1, D), rows(r, 1, M + 70, 1, D)
    q = rows(r, 1, M, Hq, D)
    check_prompt(q, k, v, 90, 2, some=13)                      # behind 70 earlier positions
    check_prompt(q, k[:, :M], v[:, :M], None, 0, some=13)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 0), (64, 0), (127, 0), (128, 0), (129, 128), (200, 129), (5, 400), (3000, 0), (600, 7),
                                          (1 << 30, 5)])
@pytest.mark.parametrize("D,Hq", [(64, 4), (256, 8)])
def test_prompt_windows(window, sinks, D, Hq):
    r, M = gen(22), 700
    q, k, v = rows(r, 1, M, Hq, D, size=2.0), rows(r, 1, M, 1, D), rows(r, 1, M, 1, D)
    check_prompt(q, k, v, window, sinks, some=23)


@pytest.mark.parametrize("window,sinks", [(100, 1), (100, 63), (100, 64), (129, 65), (65, 128), (64, 129), (300, 200), (1, 500)])
@pytest.mark.parametrize("D,Hq,M", [(64, 4, 200), (128, 4, 200), (128, 3, 90), (256, 8, 150), (64, 2, 70)])
def test_window_far_from_the_first_positions(window, sinks, D, Hq, M):
    """Tiles of which one half has first positions and the other the window's."""
    r, T = gen(60), 1150
    q, k, v = rows(r, 2, M, Hq, D, size=2.0), rows(r, 2, T, 1, D), rows(r, 2, T, 1, D)
    pos = [T - M, 733]
    k[1, 733 + M:], v[1, 733 + M:] = float("nan"), float("nan")
    check_prompt(q, k, v, window, sinks, pos=pos, some=19)


@pytest.mark.parametrize("Hq,G", [(8, 8), (24, 8)])
@pytest.mark.parametrize("B", [1, 6, 10])
def test_prompt_turns(B, Hq, G):
    """As many pairs of row tiles as leave the last turn full, nearly empty, or with nothing else."""
    r, M, D = gen(61), 300, 128
    counts = [300, 0, 1, 128, 129, 256, 257, 299, 300, 127][:B]
    q, k, v = rows(r, B, M, Hq, D), rows(r, B, M, G, D), rows(r, B, M, G, D)
    for b, c in enumerate(counts):
        k[b, c:], v[b, c:] = float("nan"), float("nan")
    check_prompt(q, k, v, 70, 3, pos=[0] * B, counts=counts, some=29)
    check_prompt(q, k, v, None, 0, pos=[0] * B, counts=counts, some=37)


@pytest.mark.parametrize("D,Hq,G", [(64, 16, 8), (128, 16, 8), (256, 16, 8)])
def test_many_short_items(D, Hq, G):
    """A window of 1: every row is its own value, and what a CTA does for 128 rows is as short as it gets, so that its
    warps run as far ahead of each other as they can."""
    r, B, M = gen(63), 6, 1500
    q, k, v = rows(r, B, M, Hq, D), rows(r, B, M, G, D), rows(r, B, M, G, D)
    pos = i32([0, 500, 0, -1, 3, 0])
    for n in range(40):
        counts = [(257 * n + 311 * b) % (M - 500) for b in range(B)]
        o, err = moe.window_attention(q, k, v, 1, pos=pos, counts=i32(counts))
        assert err_of(err) == 0
        for b, (p, c) in enumerate(zip((0, 500, 0, -1, 3, 0), counts)):
            c = c if p >= 0 else 0
            assert torch.equal(o[b, :c], v[b, max(p, 0):max(p, 0) + c].repeat_interleave(Hq // G, 1)) and not o[b, c:].any()


@pytest.mark.parametrize("D,Hq,G,M", [(64, 32, 8, 250), (128, 32, 8, 250), (256, 16, 2, 300), (64, 30, 6, 200), (128, 6, 2, 900)])
def test_prompt_rows_in_parts(D, Hq, G, M):
    """Many rows whose positions are cut into parts, some of them empty."""
    r, T, B = gen(62), 5000, 2
    q, k, v = rows(r, B, M, Hq, D, size=1.5), rows(r, B, T, G, D), rows(r, B, T, G, D)
    assert moe.window_attention_workspace(B, Hq, G, D, M, T) > 0
    pos, counts = [T - M, 90], [M, M - 5]
    k[1, 90 + M - 5:], v[1, 90 + M - 5:] = float("nan"), float("nan")
    check_prompt(q, k, v, None, 0, pos=pos, counts=counts, some=41)


def test_prompt_views_and_pieces():
    """q, k and v as views of one projection; the prompt in pieces gives what
    it gives at once, up to rounding; sequences at places of their own."""
    r, B, T, Hq, G, D = gen(23), 2, 500, 8, 2, 128
    x = rows(r, B, T, (Hq + 2 * G) * D)
    q = x[..., :Hq * D].unflatten(2, (Hq, D))
    k, v = x[..., Hq * D:(Hq + G) * D].unflatten(2, (G, D)), x[..., (Hq + G) * D:].unflatten(2, (G, D))
    check_prompt(q, k, v, 120, 4, some=9)
    check_prompt(q[:, 300:433], k, v, 120, 4, pos=[300, 300], some=9)
    check_prompt(q[:, :77], k, v, 120, 4, pos=[13, 400], counts=[77, 50], some=9, scale=0.3)
    qt = q.transpose(1, 2).contiguous().transpose(1, 2)        # heads outside
    kt, vt = k.transpose(1, 2).contiguous().transpose(1, 2), v.transpose(1, 2).contiguous().transpose(1, 2)
    a, b = check_prompt(qt, kt, vt, 120, 4, some=50), moe.window_attention(q, k, v, 120, sinks=4)[0]
    assert torch.equal(a, b)
    one = q[:1, :1].expand(1, 200, Hq, D)                      # strides of 0 in q
    check_prompt(one, k[:1], v[:1], 50, 1, some=21)
    with pytest.raises(moe.MoeError):                          # and none in k, v
        moe.window_attention(q, k[:, :1].expand(B, T, G, D), v, 50)


@pytest.mark.parametrize("D,Hq", [(64, 8), (128, 8), (256, 8)])
def test_prompt_rising_scores(D, Hq):
    r, M = gen(24), 800
    q, k, v = rows(r, 1, M, Hq, D), rows(r, 1, M, 1, D), rows(r, 1, M, 1, D)
    q[..., 0] = 2.0
    ramp = torch.cat([torch.linspace(-60, 90, 500), torch.linspace(90, -200, 300)]).to(DEV)
    k[0, :, :, 0] = (ramp * D ** 0.5 / 2).to(BF)[:, None]
    check_prompt(q, k, v, None, 0, some=17)
    check_prompt(q, k * 12, v, 150, 3, some=17)


@pytest.mark.parametrize("D,Hq,G", [(128, 8, 2), (256, 16, 2)])
def test_long_prompt(D, Hq, G):
    r, M = gen(25), 9001
    q, k, v = rows(r, 1, M, Hq, D), rows(r, 1, M, G, D), rows(r, 1, M, G, D)
    check_prompt(q, k, v, 4096, 4, some=907)
    check_prompt(q, k, v, None, 0, some=1501)


def test_few_rows_far_behind():
    """Positions cut into parts: few rows behind many positions."""
    r, T = gen(26), 20000
    for D, Hq, M in ((128, 8, 3), (128, 8, 40), (256, 16, 9), (64, 4, 300)):
        q, k, v = rows(r, 1, M, Hq, D), rows(r, 1, T, 1, D), rows(r, 1, T, 1, D)
        check_prompt(q, k, v, None, 0, some=19)
        check_prompt(q, k, v, 12345, 130, some=19)


# -------------------------------------------------------------------- prefix

@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D,Hq,G,B,M", [(64, 4, 2, 3, 1), (128, 8, 2, 4, 1), (256, 16, 2, 4, 1), (128, 32, 8, 9, 1), (256, 16, 2, 9, 3),
                                        (64, 10, 1, 5, 2), (64, 8, 8, 40, 1), (128, 4, 1, 70, 1), (256, 8, 1, 3, 8), (64, 64, 1, 5, 1)])
def test_shared_prefix(dtype, D, Hq, G, B, M):
    """Prefixes of one position to many, sequences without positions of their own before the call, idle ones, padding."""
    r, T = gen(27), 200
    lens = [M + (37 * b) % (T - M) for b in range(B)]
    cache, k, v = filled(r, T, lens, G, D, dtype, Hq=Hq, max_prefix=1300)
    q = rows(r, B, M, Hq, D, dtype=dtype, size=1.3)
    pos = [n - M for n in lens]
    counts = [M] * B
    if B > 3:
        pos[2], counts[1] = -1, M - 1
    for n in (1, 63, 64, 65, 128, 129, 1300):
        pk, pv = rows(r, n, G, D, dtype=dtype), rows(r, n, G, D, dtype=dtype, size=2.0)
        check_cache(cache, k, v, q, pos, counts=counts, prefix=(pk, pv))


def test_prefix_views():
    """A prefix as it lies in a projection or in another cache, q of a wider projection."""
    r, B, M, Hq, G, D = gen(28), 6, 2, 16, 2, 128
    lens = [20, 3, 2, 77, 9, 40]
    cache, k, v = filled(r, 100, lens, G, D, BF, Hq=Hq, max_prefix=2000)
    x = rows(r, 1500, 2 * G * D + 16)
    pre = (x[:, :G * D].unflatten(1, (G, D)), x[:, G * D:2 * G * D].unflatten(1, (G, D)))
    q = rows(r, B, M, (Hq + 1) * D)[..., :Hq * D].unflatten(2, (Hq, D))
    pos = [n - M for n in lens]
    a = check_cache(cache, k, v, q, pos, prefix=pre)
    other = moe.KVCache(1500, q_heads=G, kv_heads=G, head_dim=D)
    other.append(pre[0][None], pre[1][None], i32([0]))
    lies = (other.k[0].transpose(0, 1), other.v[0].transpose(0, 1))
    b, _ = cache.attend(q, i32(pos), prefix=lies)
    assert torch.equal(a, b)
    t = q.transpose(0, 1).contiguous().transpose(0, 1)         # rows outside the batch
    b, _ = cache.attend(t, i32(pos), prefix=lies)
    assert torch.equal(a, b)


def test_prefix_is_like_one_long_sequence():
    """The prefix and a sequence's own positions in one cache give the same, up to rounding (two roundings of weights and outputs)."""
    r, B, Hq, G, D, P = gen(29), 20, 16, 2, 256, 700
    cache, k, v = filled(r, 60, [50] * B, G, D, BF, Hq=Hq, max_prefix=P)
    pk, pv = rows(r, P, G, D), rows(r, P, G, D)
    q = rows(r, B, 1, Hq, D)
    a, _ = cache.attend(q, i32([49] * B), prefix=(pk, pv))
    whole = moe.KVCache(P + 60, batch=B, q_heads=Hq, kv_heads=G, head_dim=D)
    whole.append(pk.expand(B, P, G, D), pv.expand(B, P, G, D), i32([0] * B))
    whole.append(k, v, i32([P] * B))
    b, _ = whole.attend(q, i32([P + 49] * B))
    for i in range(B):
        _, tol = kv_ref.row(q[i, 0], torch.cat([pk, k[i, :50]]), torch.cat([pv, v[i, :50]]), D ** -0.5)
        kv_ref.close(a[i, 0], b[i, 0].double(), 2 * tol, f"sequence {i}")


# ------------------------------------------------------------- ways to call

def test_same_bits_again():
    for Hq, M in ((8, 1), (16, 8)):
        cache, k, v = filled(gen(30), 3000, [2999, 1500, 7, 2000], 2, 128, BF, Hq=Hq, max_prefix=999)
        q = rows(gen(31), 4, M, Hq, 128)
        pos, pre = i32([2999 - M, 1400, -1, 900]), (k[0, :999], v[0, :999])
        a, b = cache.attend(q, pos)[0], cache.attend(q, pos, prefix=pre)[0]
        for _ in range(5):
            assert torch.equal(cache.attend(q, pos)[0], a) and torch.equal(cache.attend(q, pos, prefix=pre)[0], b)
    q, k, v = (rows(gen(32), 2, 900, h, 128) for h in (8, 2, 2))
    a = moe.window_attention(q, k, v, 300, sinks=4)[0]
    for _ in range(5):
        assert torch.equal(moe.window_attention(q, k, v, 300, sinks=4)[0], a)


def test_out_and_scratch_are_the_callers():
    r = gen(33)
    cache, k, v = filled(r, 100, [90], 2, 64, BF, Hq=4)
    q = rows(r, 1, 3, 4, 64)
    out, err = torch.full((1, 3, 4, 64), 9.0, dtype=BF, device=DEV), i32([0])
    o, e = cache.attend(q, i32([87]), out=out, err=err)
    assert o is out and e is err and torch.equal(out, cache.attend(q, i32([87]))[0])
    shared = moe.KVCache(100, q_heads=4, kv_heads=2, head_dim=64, buffers=(cache.k, cache.v), ws=cache.ws)
    assert torch.equal(shared.attend(q, i32([87]))[0], out)
    q, k = rows(r, 1, 40, 4, 64), rows(r, 1, 5000, 2, 64)
    n = moe.window_attention_workspace(1, 4, 2, 64, 40, 5000)
    assert n > 0
    ws, out = torch.full((n,), 255, dtype=torch.uint8, device=DEV), torch.empty_like(q)
    o, _ = moe.window_attention(q, k, k, out=out, ws=ws)
    assert o is out and torch.equal(out, moe.window_attention(q, k, k)[0])
    with pytest.raises(moe.MoeError):
        moe.window_attention(q, k, k, ws=ws[:n - 1].clone())


def test_captured_and_replayed():
    """A decode step captured once is replayed with other lengths; two graphs over one scratch, one after the other."""
    r, B, W, S, T = gen(34), 3, 50, 2, 80
    for Hq, M in ((8, 1), (32, 4)):
        cache = moe.KVCache(T, batch=B, q_heads=Hq, kv_heads=2, head_dim=128, window=W, sinks=S, max_rows=M)
        total = 200
        k, v, q = rows(r, B, total, 2, 128), rows(r, B, total, 2, 128), rows(r, B, total, Hq, 128)
        kn, vn, qn, pos = k[:, :M].clone(), v[:, :M].clone(), q[:, :M].clone(), i32([0] * B)
        cache.append(kn, vn, pos)
        cache.attend(qn, pos)
        torch.cuda.synchronize()
        graph, plain = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cache.append(kn, vn, pos)
            o, _ = cache.attend(qn, pos)
            pos += M
        prompt = rows(r, 1, 300, 8, 64)
        pk = rows(r, 1, 300, 1, 64)
        with torch.cuda.graph(plain):
            po, _ = moe.window_attention(prompt, pk, pk, 100)
        for t in range(0, total, M):
            kn.copy_(k[:, t:t + M]), vn.copy_(v[:, t:t + M]), qn.copy_(q[:, t:t + M])
            graph.replay()
            if t % 52 == 0 or t >= total - M:
                for b in range(B):
                    for m in range(M):
                        s = kv_ref.seen(t + m, W, S).to(DEV)
                        want, tol = kv_ref.row(q[b, t + m], k[b, s], v[b, s], 128 ** -0.5)
                        kv_ref.close(o[b, m], want, tol, f"step {t}, row {b}, {m}")
        plain.replay()
        assert torch.equal(po, moe.window_attention(prompt, pk, pk, 100)[0])
        assert err_of(cache.err) == 0


def test_other_streams():
    """Calls on an explicit stream, and on a current stream that is not the one that made the cache."""
    r = gen(35)
    cache, k, v = filled(r, 3000, [2500, 100], 2, 256, BF, Hq=16, max_prefix=500)
    q, pos, pre = rows(r, 2, 1, 16, 256), i32([2499, 99]), (k[0, :500], v[0, :500])
    want, more = cache.attend(q, pos)[0], cache.attend(q, pos, prefix=pre)[0]
    pq, pk = rows(r, 1, 400, 8, 128), rows(r, 1, 400, 2, 128)
    prompt = moe.window_attention(pq, pk, pk, 77)[0]
    side = torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        a, _ = cache.attend(q.clone(), pos.clone(), stream=side)
        b, _ = cache.attend(q, pos, prefix=pre, stream=side)
        c, _ = moe.window_attention(pq.clone(), pk, pk, 77, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(a, want) and torch.equal(b, more) and torch.equal(c, prompt)
        with torch.cuda.stream(side):
            a, c = cache.attend(q, pos)[0], moe.window_attention(pq, pk, pk, 77)[0]
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(a, want) and torch.equal(c, prompt)


def test_two_calls_at_once():
    """Caches with scratch of their own on two streams."""
    r = gen(36)
    made = [filled(r, 4000, [4000, 3000], 2, 128, BF, Hq=16, max_rows=4) for _ in range(2)]
    qs = [rows(r, 2, m, 16, 128) for m in (1, 4)]
    pos = i32([3990, 2000])
    want = [[c.attend(q, pos)[0] for q in qs] for c, _, _ in made]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append([made[i][0].attend(q, pos, stream=s)[0] for q in qs])
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def test_offsets_past_31_bits():
    """The last sequence of a cache of more than 2^31 elements, and of keys and values as long."""
    r, B, G, D, T = gen(37), 3, 8, 256, 400000
    buf = [torch.empty((B, G, T, D), dtype=BF, device=DEV) for _ in range(2)]
    for t in buf:
        t.zero_()
    cache = moe.KVCache(T, batch=B, q_heads=32, kv_heads=G, head_dim=D, buffers=tuple(buf))
    k, v = rows(r, B, 300, G, D), rows(r, B, 300, G, D)
    for M in (1, 8):
        q, at = rows(r, B, M, 32, D), T - 300
        cache.append(k, v, i32([-1, -1, at]))
        o, err = cache.attend(q, i32([-1, -1, T - M]))
        assert err_of(err) == 0 and not o[:2].any()
        for m in range(M):
            n = T - M + m + 1
            want, tol = kv_ref.row(q[2, m], buf[0][2, :, :n].transpose(0, 1), buf[1][2, :, :n].transpose(0, 1), D ** -0.5)
            kv_ref.close(o[2, m], want, tol, f"{M} rows, {m}")
            break
    x = buf[0].view(B, T, G, D)[:, :, :, :]                    # as prompts: [B, T, G, D]
    q = rows(r, B, 20, 16, D)
    x[2, T - 200:] = rows(r, 200, G, D)
    o, _ = moe.window_attention(q, x, x, 90, sinks=1)
    for m in (0, 19):
        t = kv_ref.seen(T - 20 + m, 90, 1).to(DEV)
        want, tol = kv_ref.row(q[2, m], x[2, t], x[2, t], D ** -0.5)
        kv_ref.close(o[2, m], want, tol, f"prompt row {m}")


# --------------------------------------------------------- a run of them all

@pytest.mark.parametrize("M", [1, 4])
def test_prompt_then_tokens(M):
    """A ragged batch of prompts through window_attention and into the ring, then decode steps with
    drafts, some rejected, as a serving loop makes them."""
    r, B, Hq, G, D, W, S = gen(38), 3, 16, 2, 128, 64, 4
    total, plen = 300, [150, 40, 1]
    k, v, q = rows(r, B, total, G, D), rows(r, B, total, G, D), rows(r, B, total, Hq, D)
    cache = moe.KVCache(S + W + M - 1, batch=B, q_heads=Hq, kv_heads=G, head_dim=D, window=W, sinks=S, max_rows=M)
    n = max(plen)
    check_prompt(q[:, :n], k[:, :n], v[:, :n], W, S, pos=[0] * B, counts=plen, some=29)
    cache.append(k[:, :n], v[:, :n], i32([0] * B), counts=i32(plen))
    pos = list(plen)
    for step in range(30):
        at = [torch.arange(p, p + M, device=DEV) for p in pos]
        kn, vn = (torch.stack([x[b, at[b]] for b in range(B)]) for x in (k, v))
        if M > 1 and step % 3 == 1:                            # drafts that will be rejected: other keys and values first
            cache.append(kn + 1, vn - 1, i32(pos))
        cache.append(kn, vn, i32(pos))
        qn = torch.stack([q[b, at[b]] for b in range(B)])
        check_cache(cache, k, v, qn, pos)
        pos = [p + (M if step % 3 else 1) for p in pos]


def test_document_then_questions():
    """A document's prompt, once; many questions behind it as a shared prefix, decoded step by step."""
    r, B, Hq, G, D, P = gen(39), 12, 16, 2, 256, 513
    dk, dv, dq = rows(r, 1, P, G, D), rows(r, 1, P, G, D), rows(r, 1, P, Hq, D)
    check_prompt(dq, dk, dv, None, 0, some=111)
    cache = moe.KVCache(32, batch=B, q_heads=Hq, kv_heads=G, head_dim=D, max_prefix=P)
    k, v, q = rows(r, B, 24, G, D), rows(r, B, 24, G, D), rows(r, B, 24, Hq, D)
    pos = 0
    for M in (5, 1, 1, 8, 1):
        cache.append(k[:, pos:pos + M], v[:, pos:pos + M], i32([pos] * B))
        check_cache(cache, k, v, q[:, pos:pos + M], [pos] * B, prefix=(dk[0], dv[0]))
        pos += M


# ------------------------------------------------------------ ends of ranges

@pytest.mark.parametrize("D,M", [(64, 1), (256, 1), (128, 9)])
def test_many_heads(D, M):
    """More key/value heads than a block's threads, one query head each."""
    r, G = gen(40), 300
    q, k, v = rows(r, 1, M, G, D), rows(r, 1, 200, G, D), rows(r, 1, 200, G, D)
    check_prompt(q, k, v, 100, 2)
    if M == 1:
        cache = moe.KVCache(210, q_heads=G, kv_heads=G, head_dim=D)
        cache.append(k, v, i32([0]))
        check_cache(cache, k, v, q, [199])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_largest_batch(D):
    """1024 sequences, of 0 to 70 positions; with a prefix too."""
    B, T = 1024, 70
    lens = [(31 * b) % 71 for b in range(B)]
    cache, k, v = filled(gen(41), T, lens, 1, D, FP, Hq=2, max_rows=1, max_prefix=100)
    q = rows(gen(42), B, 1, 2, D, dtype=FP)
    pos = [n - 1 for n in lens]
    pk = rows(gen(43), 100, 1, D, dtype=FP)
    for prefix in (None, (pk, pk)):
        o, err = cache.attend(q, i32(pos), prefix=prefix)
        assert err_of(err) == 0
        for b in list(range(0, B, 61)) + [1022, 1023]:
            if pos[b] < 0:
                assert not o[b].any()
                continue
            own = [k[b, :pos[b] + 1], v[b, :pos[b] + 1]]
            if prefix:
                own = [torch.cat([pk, x]) for x in own]
            want, tol = kv_ref.row(q[b, 0], *own, D ** -0.5)
            kv_ref.close(o[b, 0], want, tol, f"sequence {b}")
    with pytest.raises(moe.MoeError):
        moe.KVCache(T, batch=1025, kv_heads=1, q_heads=2, head_dim=64)


def test_far_positions_in_a_ring():
    """Positions up to the last that a ring may have; the one behind it is refused."""
    W, S, T = 30, 3, 48
    for Hq, M in ((4, 1), (32, 4)):
        for p in ((1 << 30) - M, 123456789):
            r = gen(44)
            cache = moe.KVCache(T, q_heads=Hq, kv_heads=2, head_dim=64, window=W, sinks=S, max_rows=M)
            k, v = rows(r, 1, S + W + M, 2, 64), rows(r, 1, S + W + M, 2, 64)
            cache.append(k[:, :S], v[:, :S], i32([0]))
            cache.append(k[:, S:], v[:, S:], i32([p - W]))
            q = rows(r, 1, M, Hq, 64)
            o, err = cache.attend(q, i32([p]))
            assert err_of(err) == 0
            for m in range(M):
                sees = list(range(S)) + list(range(S + 1 + m, S + W + 1 + m))
                want, tol = kv_ref.row(q[0, m], k[0, sees], v[0, sees], 0.125)
                kv_ref.close(o[0, m], want, tol, f"row {m} at {p}")
        o, err = cache.attend(q, i32([(1 << 30) - M + 1]))
        assert err_of(err) == 1 and not o[0, -1].any()


def test_first_call_in_a_capture():
    """A prompt's call whose device has had none before is captured: its error word is the graph's."""
    from quantized_moe_decode_layer_gb300 import api
    x = rows(gen(45), 1, 90, 2, 64)
    want = moe.window_attention(x, x, x, 20)[0]
    torch.cuda.synchronize()
    kept = dict(api._window_err)
    api._window_err.clear()
    try:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o, err = moe.window_attention(x, x, x, 20)
        assert not api._window_err
        graph.replay()
        assert torch.equal(o, want) and int(err.item()) == 0
    finally:
        api._window_err.update(kept)


@pytest.mark.parametrize("D,Hq,G", [(64, 8, 4), (128, 8, 4), (256, 8, 4)])
def test_waits_that_run_out(D, Hq, G):
    """With a time limit that no wait keeps the calls return, report it and leave the device usable."""
    q, k = rows(gen(46), 2, 700, Hq, D), rows(gen(47), 2, 700, G, D)
    want = moe.window_attention(q, k, k, 300, sinks=2)[0]
    cache = moe.KVCache(64, batch=2, q_heads=8 * G, kv_heads=G, head_dim=D, max_prefix=700)
    cache.append(k[:, :60], k[:, :60], i32([0, 0]))
    few = rows(gen(48), 2, 4, 8 * G, D)
    also = cache.attend(few, i32([56, 56]), prefix=(k[0], k[0]))[0]
    torch.cuda.synchronize()
    try:
        moe.debug_set(-1, timeout_ns=1)
        _, err = moe.window_attention(q, k, k, 300, sinks=2)
        assert err_of(err) == 4
        _, err = cache.attend(few, i32([56, 56]), prefix=(k[0], k[0]))
        assert err_of(err) == moe.KVCache.ERR_TIMEOUT
    finally:
        moe.debug_set(-1, 0)
    o, err = moe.window_attention(q, k, k, 300, sinks=2)
    assert err_of(err) == 0 and torch.equal(o, want)
    o, err = cache.attend(few, i32([56, 56]), prefix=(k[0], k[0]))
    assert err_of(err) == 0 and torch.equal(o, also)
