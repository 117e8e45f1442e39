"""GPU tests of the 16-bit key/value cache and of attention over prompts at the
limits of their numbers and of what a cache may hold."""
import pytest
import torch

import kv_ref
import quantized_moe_decode_layer_gb300 as moe
from test_gpu_kv import BF, DEV, FP, err_of, gen, i32, rows

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- scores

@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("tokens", [False, True])
def test_scores_one_spacing_apart(dtype, D, tokens):
    """Two scores of 2^27, where fp32's neighbours are 16 apart: the larger ones' values.  (A weight of the others is 2^-16
    of theirs, in all 2^-16 of the sum.)  Batches of tokens and rows of a prompt so many that a CTA goes through both."""
    B, M, Hq, n, half = (300, 1, 1, 512, kv_ref.HALF[dtype]) if tokens else (1, 1300, 32, 2000, kv_ref.HALF[dtype])
    k, v = torch.zeros((B, n, 1, D), dtype=dtype, device=DEV), rows(gen(70), 1, n, 1, D, dtype=dtype).expand(B, n, 1, D).contiguous()
    k[..., 0] = 64.0
    k[:, 256:, 0, 1] = 1.0                               # q . k: 64 and its neighbour in fp32
    q = torch.zeros((B, M, Hq, D), dtype=dtype, device=DEV)
    q[..., 0], q[..., 1] = 1.0, 2.0 ** -17
    at = torch.arange(n - M + 1, n + 1, device=DEV)[:, None] - 256.0
    x = v[0, 256:, 0].double()
    want, size = x.cumsum(0)[-M:] / at, x.abs().cumsum(0)[-M:] / at
    tol = half * want.abs() + (half + (2 * n + 64) * kv_ref.E23) * size + 2.0 ** -16 * 2 * v.double().abs().max()
    for step in range(64):                               # half of them make the first score an odd multiple of 16
        scale = 2.0 ** 21 * 0.6931471805599453 * (1 + step * 2.0 ** -23)
        o, err = moe.window_attention(q, k, v, scale=scale)
        assert err_of(err) == 0
        kv_ref.close(o, want[None, :, None], tol[None, :, None], f"scale {step}")


def _sizes(D):
    """Scales that make scores of 2^0 to 2^40, with full mantissas."""
    return [1.2345 * 2.0 ** e * D ** -0.5 for e in (0, 5, 9, 10, 11, 13, 16, 19, 20, 21, 23, 24, 25, 26, 27, 28, 29, 30, 31, 32, 33, 36, 40)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_visible_position_at_any_score(dtype, D):
    """A window of 1: the output is the value, however large the score: as prompts, tokens, drafts."""
    r, n, G = gen(71), 300, 2
    q, k, v = rows(r, 1, n, 8, D, dtype=dtype), rows(r, 1, n, G, D, dtype=dtype), rows(r, 1, n, G, D, dtype=dtype)
    want = v.repeat_interleave(4, 2)
    caches = []
    for M, Hq in ((1, 2), (4, 8), (8, 8)):
        c = moe.KVCache(M + 20, q_heads=Hq, kv_heads=G, head_dim=D, dtype=dtype, window=1, max_rows=M)
        c.append(k, v, i32([0]))
        caches.append((c, M, Hq))
    for scale in _sizes(D):
        o, err = moe.window_attention(q, k, v, 1, scale=scale)
        assert err_of(err) == 0 and torch.equal(o, want), scale
        for c, M, Hq in caches:
            o, _ = c.attend(q[:, n - M:, ::8 // Hq].contiguous(), i32([n - M]), scale=scale)
            assert torch.equal(o, want[:, n - M:, ::8 // Hq]), (scale, M)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [2, 5, 150])
def test_few_visible_positions_at_any_score(dtype, D, window):
    """A mean of the visible values; and where one score is above all others by more than all errors, its value.  (A weight
    and the output are rounded: half a step each.)"""
    r, n, half = gen(72), 300, kv_ref.HALF[dtype]
    q, k, v = rows(r, 1, n, 4, D, dtype=dtype), rows(r, 1, n, 1, D, dtype=dtype), rows(r, 1, n, 1, D, dtype=dtype)
    at = torch.arange(n, device=DEV)
    sees = (at[None] <= at[:, None]) & (at[None] > at[:, None] - window)
    vd = v[0, :, 0].double()
    low = torch.stack([vd[max(0, p - window + 1):p + 1].amin(0) for p in range(n)])[:, None]
    high = torch.stack([vd[max(0, p - window + 1):p + 1].amax(0) for p in range(n)])[:, None]
    edge = 2.01 * half * torch.maximum(low.abs(), high.abs()) + 2.0 ** -24
    z1 = torch.einsum("mhd,td->mht", q[0].double(), k[0, :, 0].double())
    a1 = torch.einsum("mhd,td->mht", q[0].double().abs(), k[0, :, 0].double().abs())
    for scale in _sizes(D):
        z = (z1 * scale).masked_fill(~sees[:, None], -1e300)
        top = z.topk(2, -1)
        err = 2 * (D + 6) * kv_ref.E23 * (a1 * scale).masked_fill(~sees[:, None], 0).amax(-1)
        clear = top.values[..., 0] - top.values[..., 1] > err + 40
        o, e = moe.window_attention(q, k, v, window, scale=scale)
        assert err_of(e) == 0
        o = o[0].double()
        assert bool(((o >= low - edge) & (o <= high + edge)).all()), scale
        best = vd[top.indices[..., 0]]
        assert scale < 2 ** 9 or bool(clear.any())
        assert bool(((o - best).abs() <= 2.01 * half * best.abs() + 2.0 ** -24)[clear].all()), scale


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("low", [17.375, 20.25, 24.0, 25.125, 28.0])
def test_many_small_weights_in_fp16(D, low):
    """A strong first position whose values are 0 before 131071 whose weights are 2^-low of its own: rows enough that they are
    not cut into many parts, and single tokens.  A weight below 2^-21 of the reference is off by 2^-32 of it (a weight of 1 is 2^7
    in fp16, whose smallest step is 2^-24); the largest weight is at least the reference."""
    n, half, r = 1 << 17, kv_ref.HALF[FP], gen(73)
    k, v = torch.zeros((1, n, 1, D), dtype=FP, device=DEV), rows(r, 1, n, 1, D, dtype=FP).abs() + 0.5
    k[0, 0, 0, 0], v[0, 0] = low, 0.0
    scale, w = 0.6931471805599453, 2.0 ** -low                            # scores in units of log2

    def check(got, seen, what):
        x = v[0, :seen, 0].double()
        want = w * x.sum(0) / (1 + w * (seen - 1))
        tol = ((2 * half + 2 * (D + 6) * kv_ref.E23 * low + 2.0 ** -21 + (2 * n + 64) * kv_ref.E23) * want + n * 2.0 ** -32 * x.max() +
               2.0 ** -25)
        kv_ref.close(got, want, tol, what)
    for M, Hq in ((1300, 32), (1, 1), (1, 32)):
        q = torch.zeros((1, M, Hq, D), dtype=FP, device=DEV)
        q[..., 0] = 1.0
        o, err = moe.window_attention(q, k, v, scale=scale)
        assert err_of(err) == 0
        for m in sorted({0, M // 2, M - 1}):
            check(o[0, m], n - M + m + 1, f"weights of 2^-{low}, row {m} of {M}")


# -------------------------------------------------------------- what is past

@pytest.mark.parametrize("D,Hq,M", [(64, 4, 8), (128, 4, 8), (128, 3, 6), (256, 16, 2), (256, 8, 8), (64, 64, 8), (128, 64, 8), (64, 2, 4)])
@pytest.mark.parametrize("W,S,extra", [(100, 4, 3), (64, 0, 4), (57, 70, 3), (7, 3, 50), (200, 1, 120), (1, 0, 3)])
def test_rejected_rows_in_a_full_ring(D, Hq, M, W, S, extra):
    """Drafts behind a sequence's end, some way around the ring: their keys and values are NaN and infinity,
    after padding, after all rows were rejected, and after a step back of three more."""
    T = S + W + M - 1 + extra
    ends = sorted({T - M, T - 1, T, T + 1, T + 9, 2 * T - S - M, 2 * T - S - 1, 2 * T - S, 2 * T - S + 3, T + 61, T + 64, T + 67, 3 * T + 17})
    B, n = len(ends), max(ends) + M + 1
    r = gen(74)
    k, v, q = rows(r, B, n, 1, D), rows(r, B, n, 1, D), rows(r, B, M, Hq, D, size=1.5)
    cache = moe.KVCache(T, batch=B, q_heads=Hq, kv_heads=1, head_dim=D, window=W, sinks=S, max_rows=M)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    cache.append(k, v, i32([0] * B), counts=i32(ends))
    bad = torch.full((B, M, 1, D), float("nan"), dtype=BF, device=DEV)
    bad[:, ::2] = float("inf")
    cache.append(bad, bad, i32(ends))
    for back, counts in ((0, [1 + b % M for b in range(B)]), (0, [1] * B), (3, [1 + b % 2 for b in range(B)])):
        pos = [max(e - back, 0) for e in ends]
        at = torch.tensor(pos, device=DEV)[:, None] + torch.arange(M, device=DEV)
        b = torch.arange(B, device=DEV)[:, None]
        cache.append(bad, bad, i32(pos))
        cache.append(k[b, at], v[b, at], i32(pos), counts=i32(counts))
        o, err = cache.attend(q, i32(pos), counts=i32(counts))
        assert err_of(err) == 0

        def of(x):
            return lambda b, m: x[b, kv_ref.seen(pos[b] + m, W, S).to(DEV)]
        kv_ref.check_rows(o, q, of(k), of(v), lambda b, m: m < counts[b], D ** -0.5)


@pytest.mark.parametrize("D,Hq", [(64, 64), (128, 64), (256, 64), (256, 8)])
@pytest.mark.parametrize("W,S,extra", [(128, 130, 1), (300, 300, 1), (600, 4, 60), (1000, 130, 9)])
def test_rejected_rows_in_any_tile(D, Hq, W, S, extra):
    """Rejected rows in tiles that others follow, many times over: values of the tiles before and behind stay as they are."""
    M, B = 4, 40
    T = S + W + M - 1 + extra
    r = gen(85)
    ends = [T + 3 + (37 * b) % (2 * T) for b in range(B)]
    n = max(ends)
    k, v, q = rows(r, B, n, 1, D), rows(r, B, n, 1, D), rows(r, B, M, Hq, D)
    cache = moe.KVCache(T, batch=B, q_heads=Hq, kv_heads=1, head_dim=D, window=W, sinks=S, max_rows=M)
    cache.append(k, v, i32([0] * B), counts=i32(ends))
    bad = torch.full((B, M, 1, D), float("nan"), dtype=BF, device=DEV)
    cache.append(bad, bad, i32(ends), counts=i32([min(M, extra)] * B))
    pos = [e - M for e in ends]
    want = None
    for _ in range(30):
        o, err = cache.attend(q, i32(pos))
        assert err_of(err) == 0
        want = o if want is None else want
        assert torch.equal(o, want)
    for b in range(0, B, 5):
        sees = _sees(pos[b], M, ends[b], W, S)
        kv_ref.close(o[b], *_definition(q[b], k[b, :ends[b]], v[b, :ends[b]], sees, D ** -0.5), f"sequence {b}")


# --------------------------------------------------------------------- waits

@pytest.mark.parametrize("D,Hq,G", [(64, 32, 8), (128, 32, 8), (256, 16, 2), (128, 24, 8), (64, 24, 8)])
def test_waits_that_run_out_among_many_items(D, Hq, G):
    """Limits at which waits give up in a CTA's first items, in later ones or not at all; with 128 columns the last turn's items
    are cut in two, with groups of three outputs go without boxes, few rows leave parts.  A call returns and reports it, or is right;
    the device stays usable."""
    q, k = rows(gen(75), 2, 2048, Hq, D), rows(gen(76), 2, 2048, G, D)
    few = rows(gen(77), 2, 40, Hq, D)
    counts = i32([2048, 700])
    calls = [lambda: moe.window_attention(q, k, k, 40, sinks=2), lambda: moe.window_attention(q, k, k, pos=i32([0, 0]), counts=counts),
             lambda: moe.window_attention(few, k, k)]
    want = [f()[0] for f in calls]
    torch.cuda.synchronize()
    errs = set()
    try:
        for ns in (1, 200, 1000, 3000, 10000, 100000):
            moe.debug_set(-1, timeout_ns=ns)
            for f, w in zip(calls, want):
                o, err = f()
                e = err_of(err)
                errs.add(e)
                assert e in (0, 4) and (e or torch.equal(o, w))
    finally:
        moe.debug_set(-1, 0)
    assert 4 in errs
    for f, w in zip(calls, want):
        o, err = f()
        assert err_of(err) == 0 and torch.equal(o, w)


# ------------------------------------------------------------------ prefixes

@pytest.mark.parametrize("B", [2, 40])
def test_expanded_prefix(B):
    """One head's prefix for two, one position's for many: refused for any batch; a dimension of one entry may have any stride."""
    r = gen(78)
    cache = moe.KVCache(20, batch=B, q_heads=4, kv_heads=2, head_dim=64, max_prefix=50)
    q, x = rows(r, B, 1, 4, 64), rows(r, 50, 2, 64)
    k = rows(r, B, 1, 2, 64)
    cache.append(k, k, i32([0] * B))
    for bad in (x[:1].expand(50, 2, 64), x[:, :1].expand(50, 2, 64)):
        for prefix in ((bad, x), (x, bad)):
            with pytest.raises(moe.MoeError):
                cache.attend(q, i32([0] * B), prefix=prefix)
    one = x[:1].as_strided((1, 2, 64), (0, 64, 1))
    a, _ = cache.attend(q, i32([0] * B), prefix=(one, one))
    b, err = cache.attend(q, i32([0] * B), prefix=(x[:1], x[:1]))
    assert err_of(err) == 0 and torch.equal(a, b)


# ------------------------------------------------------------------- threads

def test_first_call_of_a_thread():
    """A thread that has made no CUDA call: prompts, rows over a cache, behind a prefix, and the one-sequence decode attention."""
    import threading
    x, k = rows(gen(80), 1, 90, 4, 64), rows(gen(81), 1, 90, 2, 64)
    cache = moe.KVCache(100, batch=1, q_heads=4, kv_heads=2, head_dim=64, max_prefix=90)
    cache.append(k, k, i32([0]))
    q, pos, err = rows(gen(82), 1, 8, 32, 64), i32([82]), i32([0])
    many = moe.KVCache(100, batch=1, q_heads=32, kv_heads=2, head_dim=64, max_prefix=90, buffers=(cache.k, cache.v))
    old = moe.AttnCache(64)
    oq, oout = rows(gen(83), 2, 16, 256), torch.empty((2, 16, 256), device=DEV)
    out, few = torch.empty_like(x), torch.empty_like(q)
    calls = [lambda: moe.window_attention(x, k, k, 20, out=out, err=err)[0], lambda: many.attend(q, pos, out=few, err=err)[0],
             lambda: many.attend(q, pos, prefix=(k[0], k[0]), out=few, err=err)[0], lambda: old.attend(oq, 3, out=oout, err=err)[0]]
    for f in calls:
        o = f()
        want, failed = o.clone(), []
        o.zero_()

        def work():
            try:
                f()
            except Exception as e:   # noqa: BLE001
                failed.append(e)
        t = threading.Thread(target=work)
        torch.cuda.synchronize()
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert not failed, failed
        assert torch.equal(o, want)
    assert err_of(err) == 0


# -------------------------------------------------------------- error words

def test_error_words_are_not_shared():
    """A call's error shows in no result of another thread, stream or graph; it stays until the caller clears it."""
    import threading
    x = rows(gen(79), 1, 90, 2, 64)
    good, bad = i32([0]), i32([1])                        # 90 rows from position 1 on: one too many

    def call(pos, **kw):
        return moe.window_attention(x, x, x, 20, pos=pos, **kw)[1]
    call(good)
    side, found = torch.cuda.Stream(), {}
    side.wait_stream(torch.cuda.current_stream())

    def work(name, pos, **kw):
        for _ in range(50):
            err = call(pos, **kw)
        torch.cuda.synchronize()
        found[name] = int(err)
    threads = [threading.Thread(target=work, args=("bad", bad)), threading.Thread(target=work, args=("good", good)),
               threading.Thread(target=work, args=("bad there", bad), kwargs=dict(stream=side)),
               threading.Thread(target=work, args=("good there", good), kwargs=dict(stream=side))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert found == {"bad": 1, "good": 0, "bad there": 1, "good there": 0}
    there = call(bad, stream=side)
    torch.cuda.synchronize()
    assert int(there) == 1 and int(call(good)) == 0
    with torch.cuda.stream(side):
        assert int(call(good)) == 1                       # this thread's word of that stream
        there.zero_()
        assert int(call(good)) == 0
    pos, graph = i32([1]), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        err = call(pos)
    graph.replay()
    assert int(err) == 1 and int(call(good)) == 0
    pos.zero_()
    graph.replay()
    assert int(err) == 0


def test_error_word_made_in_inference_mode():
    x, stream = rows(gen(79), 1, 90, 2, 64), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        with torch.inference_mode():
            moe.window_attention(x, x, x, 20, pos=i32([1]))
        _, err = moe.window_attention(x, x, x, 20)
        assert int(err) == 1
        err.zero_()


# ----------------------------------------------------------- the last rows

@pytest.mark.parametrize("M", [1, 8])
def test_all_rows_far_in_a_large_cache(M):
    """Every row of a call on the last sequence of a cache of more than 2^31 elements, in its first and last head."""
    r, B, G, D, T = gen(84), 3, 8, 256, 400000
    buf = [torch.zeros((B, G, T, D), dtype=BF, device=DEV) for _ in range(2)]
    cache = moe.KVCache(T, batch=B, q_heads=32, kv_heads=G, head_dim=D, buffers=tuple(buf))
    k, v, q = rows(r, B, 300, G, D), rows(r, B, 300, G, D), rows(r, B, M, 32, D)
    cache.append(k, v, i32([-1, -1, T - 300]))
    o, err = cache.attend(q, i32([-1, -1, T - M]))
    assert err_of(err) == 0 and not o[:2].any()
    for m in range(M):
        for g in (0, G - 1):
            h, n = slice(4 * g, 4 * g + 4), T - M + m + 1
            want, tol = kv_ref.row(q[2, m, h], buf[0][2, g, :n, None], buf[1][2, g, :n, None], D ** -0.5)
            kv_ref.close(o[2, m, h], want, tol, f"row {m}, head {g}")


# ------------------------------------------------------------ random shapes

def _definition(q, k, v, sees, scale):
    """(o, tolerance) of rows q [m, Hq, D] over k, v [n, Hkv, D], in 64 bits; sees [m, n].  As kv_ref.row, with what fp16's small
    weights lose as test_many_small_weights_in_fp16 has it."""
    G, n, half = q.shape[1] // k.shape[1], k.shape[0], kv_ref.HALF[q.dtype]
    qd, kd, vd = q.double(), k.double().repeat_interleave(G, 1), v.double().repeat_interleave(G, 1)
    s = torch.einsum("mhd,nhd->hmn", qd, kd) * scale
    size = (torch.einsum("mhd,nhd->hmn", qd.abs(), kd.abs()) * scale).masked_fill(~sees, 0).amax(-1).t()[..., None]
    w = s.masked_fill(~sees, -torch.inf).softmax(-1)
    o, oabs = torch.einsum("hmn,nhd->mhd", w, vd), torch.einsum("hmn,nhd->mhd", w, vd.abs())
    tol = half * o.abs() + (half + 2 * ((q.shape[2] + 6) * kv_ref.E23 * size + 2.0 ** -22) + (2 * n + 64) * kv_ref.E23) * oabs
    if q.dtype is FP:
        tol = tol + n * 2.0 ** -32 * vd.abs().max() + 2.0 ** -25
    return o, tol


def _sees(pos, count, n, window, sinks):
    p, t = torch.arange(pos, pos + count, device=DEV)[:, None], torch.arange(n, device=DEV)
    return (t <= p) & ((t > p - (window or 1 << 40)) | (t < sinks))


@pytest.mark.parametrize("seed", range(60))
def test_random_prompts(seed):
    """Shapes, windows, lengths and padding at random, NaN in all that is past a sequence."""
    import random
    r, g = random.Random(seed), gen(1000 + seed)
    D, G, dt = r.choice((64, 128, 256)), r.choice((1, 2, 3, 4, 5, 7, 8, 16, 32, 64)), r.choice((BF, FP))
    Hkv, B, M = r.choice((1, 2, 3)) if G < 16 else 1, r.choice((1, 2, 3, 6)), int(2 ** r.uniform(0, 10))
    T = M + int(2 ** r.uniform(0, 11)) - 1
    while B * M * G * Hkv * T > 1 << 25:
        M = max(1, M // 2)
        T = max(M, T // 2)
    W = r.choice((None, 1, 2, 63, 64, 65, 100, 128, 129, 500, int(2 ** r.uniform(0, 11))))
    S = 0 if W is None else r.choice((0, 0, 1, 4, 63, 64, 65, 130, 300))
    q, k, v = rows(g, B, M, G * Hkv, D, dtype=dt), rows(g, B, T, Hkv, D, dtype=dt), rows(g, B, T, Hkv, D, dtype=dt)
    ragged = r.random() < 0.6
    counts = [r.choice((0, 1, M, r.randint(0, M))) if ragged else M for _ in range(B)]
    pos = [r.randint(0, T - c) if r.random() > 0.1 else -1 for c in counts] if r.random() < 0.7 else [T - M] * B
    for b in range(B):
        end = pos[b] + counts[b] if pos[b] >= 0 else 0
        k[b, end:], v[b, end:] = float("nan"), float("nan")
    o, err = moe.window_attention(q, k, v, W, sinks=S, pos=i32(pos), counts=i32(counts) if ragged else None)
    assert err_of(err) == 0
    for b in range(B):
        c = counts[b] if pos[b] >= 0 else 0
        assert not o[b, c:].any()
        if c:
            n = pos[b] + c
            kv_ref.close(o[b, :c], *_definition(q[b, :c], k[b, :n], v[b, :n], _sees(pos[b], c, n, W, S), D ** -0.5), f"sequence {b}")


@pytest.mark.parametrize("seed", range(60))
def test_random_caches(seed):
    """The same over rings, with rejected rows behind the last position, and over linear caches behind prefixes."""
    import random
    r, g = random.Random(seed), gen(2000 + seed)
    D, G, dt = r.choice((64, 128, 256)), r.choice((1, 2, 4, 5, 8, 16, 32, 64)), r.choice((BF, FP))
    Hkv, M, B = r.choice((1, 2, 3)) if G < 16 else 1, r.randint(1, 8), r.choice((1, 2, 4, 9, 33))
    W, S, P = None, 0, 0
    if r.random() < 0.6:
        W, S = r.choice((1, 7, 64, 100, 128, 300, 1000)), r.choice((0, 1, 4, 64, 70, 130))
        T = S + W + M - 1 + r.choice((0, 1, 8, 50, 200))
        top = 3 * T + 5
    else:
        T = top = max(M, r.choice((M, 70, 300, 1500)))
        P = r.choice((0, 1, 100, 129, 1000, 4000))
    ends = [r.choice((0, M, top, r.randint(0, top))) for _ in range(B)]        # positions with the call's rows
    counts = [min(r.choice((M, M, 0, r.randint(0, M))), e) for e in ends]
    pos = [e - c if c or r.random() < 0.5 else -1 for e, c in zip(ends, counts)]
    n = max(max(ends), 1)
    k, v = rows(g, B, n, Hkv, D, dtype=dt), rows(g, B, n, Hkv, D, dtype=dt)
    cache = moe.KVCache(T, batch=B, q_heads=G * Hkv, kv_heads=Hkv, head_dim=D, dtype=dt, window=W, sinks=S, max_rows=M, max_prefix=P)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    cache.append(k, v, i32([0 if e else -1 for e in ends]), counts=i32(ends))
    # rows behind the last one, as many as leave what the first row sees
    room = [min(M, T - e if W is None else T - S - W - c + 1) for e, c in zip(ends, counts)]
    bad = torch.full((B, M, Hkv, D), float("nan"), dtype=dt, device=DEV)
    cache.append(bad, bad, i32([e if x > 0 else -1 for e, x in zip(ends, room)]), counts=i32([max(x, 0) for x in room]))
    assert err_of(cache.err) == 0
    q = rows(g, B, M, G * Hkv, D, dtype=dt)
    prefix = (rows(g, P, Hkv, D, dtype=dt), rows(g, P, Hkv, D, dtype=dt)) if P else None
    o, err = cache.attend(q, i32(pos), counts=i32(counts), prefix=prefix)
    assert err_of(err) == 0
    for b in range(B):
        c = counts[b] if pos[b] >= 0 else 0
        assert not o[b, c:].any()
        if c:
            e, sees, own = ends[b], _sees(pos[b], c, ends[b], W, S), (k[b, :ends[b]], v[b, :ends[b]])
            if P:
                own = [torch.cat([x, y]) for x, y in zip(prefix, own)]
                sees = torch.cat([torch.ones((c, P), dtype=torch.bool, device=DEV), sees], 1)
            kv_ref.close(o[b, :c], *_definition(q[b, :c], *own, sees, D ** -0.5), f"sequence {b} of {e}")
