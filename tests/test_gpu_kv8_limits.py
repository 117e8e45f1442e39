"""GPU tests of the 8-bit key/value cache at the limits of its numbers, and on
streams other than the one that made it."""
import pytest
import torch

import quantized_moe_decode_layer_gb300 as moe
from test_gpu_kv8 import DEV, E23, err_of, filled, gen, i32, rows

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ attention

def test_scores_one_spacing_apart():
    """Scores of 2^27, where fp32's neighbours are 16 apart: the output is still
    a weighted mean of the values."""
    D = 64
    cache = moe.KV8Cache(40960, q_heads=1, kv_heads=1, head_dim=D, block=16)
    r = gen(40)
    k, v = torch.zeros((1, 1024, 1, D), device=DEV), rows(r, 1, 1024, 1, D, dtype=torch.float32)
    k[..., 0] = 64.0
    k[0, 256:, 0, 1] = 1.0                               # q . k: 64 and its neighbour in fp32
    cache.append(k, v, i32([0]))
    low, high = (f(cache.v[0, 0, :1024].double() * cache.v_scale[0, 0, :64].repeat_interleave(16)[:, None].double(), 0)
                 for f in (torch.amin, torch.amax))
    q = torch.zeros((1, 1, 1, D), dtype=torch.bfloat16, device=DEV)
    q[..., 0], q[..., 1] = 1.0, 2.0 ** -17
    for step in range(64):                               # half of them make the first score an odd multiple of 16
        scale = 2.0 ** 21 * 0.6931471805599453 * (1 + step * 2.0 ** -23)
        o, _ = cache.attend(q, i32([1023]), scale=scale)
        assert ((o[0, 0, 0].double() >= low - 1e-4) & (o[0, 0, 0].double() <= high + 1e-4)).all(), step


def one_head(cache, q, n, scale):
    """In 64 bits: the output of rows q [M, heads, D] over a cache of one
    key/value head whose first n positions all rows see, and its tolerance.

    A score is off by (D + 4) 2^-23 of scale * sum |q_d k_d| (test_gpu_kv8), its
    exponential by that and a few 2^-23 more, and a weight by 2^-22 when it is
    split; what this does to each term counts with the term's own weight, twice
    for the normaliser.  Sums add up to 1024 + chunks terms in a row.  Beside that, a
    weight is off by 2^-18 of the largest weight * step among the 64 positions around it
    (of the largest weight times the largest step, where that is less than 16 times as much),
    in units of its own step."""
    blk = cache.block
    step = [s[0, 0].repeat_interleave(blk)[:n, None].double() for s in (cache.k_scale, cache.v_scale)]
    k, code = cache.k[0, 0, :n].float().double() * step[0], cache.v[0, 0, :n].float().double()
    v = code * step[1]
    z, a = torch.einsum("mhd,td->mht", q.double(), k) * scale, torch.einsum("mhd,td->mht", q.double().abs(), k.abs()) * scale
    w = torch.softmax(z, -1)
    e = (cache.head_dim + 12) * E23 * a + 8 * E23 + 2.0 ** -22
    o, oabs = w @ v, w @ v.abs()
    most, wide, both = (torch.nn.functional.pad(x, (0, -n % 64)).unflatten(-1, (-1, 64)).amax(-1).repeat_interleave(64, -1)[..., :n]
                        for x in (w, step[1][:, 0], w * step[1][:, 0]))
    top = torch.minimum(most * wide, 16 * both)
    tol = (w * e) @ v.abs() + (w * e).sum(-1, keepdim=True) * o.abs() + 2 * (1024 + cache.T_cap // 128) * E23 * oabs
    return o, tol + 2.0 ** -18 * (top @ code.abs()) + 1e-37


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("M", [1, 2])
def test_weight_behind_a_block_of_far_larger_values(fmt, D, M):
    """A block of 16 whose values are 2^ratio times the others' and whose weights are 2^-low
    of theirs, at the start of a warp's share of a chunk or inside it: the others' output stays."""
    n, T = 700, 40960
    for i, (ratio, low, at) in enumerate([(16, 100, 0), (20, 100, 0), (24, 100, 0), (28, 100, 16), (32, 100, 0), (40, 60, 0),
                                          (48, 100, 32), (64, 100, 0), (100, 100, 0), (100, 118, 0), (60, 40, 0), (100, 110, 320),
                                          (32, 100, 672), (None, -30, 0), (None, -80, 0), (None, -60, 256)]):
        r = gen(41 + i)
        cache = moe.KV8Cache(T, q_heads=8, kv_heads=1, head_dim=D, block=16, fmt=fmt)
        k, v = rows(r, 1, n, 1, D, dtype=torch.float32), rows(r, 1, n, 1, D, dtype=torch.float32)
        q = rows(r, 1, M, 8, D)
        q[..., 0] = 8.0
        k[..., 0] = 0.0
        k[:, at:at + 16] = 0.0
        k[:, at:at + 16, :, 0] = -low * 0.6931471805599453 * D ** 0.5 / 8
        v[:, at:at + 16] *= 0.0 if ratio is None else 2.0 ** ratio        # None: nothing but zeros where the weight is
        cache.append(k, v, i32([0]))
        for m in range(M):
            o, tol = one_head(cache, q[0, m:m + 1], n - M + 1 + m, D ** -0.5)
            got, _ = cache.attend(q, i32([n - M]))
            d = (got[0, m:m + 1].double() - o).abs()
            assert (d <= tol).all(), f"2^{ratio}, weight 2^-{low}, at {at}: worst {float((d / tol).max()):.3g} tolerances"


@pytest.mark.parametrize("fmt,D,Hq,G,T,n", [("int8", 256, 16, 2, 2048, 1500), ("e4m3", 128, 8, 1, 40960, 700), ("int8", 64, 4, 4, 40960, 40000)])
def test_values_of_any_size(fmt, D, Hq, G, T, n):
    """Values times a power of two give exactly the output times it, up to where sums of
    values would overflow."""
    r = gen(60)
    k, v, q = rows(r, 1, n, G, D), rows(r, 1, n, G, D, dtype=torch.float32), rows(r, 1, 2, Hq, D)
    want = None
    for e in (0, -90, -30, 60, 118, 124):
        cache = moe.KV8Cache(T, q_heads=Hq, kv_heads=G, head_dim=D, block=16, fmt=fmt)
        cache.append(k.float(), v * 2.0 ** e, i32([0]))
        o, _ = cache.attend(q, i32([n - 2]))
        want = o.double() if want is None else want
        assert torch.equal(o.double(), want * 2.0 ** e), e


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows_do_not_interact_over_uneven_blocks(fmt, D):
    """Steps of values 2^-60 to 2^60 apart, near the largest and the smallest, whole blocks of zeros, scores
    of a few and of a hundred: every row of a call is bitwise the one-row call at its position, alone or beside
    another sequence."""
    for case, (T, n, spread, size, base) in enumerate([(40960, 1500, 60, 40.0, 0), (40960, 1500, 3, 1.0, 0), (512, 300, 60, 5.0, 0),
                                                       (40960, 1100, 0, 100.0, 0), (40960, 1100, 2, 10.0, 122), (40960, 1100, 4, 30.0, -115)]):
        r = gen(70 + case)
        cache = moe.KV8Cache(T, batch=2, q_heads=3, kv_heads=1, head_dim=D, block=16, fmt=fmt)
        k, v = rows(r, 2, n, 1, D, dtype=torch.float32), rows(r, 2, n, 1, D, dtype=torch.float32)
        blocks = -(-n // 16)
        e = torch.randint(-spread, spread + 1, (2, blocks), generator=r, device=DEV).float()
        s = torch.exp2(e) * (torch.rand((2, blocks), generator=r, device=DEV) > 0.1)
        v *= s.repeat_interleave(16, 1)[:, :n, None, None] * 2.0 ** base
        cache.append(k, v, i32([0, 0]))
        q = rows(r, 2, 8, 3, D, size=size)
        for first in (n - 8, n - 13, 321):
            got, _ = cache.attend(q, i32([first, first - 5]))
            assert torch.isfinite(got).all()
            for m in range(8):
                one, _ = cache.attend(q[:, m:m + 1], i32([first + m, -1]))
                two, _ = cache.attend(q[:, m:m + 1], i32([-1, first - 5 + m]))
                assert torch.equal(one[0, 0].view(torch.int32), got[0, m].view(torch.int32)), (case, first, m)
                assert torch.equal(two[1, 0].view(torch.int32), got[1, m].view(torch.int32)), (case, first, m)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_largest_numbers_stay_finite(fmt, dtype):
    """The type's largest number, and infinities, which count as it, come back as
    finite ones: at most the largest of the result's type."""
    D, big = 64, torch.finfo(dtype).max
    cache = moe.KV8Cache(32, q_heads=2, kv_heads=1, head_dim=D, block=16, fmt=fmt)
    v = torch.zeros((1, 32, 1, D), dtype=dtype, device=DEV)
    v[0, :16, 0, 0], v[0, :16, 0, 1], v[0, :16, 0, 2] = big, -big, big / 2
    v[0, 16:, 0, 0], v[0, 16:, 0, 1] = float("inf"), -float("inf")
    cache.append(torch.zeros_like(v), v, i32([0]))
    assert err_of(cache) == moe.KV8Cache.ERR_NONFINITE
    code = cache.v[0, 0, :, :3].float().double() * cache.v_scale[0, 0].repeat_interleave(16)[:, None].double()
    assert ((code[:16] - torch.tensor([big, -big, big / 2], device=DEV, dtype=torch.float64)).abs() <= 2.0 ** 124).all()
    top = torch.finfo(torch.bfloat16).max
    assert torch.equal(cache.read(None, 32)[1][0, :, 0, :3].double(), code.clamp(-top, top))
    q = torch.zeros((1, 1, 2, D), dtype=torch.bfloat16, device=DEV)
    for out in (torch.float32, torch.bfloat16):
        top = torch.finfo(out).max
        for pos in (0, 9, 31):
            o, _ = cache.attend(q, i32([pos]), out_dtype=out)
            want = code[:pos + 1].mean(0).clamp(-top, top)
            assert torch.isfinite(o).all()
            assert ((o[0, 0, :, :3].double() - want).abs() <= want.abs() * (2.0 ** -8 if out == torch.bfloat16 else 2.0 ** -18)).all()


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16, torch.float16])
def test_nan_is_an_output_of_every_type(out):
    """A query with a NaN or an infinity gives NaN, and not the type's largest number."""
    cache = moe.KV8Cache(32, q_heads=3, kv_heads=1, head_dim=64, block=16)
    k = rows(gen(63), 1, 20, 1, 64)
    cache.append(k, k, i32([0]))
    q = rows(gen(64), 1, 1, 3, 64)
    q[0, 0, 0, 5], q[0, 0, 2, 7] = float("nan"), float("inf")
    o, _ = cache.attend(q, i32([19]), out_dtype=out)
    assert o[0, 0, 0].isnan().all() and o[0, 0, 2].isnan().all() and torch.isfinite(o[0, 0, 1]).all()


# -------------------------------------------------------------------- streams

def busy(stream):
    with torch.cuda.stream(stream):
        torch.cuda._sleep(100_000_000)


def test_what_an_explicit_stream_reads_is_kept():
    """A caller may drop a call's inputs right after it: their memory is not
    handed out while the call's stream still has to read it."""
    B, G, D = 1, 2, 64
    cache, r = filled(B, 4, G, D, 64, 16, "int8", [40], 61, weights=True)
    dst = moe.KV8Cache(64, batch=B, q_heads=4, kv_heads=G, head_dim=D, block=16)
    st = torch.cuda.Stream()
    f32 = torch.float32
    make = {"k": lambda: rows(r, B, 3, G, D), "q": lambda: rows(r, B, 3, 4, D), "pos": lambda: i32([37]), "acc": lambda: torch.zeros((B, G, 64), device=DEV),
            "out": lambda: torch.empty((B, 3, 4, D), device=DEV, dtype=f32), "err": lambda: torch.zeros(1, dtype=torch.int32, device=DEV)}
    calls = [(("k", "k", "pos", "pos", "err"), lambda k, v, pos, counts, err: cache.append(k, v, pos, counts=counts, err=err, stream=st)),
             (("pos", "pos"), lambda start, lens: cache.read(start, 3, lens=lens, stream=st)),
             (("q", "pos", "pos", "acc", "acc", "out", "err"), lambda q, pos, counts, acc, acc_in, out, err:
              cache.attend(q, pos, counts=counts, acc=acc, acc_in=acc_in, out=out, err=err, stream=st) and None),
             (("pos", "acc", "acc", "err"), lambda lens, acc, dacc, err: cache.evict_into(dst, lens, acc, 8, dst_acc=dacc, err=err, stream=st))]
    for names, call in calls:
        spare = [make[x]() for x in 3 * names]                # below, neither an allocation nor a
        call(*spare[:len(names)])                             # kernel's loading waits for the device
        torch.cuda.synchronize()
        del spare
        args = [make[x]() for x in names]
        torch.cuda.synchronize()
        busy(st)
        result = call(*args)
        freed = {t.data_ptr() for t in args}
        del args
        new = [make[x]() for x in names]
        assert not st.query() and not freed & {t.data_ptr() for t in new}, names
        torch.cuda.synchronize()
        del result, new


@pytest.mark.parametrize("explicit", [True, False])
def test_a_dropped_caches_memory_is_kept(explicit):
    """The cache's own buffers, scratch and error word, used on another stream
    than they were made on, outlive the cache until that stream is done."""
    q, pos = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16, device=DEV), i32([0])
    st = torch.cuda.Stream()
    cache = moe.KV8Cache(4096, q_heads=4, kv_heads=2, head_dim=64, block=16)
    cache.attend(q, pos)
    parts = (cache.k, cache.v, cache.k_scale, cache.v_scale, cache.ws, cache.err)
    shapes, freed = [(t.shape, t.dtype) for t in parts], {t.data_ptr() for t in parts}
    spare = [torch.empty(s, dtype=d, device=DEV) for s, d in 2 * shapes]       # no allocation below waits for the device
    del parts, spare
    torch.cuda.synchronize()
    busy(st)
    if explicit:
        o = cache.attend(q, pos, stream=st)[0]
    else:
        with torch.cuda.stream(st):
            o = cache.attend(q, pos)[0]
    del cache
    new = [torch.empty(s, dtype=d, device=DEV) for s, d in shapes]
    assert not st.query() and not freed & {t.data_ptr() for t in new}
    torch.cuda.synchronize()
    del o


@pytest.mark.parametrize("explicit", [True, False])
def test_a_new_cache_is_ready_on_any_stream(explicit):
    """The first call on a stream comes after the cache's own initialisation."""
    k, pos = rows(gen(62), 1, 16, 1, 64), i32([0])
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy(torch.cuda.current_stream())
    cache = moe.KV8Cache(64, q_heads=1, kv_heads=1, head_dim=64, block=16)
    if explicit:
        cache.append(k, k, pos, stream=st)
    else:
        with torch.cuda.stream(st):
            cache.append(k, k, pos)
    torch.cuda.synchronize()
    assert cache.k[0, 0, :16].any() and (cache.k_scale[0, 0, :1] > 0).all()


def test_a_result_dropped_by_its_reader_is_kept():
    """A result of an explicit stream that the current stream reads and drops is
    not handed to that stream's next call before it has been read."""
    cache, r = filled(1, 4, 2, 64, 64, 16, "int8", [40], 65)
    q, pos = rows(r, 1, 1, 4, 64), i32([39])
    st, cur = torch.cuda.Stream(), torch.cuda.current_stream()
    zero, seen = torch.zeros_like(q), torch.empty((1, 1, 4, 64), device=DEV)
    st.wait_stream(cur)
    o = cache.attend(q, pos, stream=st)[0]
    spare = cache.attend(q, pos, stream=st)[0]
    cur.wait_stream(st)
    seen.copy_(o)
    del spare
    torch.cuda.synchronize()
    busy(cur)
    seen.copy_(o)
    at = o.data_ptr()
    del o
    again = cache.attend(zero, pos, stream=st)[0]
    assert not cur.query() and again.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(seen, cache.attend(q, pos)[0])


def test_first_call_of_a_stream_in_a_capture():
    """A stream's first call may be one that is captured, on a fork of the
    captured stream too; eager calls on it wait as ever."""
    cache, r = filled(1, 4, 2, 64, 64, 16, "int8", [40], 66)
    q, pos = rows(r, 1, 1, 4, 64), i32([39])
    want = cache.attend(q, pos)[0]
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        a = cache.attend(q, pos)[0]
        st.wait_stream(torch.cuda.current_stream())
        b = cache.attend(q, pos, stream=st)[0]
        torch.cuda.current_stream().wait_stream(st)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)
    assert torch.equal(cache.attend(q, pos, stream=st)[0].cpu(), want.cpu())


# ------------------------------------------------------------- what a code keeps

@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_values_stay_near_what_was_appended(fmt):
    """Through blocks that grow and evictions that gather values of other steps: within
    one step (int8), or 2^-4 of the value and 2^-9 of a step (e4m3), of the largest step that a
    value has had.  (A rounding is off by half a step, or 2^-4 |x| and by 2^-10 steps below 2^-6
    steps; a value is rounded again only to a step at least twice any before, so these
    halves add up to less than twice the last.)"""
    B, G, D, T, block = 2, 2, 64, 256, 16
    a, c = (moe.KV8Cache(T, batch=B, q_heads=2, kv_heads=G, head_dim=D, block=block, fmt=fmt) for _ in range(2))
    r = gen(80)
    x = torch.zeros((2, B, G, T, D), dtype=torch.float64, device=DEV)         # what was appended where
    largest = torch.zeros((2, B, G, T), dtype=torch.float64, device=DEV)      # the steps it has had
    n, worst = 0, 0.0

    def look():
        nonlocal worst
        for i, (codes, steps) in enumerate(((a.k, a.k_scale), (a.v, a.v_scale))):
            step = steps.double().repeat_interleave(block, 2)
            largest[i, :, :, :n] = torch.maximum(largest[i], step)[:, :, :n]
            got = codes.float().double() * step[..., None]
            s, d = largest[i, :, :, :n, None], (got - x[i])[:, :, :n].abs()
            bound = s if fmt == "int8" else x[i, :, :, :n].abs() * 2.0 ** -4 + s * 2.0 ** -9
            assert (d <= bound).all(), float((d / bound).max())
            worst = max(worst, float((d / s).max()))

    for turn in range(150):
        m = 1 + turn % 4
        size = 2.0 ** float(torch.randint(-12, 12, (1,), generator=r, device=DEV))
        rows_ = torch.randn((2, B, m, G, D), generator=r, device=DEV) * size
        a.append(rows_[0], rows_[1], i32([n] * B))
        x[:, :, :, n:n + m] = rows_.transpose(2, 3).double()
        largest[:, :, :, n:n + m] = 0.0
        n += m
        look()
        if n > T - 8:
            acc = torch.rand((B, G, T), generator=r, device=DEV)
            idx, lens = a.evict_into(c, i32([n] * B), acc, 100, sinks=2, recent=3)
            at = idx.long()
            x[:, :, :, :100] = torch.gather(x, 3, at.expand(2, B, G, 100)[..., None].expand(2, B, G, 100, D))
            largest[..., :100] = torch.gather(largest, 3, at.expand(2, B, G, 100))
            a, c, n = c, a, 100
            look()
    # int8: within a step; e4m3 is not (codes of 256 to 448 are 32 apart)
    assert worst <= 1.0 if fmt == "int8" else worst > 1.0


# ------------------------------------------------------------------- scratch

def test_caches_share_scratch():
    """Caches whose calls follow one another, of unequal shapes, over the scratch of the
    largest; scratch that is too small or no such tensor is refused."""
    big, r = filled(2, 16, 2, 128, 4096, 64, "int8", [4000, 1234], 90, weights=True)
    small, _ = filled(1, 8, 2, 64, 512, 32, "e4m3", [500], 91)
    q, qs = rows(r, 2, 3, 16, 128), rows(r, 1, 8, 8, 64)
    acc, acc2 = torch.zeros((2, 2, 4096), device=DEV), torch.zeros((2, 2, 4096), device=DEV)
    want, _ = big.attend(q, i32([3997, 1231]), acc=acc)
    wants, _ = small.attend(qs, i32([492]))
    over = moe.KV8Cache(512, batch=1, q_heads=8, kv_heads=2, head_dim=64, block=32, fmt="e4m3",
                        buffers=(small.k, small.v, small.k_scale, small.v_scale), ws=big.ws)
    assert over.ws is big.ws and over.ws.numel() > small.ws.numel()
    for _ in range(3):
        a, _ = over.attend(qs, i32([492]))
        b, _ = big.attend(q, i32([3997, 1231]), acc=acc2, acc_in=torch.zeros_like(acc2))
        assert torch.equal(a, wants) and torch.equal(b, want) and torch.equal(acc2, acc)
    for bad in (small.ws, big.ws.view(torch.int32), big.ws.cpu(), big.ws[:-1], big.ws.view(2, -1)):
        with pytest.raises(ValueError):
            moe.KV8Cache(4096, batch=2, q_heads=16, kv_heads=2, head_dim=128, weights=True, ws=bad)
    with pytest.raises(moe.MoeError):                     # not on a 16-byte boundary: refused by the call
        odd = moe.KV8Cache(512, batch=1, q_heads=8, kv_heads=2, head_dim=64, block=32, ws=big.ws[1:])
        odd.attend(qs, i32([0]))
    torch.cuda.synchronize()
