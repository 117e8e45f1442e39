"""The 16-bit key/value cache's calls without a GPU: sizes and refusals, which
come before any launch."""
import ctypes as C

import pytest
import torch

import quantized_moe_decode_layer_gb300 as moe
from quantized_moe_decode_layer_gb300 import _lib
from quantized_moe_decode_layer_gb300._lib import Kv, Rows, Window

FAKE = 1 << 30   # never dereferenced: every call below is refused first


def cache(batch=2, q_heads=16, kv_heads=2, head_dim=256, T_cap=128, type=0, window=0, sinks=0, at=FAKE):
    return Kv(batch, q_heads, kv_heads, head_dim, T_cap, type, window, sinks, at, at + (1 << 26))


def row(at=FAKE, type=0, seq=0, row=0, head=0):
    return Rows(at, type, seq, row, head)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), 1), (dict(kv_heads=0), 1), (dict(q_heads=0), 1), (dict(T_cap=0), 1), (dict(window=-1), 1), (dict(sinks=-1), 1),
    (dict(sinks=1), 1), (dict(window=128, sinks=1), 1), (dict(window=129), 1), (dict(type=2), 2), (dict(head_dim=96), 2),
    (dict(q_heads=15), 2), (dict(q_heads=130), 2), (dict(batch=1025), 2), (dict(T_cap=(1 << 22) + 1), 2),
    (dict(kv_heads=1025, q_heads=1025), 2)])
def test_shapes_refused(kw, code):
    L, n = moe.lib(), C.c_size_t()
    c, r = cache(**kw), row()
    r16 = row(type=kw.get("type", 0))
    assert L.moe_kv_attn_workspace_size(c, 1, 0, n) == code
    assert L.moe_kv_append(c, r, r, 1, FAKE, None, FAKE, None) == code
    assert L.moe_kv_attn(c, r16, 1, FAKE, None, None, None, 0, 1.0, FAKE, FAKE, 1 << 40, FAKE, None) == code


def test_append_refusals():
    L = moe.lib()

    def app(k=row(), v=row(), M=1, pos=FAKE, err=FAKE, c=cache()):
        return L.moe_kv_append(c, k, v, M, pos, None, err, None)
    assert app(c=None) == 1 and app(k=None) == 1 and app(v=None) == 1 and app(pos=None) == 1 and app(err=None) == 1
    assert app(M=0) == 1 and app(M=129) == 1 and app(M=(1 << 22) + 1, c=cache(window=10)) == 1
    for bad in (row(None), row(type=3), row(type=-1), row(FAKE + 1), row(seq=-1), row(row=-8), row(head=-8), row(type=1)):
        assert app(k=bad) == 1
    half = cache()
    half.v_dev = None
    assert app(c=half) == 1
    half.v_dev = FAKE + 8
    assert app(c=half) == 1


def test_attention_refusals():
    L, n = moe.lib(), C.c_size_t()
    assert L.moe_kv_attn_workspace_size(cache(), 0, 0, n) == 1 and L.moe_kv_attn_workspace_size(cache(), 9, 0, n) == 1
    assert L.moe_kv_attn_workspace_size(cache(), 1, -1, n) == 1 and L.moe_kv_attn_workspace_size(cache(), 1, 0, None) == 1
    assert L.moe_kv_attn_workspace_size(cache(), 1, (1 << 22) + 1, n) == 1
    assert L.moe_kv_attn_workspace_size(None, 1, 0, n) == 1
    assert L.moe_kv_attn_workspace_size(cache(window=120), 9 - 1, 0, n) == 0                 # 120 + 7 of 128
    assert L.moe_kv_attn_workspace_size(cache(window=122), 8, 0, n) == 1
    assert L.moe_kv_attn_workspace_size(cache(window=100), 1, 64, n) == 1                    # a prefix and a window
    assert L.moe_kv_attn_workspace_size(cache(), 1, 0, n) == 0
    need = n.value

    def at(c=cache(), q=row(), M=4, pos=FAKE, pk=None, pv=None, P=0, scale=1.0, o=FAKE, ws=FAKE, nb=1 << 40, err=FAKE):
        return L.moe_kv_attn(c, q, M, pos, None, pk, pv, P, scale, o, ws, nb, err, None)
    assert at(q=None) == 1 and at(M=0) == 1 and at(M=9) == 1 and at(pos=None) == 1 and at(o=None) == 1 and at(o=FAKE + 8) == 1
    assert at(M=1, ws=None) == 1 and at(M=1, ws=FAKE + 4) == 1 and at(err=None) == 1
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert at(scale=s) == 1
    for bad in (row(FAKE + 8), row(type=1), row(type=2), row(seq=4), row(row=-8), row(head=12)):
        assert at(q=bad) == 1 and at(pk=bad, pv=row(), P=5) == 1 and at(pk=row(), pv=bad, P=5) == 1
    assert at(pk=row(), P=5) == 1 and at(pk=row(), pv=row(), P=0) == 1 and at(P=5) == 1 and at(pk=row(), pv=row(), P=-1) == 1
    assert at(c=cache(window=64), pk=row(), pv=row(), P=5) == 1
    assert at(c=cache(T_cap=3)) == 1
    assert at(M=1, nb=need - 1) == 3 and at(M=1, nb=0, pk=row(), pv=row(), P=5) == 3


def test_prompt_refusals():
    L, n = moe.lib(), C.c_size_t()

    def shape(batch=2, q_heads=16, kv_heads=2, head_dim=128, rows=70, positions=100, window=10, sinks=2):
        return Window(batch, q_heads, kv_heads, head_dim, rows, positions, window, sinks)
    far = dict(seq=1 << 20, row=1024, head=128)

    def at(s=shape(), q=row(**far), k=row(**far), v=row(**far), scale=1.0, o=FAKE, ws=FAKE, nb=1 << 40, err=FAKE):
        return L.moe_window_attn(s, q, k, v, None, None, scale, o, ws, nb, err, None)
    for kw, code in ((dict(batch=0), 1), (dict(rows=0), 1), (dict(rows=101), 1), (dict(window=-1), 1), (dict(window=0), 1), (dict(sinks=-1), 1),
                     (dict(head_dim=80), 2), (dict(q_heads=17), 2), (dict(q_heads=130), 2), (dict(batch=1025), 2),
                     (dict(positions=(1 << 22) + 1), 2)):
        assert L.moe_window_attn_workspace_size(shape(**kw), n) == code and at(s=shape(**kw)) == code
    assert L.moe_window_attn_workspace_size(shape(), None) == 1 and L.moe_window_attn_workspace_size(None, n) == 1
    for bad in (None, row(None), row(FAKE + 8, **far), row(type=1, **far), row(type=2, **far), row(seq=4), row(seq=8, row=-8)):
        assert at(k=bad) == 1 and at(v=bad) == 1
    assert at(q=None) == 1 and at(q=row(type=2, **far)) == 1 and at(q=row(FAKE + 2, **far)) == 1
    for zero in ("seq", "row", "head"):                       # an expanded dimension of keys or values
        assert at(k=row(**{**far, zero: 0})) == 1 and at(v=row(**{**far, zero: 0})) == 1
    assert at(o=None) == 1 and at(o=FAKE + 8) == 1 and at(err=None) == 1 and at(scale=0.0) == 1
    few = shape(rows=1, batch=1, positions=5000, window=0, sinks=0)
    assert L.moe_window_attn_workspace_size(few, n) == 0 and n.value > 0
    assert at(s=few, ws=None) == 1 and at(s=few, ws=FAKE + 4) == 1 and at(s=few, nb=n.value - 1) == 3


def test_workspace_covers_every_smaller_call():
    """The scratch for max_rows rows and a prefix is enough for fewer rows and without one."""
    L, n = moe.lib(), C.c_size_t()
    for q, g in ((8, 8), (16, 2), (64, 1), (10, 2)):
        for B in (1, 5, 60, 300):
            sizes = []
            for M in range(1, 9):
                for P in (0, 7, 100000):
                    assert L.moe_kv_attn_workspace_size(cache(batch=B, q_heads=q, kv_heads=g, T_cap=5000), M, P, n) == 0
                    sizes.append((M, P, n.value))
            most = sizes[-1][2]
            assert all(s <= most for _, _, s in sizes)


def test_binding_refuses_before_the_library():
    for kw in (dict(dtype=torch.float32), dict(window=0)):
        with pytest.raises(ValueError):
            moe.KVCache(128, device="cpu", **kw)
    for kw in (dict(max_rows=9), dict(window=200), dict(window=50, max_prefix=9), dict(head_dim=80), dict(sinks=3)):
        with pytest.raises(moe.MoeError):
            moe.KVCache(128, device="cpu", **kw)
    with pytest.raises(ValueError):
        moe.KVCache(128, device="cpu")                        # host buffers
    x = torch.zeros((1, 8, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.window_attention(x, x, x)
    assert C.sizeof(Kv) == 48 and C.sizeof(Window) == 32
    assert {"moe_kv_append", "moe_kv_attn", "moe_window_attn"} <= set(_lib.SYMBOLS)


@pytest.mark.parametrize("window,sinks", [(0, 0), (-1, 0), (2 ** 31, 0), (2 ** 32 + 5, 0), (7, -1), (7, 2 ** 31), (7, 2 ** 32 + 1)])
def test_windows_outside_32_bits(window, sinks):
    """None of them reaches the library, which would see their low 32 bits."""
    with pytest.raises(ValueError, match="window must be"):
        moe.window_attention_workspace(1, 8, 2, 64, 1000, 1000, window, sinks)
    with pytest.raises(ValueError, match="window must be"):
        moe.KVCache(2000, q_heads=8, kv_heads=2, head_dim=64, window=window, sinks=sinks, device="cpu")


@pytest.mark.parametrize("q_heads,batch", [(2, 2), (16, 2), (16, 64)])
def test_expanded_prefixes_refused(q_heads, batch):
    """Positions or heads of a prefix that lie at one place, whatever the number of rows: few and many take different kernels."""
    L = moe.lib()
    c, far, q = cache(batch=batch, q_heads=q_heads), dict(row=512, head=256), row(seq=8192, row=4096, head=256)
    for zero in ("row", "head"):
        bad = row(**{**far, zero: 0})
        for k, v in ((bad, row(**far)), (row(**far), bad)):
            assert L.moe_kv_attn(c, q, 1, FAKE, None, k, v, 5, 1.0, FAKE, FAKE, 1 << 40, FAKE, None) == 1
