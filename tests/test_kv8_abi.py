"""The 8-bit key/value cache's calls without a GPU: sizes and refusals, which
come before any launch."""
import ctypes as C

import pytest
import torch

import quantized_moe_decode_layer_gb300 as moe
from quantized_moe_decode_layer_gb300 import _lib
from quantized_moe_decode_layer_gb300._lib import Kv8, Rows

FAKE = 1 << 30   # never dereferenced: every call below is refused first


def cache(batch=2, q_heads=16, kv_heads=2, head_dim=256, T_cap=128, block=64, fmt=0, at=FAKE):
    return Kv8(batch, q_heads, kv_heads, head_dim, T_cap, block, fmt, at, at + (1 << 26), at + (2 << 26), at + (3 << 26))


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), 1), (dict(kv_heads=0), 1), (dict(T_cap=0), 1), (dict(T_cap=100), 1), (dict(fmt=2), 2),
    (dict(head_dim=96), 2), (dict(block=8), 2), (dict(block=48, T_cap=96), 2), (dict(q_heads=15), 2),
    (dict(q_heads=130), 2), (dict(batch=1025), 2), (dict(T_cap=(1 << 22) + 64), 2), (dict(kv_heads=1025, q_heads=1025), 2)])
def test_shapes_refused(kw, code):
    L, n = moe.lib(), C.c_size_t()
    c, r = cache(**kw), Rows(FAKE, 0, 0, 0, 0)
    assert L.moe_kv8_attn_workspace_size(C.byref(c), 1, 0, C.byref(n)) == code
    assert L.moe_kv8_append(C.byref(c), C.byref(r), C.byref(r), 1, FAKE, None, FAKE, None) == code
    assert L.moe_kv8_read(C.byref(c), None, 1, None, FAKE, FAKE, None) == code
    assert L.moe_kv8_attn(C.byref(c), C.byref(r), 1, FAKE, None, 1.0, FAKE, 0, None, None, 1.0, FAKE, 1 << 40, FAKE, None) == code
    ok = cache(at=2 * FAKE)
    assert L.moe_kv8_evict(C.byref(c), C.byref(ok), FAKE, FAKE, 1, 0, 0, None, FAKE, FAKE, FAKE, None) == code


def test_append_and_read_refusals():
    L, c, r = moe.lib(), cache(), Rows(FAKE, 0, 0, 0, 0)

    def app(k=r, v=r, M=1, pos=FAKE, err=FAKE, c=c):
        return L.moe_kv8_append(C.byref(c) if c else None, C.byref(k) if k else None, C.byref(v) if v else None, M, pos, None, err, None)
    assert app(c=None) == 1 and app(k=None) == 1 and app(v=None) == 1 and app(pos=None) == 1 and app(err=None) == 1
    assert app(M=0) == 1 and app(M=129) == 1
    for bad in (Rows(None, 0, 0, 0, 0), Rows(FAKE, 3, 0, 0, 0), Rows(FAKE, -1, 0, 0, 0), Rows(FAKE + 1, 0, 0, 0, 0),
                Rows(FAKE, 0, -1, 0, 0), Rows(FAKE, 0, 0, -8, 0), Rows(FAKE, 0, 0, 0, -8), Rows(FAKE, 1, 0, 0, 0)):
        assert app(k=bad) == 1
    assert app(k=Rows(FAKE + 2, 2, 0, 0, 0), v=Rows(FAKE, 2, 0, 0, 0)) == 1
    half = cache()
    half.v_dev = None
    assert app(c=half) == 1
    half.v_dev = FAKE + 8
    assert app(c=half) == 1
    for n, k, v in ((0, FAKE, FAKE), (129, FAKE, FAKE), (1, None, FAKE), (1, FAKE, FAKE + 2)):
        assert L.moe_kv8_read(C.byref(c), None, n, None, k, v, None) == 1


def test_attention_refusals():
    L, c, n = moe.lib(), cache(), C.c_size_t()
    assert L.moe_kv8_attn_workspace_size(C.byref(c), 0, 0, C.byref(n)) == 1
    assert L.moe_kv8_attn_workspace_size(C.byref(c), 9, 0, C.byref(n)) == 1
    assert L.moe_kv8_attn_workspace_size(C.byref(c), 1, 0, None) == 1
    assert L.moe_kv8_attn_workspace_size(C.byref(c), 4, 0, C.byref(n)) == 0
    need = n.value
    assert L.moe_kv8_attn_workspace_size(C.byref(c), 4, 1, C.byref(n)) == 0
    # the scores of 4 rows of 8 heads, fp32
    assert n.value - need == 2 * 2 * 128 * 32 * 4

    def at(q=Rows(FAKE, 0, 0, 0, 0), M=4, pos=FAKE, o=FAKE, ot=2, ain=None, acc=None, ws=FAKE, nb=1 << 40, err=FAKE):
        return L.moe_kv8_attn(C.byref(c), C.byref(q) if q else None, M, pos, None, 1.0, o, ot, ain, acc, 1.0, ws, nb, err, None)
    assert at(q=None) == 1 and at(q=Rows(FAKE, 2, 0, 0, 0)) == 1 and at(M=0) == 1 and at(M=9) == 1 and at(pos=None) == 1
    assert at(o=None) == 1 and at(o=FAKE + 2) == 1 and at(ot=3) == 1 and at(ain=FAKE) == 1 and at(ws=None) == 1
    assert at(ws=FAKE + 4) == 1 and at(err=None) == 1
    assert at(acc=FAKE, ain=FAKE + 4) == 1                        # overlapping, not the same
    assert at(nb=need - 1) == 3 and at(acc=FAKE, nb=n.value - 1) == 3


def test_evict_refusals():
    L, s, d = moe.lib(), cache(), cache(at=2 * FAKE)
    far = 8 * FAKE

    def ev(s=s, d=d, lens=far, acc=far + 4096, budget=64, sinks=4, recent=8, dacc=None, idx=far + (1 << 20), out=far + (2 << 20), err=FAKE):
        return L.moe_kv8_evict(C.byref(s), C.byref(d), lens, acc, budget, sinks, recent, dacc, idx, out, err, None)
    assert ev(lens=None) == 1 and ev(acc=None) == 1 and ev(idx=None) == 1 and ev(out=None) == 1 and ev(err=None) == 1
    assert ev(budget=0) == 1 and ev(budget=129) == 1 and ev(sinks=-1) == 1 and ev(recent=-1) == 1
    assert ev(sinks=60, recent=5) == 1 and ev(sinks=65, recent=0) == 1
    for kw in (dict(batch=1), dict(kv_heads=1), dict(head_dim=128), dict(block=32), dict(fmt=1)):
        assert ev(d=cache(at=2 * FAKE, **kw)) == 1
    assert ev(d=s) == 1 and ev(d=cache(at=FAKE + 64)) == 1        # into itself
    assert ev(out=far) == 1 and ev(dacc=far + 4096) == 1 and ev(idx=far + 4096) == 1 and ev(dacc=far + (1 << 20)) == 1


def test_binding_refuses_before_the_library():
    with pytest.raises(ValueError):
        moe.KV8Cache(128, fmt="int4", device="cpu")
    with pytest.raises(moe.MoeError):
        moe.KV8Cache(100, device="cpu")
    with pytest.raises(moe.MoeError):
        moe.KV8Cache(128, max_rows=9, device="cpu")
    with pytest.raises(ValueError):
        moe.KV8Cache(128, device="cpu")                           # host buffers
    assert C.sizeof(Kv8) == 64 and C.sizeof(Rows) == 40
    assert {"moe_kv8_append", "moe_kv8_attn", "moe_kv8_evict", "moe_kv8_read"} <= set(_lib.SYMBOLS)
