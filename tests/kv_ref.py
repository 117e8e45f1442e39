"""Attention with a window, first positions and a shared prefix in 64 bits, row
by row, and how far the kernels may be from it.

Tolerance, from the arithmetic.  A score is an fp32 sum of D exact products (a
tensor core may truncate: a step of 2^-23 each) and takes a scale and a
subtraction: |e| <= (D + 6) 2^-23 smax, smax the largest scale * sum_d |q_d k_d|
that the row sees; the exponential adds 2^-22 of itself.  Errors e of all weights
move the weighted mean by at most 2 e oabs, oabs = sum_t w_t |v_t|.  A weight is rounded
once to the 16-bit type for its product: half a step (2^-8, 2^-11) of itself, of
oabs in all; below 2^-14 of the reference an fp16 weight is off by 2^-25 of it
(the largest weight is at least the reference).  Sums over n positions add at most one
2^-23 an addition, for numerator and denominator; joining parts is among 64 more.  The
output is rounded once more: half a step of itself (fp16: 2^-25 at least)."""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
E23 = 2.0 ** -23


def seen(p, window, sinks):
    """Positions that the row at position p sees."""
    lo = 0 if window is None else max(0, p - window + 1)
    return torch.cat([torch.arange(min(sinks, lo)), torch.arange(lo, p + 1)])


def slots(t, window, sinks, T):
    return t if window is None else torch.where(t < T, t, sinks + (t - sinks) % (T - sinks))


def row(q, k, v, scale):
    """(o, tolerance) in 64 bits of one row q [Hq, D] over k, v [n, Hkv, D]."""
    Hq, D = q.shape
    n, Hkv, _ = k.shape
    G = Hq // Hkv
    qd, kd, vd = q.double().view(Hkv, G, D), k.double(), v.double()
    s = torch.einsum("hgd,nhd->hgn", qd, kd) * scale
    smax = (torch.einsum("hgd,nhd->hgn", qd.abs(), kd.abs()) * scale).amax(-1, keepdim=True)
    w = torch.softmax(s, -1)
    o = torch.einsum("hgn,nhd->hgd", w, vd)
    oabs = torch.einsum("hgn,nhd->hgd", w, vd.abs())
    half = HALF[q.dtype]
    ew = (D + 6) * E23 * smax + 2.0 ** -22
    tol = half * o.abs() + (half + 2 * ew + (2 * n + 64) * E23) * oabs
    if q.dtype is torch.float16:
        tol = tol + n * 2.0 ** -25 * vd.abs().amax(0).amax(-1)[:, None, None] + 2.0 ** -25
    return o.reshape(Hq, D), tol.reshape(Hq, D)


def close(got, want, tol, what):
    d = (got.double() - want).abs()
    assert bool((d <= tol).all()), f"{what}: worst {float((d / tol).nan_to_num(1e30).max()):.3g} tolerances"


def check_rows(o, q, keys, values, lives, scale, what=""):
    """o [B, M, Hq, D] against its definition.  keys(b, m), values(b, m): what row m of sequence b sees, [n, Hkv, D];
    lives(b, m): whether it sees anything (else zeros)."""
    B, M = q.shape[:2]
    for b in range(B):
        for m in range(M):
            if not lives(b, m):
                assert not o[b, m].any(), f"{what} row {b}, {m} is not zero"
                continue
            want, tol = row(q[b, m], keys(b, m), values(b, m), scale)
            close(o[b, m], want, tol, f"{what} row {b}, {m}")
