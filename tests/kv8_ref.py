"""The 8-bit key/value cache in 64 bits, position by position: what the
kernels are compared with."""
import math

import torch

MIN_E = -126
LIMIT = {"int8": 127.5, "e4m3": 448.0}
LARGEST = {torch.bfloat16: torch.finfo(torch.bfloat16).max, torch.float16: 65504.0, torch.float32: torch.finfo(torch.float32).max}


def step_exp(largest: float, fmt: str) -> int:
    """Smallest e >= -126 with largest <= limit * 2^e."""
    if largest <= 0:
        return MIN_E
    e = math.frexp(largest)[1] - 12
    while largest > math.ldexp(LIMIT[fmt], e):
        e += 1
    return max(e, MIN_E)


def round_codes(y: torch.Tensor, fmt: str) -> torch.Tensor:
    """Doubles in units of the step to the nearest code, ties to even."""
    if fmt == "int8":
        return torch.round(y).clamp(-127, 127)
    e = torch.frexp(y)[1].sub(1).clamp(min=-6)          # |y| = 1.f * 2^e
    ulp = torch.ldexp(torch.ones_like(y), e - 3)
    return torch.round(y / ulp) * ulp


def clean(x: torch.Tensor) -> torch.Tensor:
    """Infinities as the type's largest value, NaN as zero, in double."""
    d = x.double()
    return torch.where(d.isnan(), 0.0, d).clamp(-LARGEST[x.dtype], LARGEST[x.dtype])


class Ref:
    """codes (in units of the step) [2][B][G][T][D] and exponents [2][B][G][T / block]."""

    def __init__(self, batch, kv_heads, dim, T_cap, block, fmt):
        self.codes = torch.zeros((2, batch, kv_heads, T_cap, dim), dtype=torch.float64)
        self.exp = torch.full((2, batch, kv_heads, T_cap // block), MIN_E, dtype=torch.int64)
        self.block, self.fmt, self.T_cap = block, fmt, T_cap

    def values(self, which, b, g, n):
        e = self.exp[which, b, g].repeat_interleave(self.block)[:n]
        return self.codes[which, b, g, :n] * torch.ldexp(torch.ones(n, dtype=torch.float64), e)[:, None]

    def append(self, k_new, v_new, pos, counts=None):
        B, M = k_new.shape[:2]
        for which, new in enumerate((clean(k_new.cpu()), clean(v_new.cpu()))):
            for b in range(B):
                p = int(pos[b])
                if p < 0:
                    continue
                n = min(M if counts is None else max(0, min(int(counts[b]), M)), self.T_cap - p)
                for g in range(new.shape[2]):
                    for j in range(p // self.block, (p + n - 1) // self.block + 1 if n > 0 else 0):
                        t0 = j * self.block
                        a, z = max(t0, p), min(t0 + self.block, p + n)
                        x = new[b, a - p:z - p, g]
                        e = step_exp(float(x.abs().max()), self.fmt)
                        was = int(self.exp[which, b, g, j])
                        if a > t0:
                            e = max(e, was)
                            old = self.codes[which, b, g, t0:a]
                            self.codes[which, b, g, t0:a] = round_codes(old * 2.0 ** (was - e), self.fmt)
                        self.codes[which, b, g, a:z] = round_codes(x * 2.0 ** -e, self.fmt)
                        self.exp[which, b, g, j] = e

    def attend(self, q, pos, counts=None, scale=None):
        """(o, sum of w |v|, largest sum |q k| * scale) per row and head, and
        the weights [B][M][Hq][T]."""
        q = q.double().cpu()
        B, M, Hq, D = q.shape
        G = self.codes.shape[2]
        scale = D ** -0.5 if scale is None else scale
        o = torch.zeros((B, M, Hq, D), dtype=torch.float64)
        oabs, smax = torch.zeros_like(o), torch.zeros((B, M, Hq, 1), dtype=torch.float64)
        w = torch.zeros((B, M, Hq, self.T_cap), dtype=torch.float64)
        for b in range(B):
            p = int(pos[b])
            if p < 0:
                continue
            rows = min(M if counts is None else max(0, min(int(counts[b]), M)), self.T_cap - p)
            for g in range(G):
                k, v = self.values(0, b, g, p + max(rows, 0)), self.values(1, b, g, p + max(rows, 0))
                for m in range(rows):
                    for h in range(g * Hq // G, (g + 1) * Hq // G):
                        n = p + m + 1
                        x = torch.softmax(k[:n] @ q[b, m, h] * scale, 0)
                        w[b, m, h, :n] = x
                        o[b, m, h] = x @ v[:n]
                        oabs[b, m, h] = x @ v[:n].abs()
                        smax[b, m, h] = (k[:n].abs() @ q[b, m, h].abs()).max() * abs(scale)
        return o, oabs, smax, w

    def kept(self, n, acc, budget, sinks, recent):
        if n <= budget:
            return list(range(max(n, 0)))
        forced = sorted(set(range(sinks)) | set(range(n - recent, n)))
        rest = [t for t in range(sinks, n - recent)]
        rank = {t: (-math.inf if math.isnan(acc[t]) else acc[t]) for t in rest}
        nan = {t: math.isnan(acc[t]) for t in rest}
        rest.sort(key=lambda t: (nan[t], -rank[t], t))
        return sorted(forced + rest[:budget - len(forced)])

    def evict(self, dst, lens, acc, budget, sinks, recent):
        idx = [[self.kept(min(int(lens[b]), self.T_cap), acc[b, g].tolist(), budget, sinks, recent)
                for g in range(self.codes.shape[2])] for b in range(self.codes.shape[1])]
        for which in range(2):
            for b, heads in enumerate(idx):
                for g, keep in enumerate(heads):
                    x = self.values(which, b, g, self.T_cap)[keep]
                    for t0 in range(0, len(keep), self.block):
                        z = min(t0 + self.block, len(keep))
                        e = step_exp(float(x[t0:z].abs().max()), self.fmt)
                        dst.exp[which, b, g, t0 // self.block] = e
                        dst.codes[which, b, g, t0:z] = round_codes(x[t0:z] * 2.0 ** -e, self.fmt)
        return idx


def of_cache(cache) -> Ref:
    """The state of a KV8Cache as a Ref."""
    r = Ref(cache.batch, cache.kv_heads, cache.head_dim, cache.T_cap, cache.block, cache.fmt)
    for which, (c, s) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
        r.codes[which] = c.cpu().float().double()
        r.exp[which] = torch.frexp(s.cpu())[1].long() - 1
    return r
