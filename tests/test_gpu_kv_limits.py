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
