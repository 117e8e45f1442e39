"""GPU tests of the 8-bit key/value cache at the limits of its numbers."""
import pytest
import torch

import quantized_moe_decode_layer_gb300 as moe
from test_gpu_kv8 import DEV, gen, i32, rows

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
