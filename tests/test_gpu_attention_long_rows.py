"""Long rows in which one key outweighs each of the others, which together weigh about as much: their probabilities are
float16 subnormals relative to the row's maximum."""
import math

import pytest
import torch

import transformer_layer_pre_b200 as tlp
from test_gpu_attention import DT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [8, 96])
@pytest.mark.parametrize("first", [True, False])
def test_many_small_probabilities_next_to_a_large_one(dtype, d, first):
    """Scores 12.5 for one key and 0 for the others: P = e^-12.5 = 62.5 * 2^-24 relative to the maximum, so that its
    rounding in float16 would be 2^-7 of it for all of them alike.  V is 0 at the one key and 1 at the others.
    Bound, relative: P and O rounded, u each; float32 sums, one last place (2^-23) for each of seq / 16 products and for
    each of seq / 64 tile sums; 2^-17 for the exponentials (2^-22 each, and 13 last places of 12.5 log2 e)."""
    s, dt = 150469, DT[dtype]
    k = torch.zeros(1, s, 1, d, device="cuda", dtype=dt)
    v = torch.ones_like(k)
    one = 0 if first else s - 1
    k[0, one, 0, 0] = 12.5
    v[0, one] = 0
    q = torch.zeros_like(k)
    q[..., 0] = 1
    o, lse = tlp.attention_forward(q, k, v, scale=1.0)
    tlp.device_check()
    rest = (s - 1) * math.exp(-12.5)
    u = torch.finfo(dt).eps / 2
    want = rest / (1 + rest)
    assert float((o.double() - want).abs().max()) <= want * (2 * u + (s / 16 + s / 64) * 2.0 ** -23 + 2.0 ** -17)
    assert float((lse.double() - 12.5 - math.log(1 + rest)).abs().max()) <= (s / 64) * 2.0 ** -23 + 16 * 2.0 ** -23 * 13
