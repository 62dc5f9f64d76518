"""The attention backward on padded batches whose items go on, within one block, between rows with keys and without
any: against the float64 reference within its elementwise bounds (attention_ref), and the same bits on every repeat."""
import math

import pytest
import torch

import attention_ref as ref
import transformer_layer_pre_b200 as tlp
from test_gpu_attention import DT, _check

pytestmark = pytest.mark.gpu


def _padded(b, s, order, g):
    """Sequences of no key, of 1 to 64, of about half and of all, whole 128-key runs removed in the last kind."""
    m = torch.zeros(b, s, device="cuda")
    at = torch.arange(s, device="cuda")
    for i in range(b):
        kind = order[i % len(order)]
        if kind == "none":
            m[i] = -math.inf
        elif kind == "few":
            m[i, int(torch.randint(1, 65, (1,), generator=g, device="cuda")):] = -math.inf
        elif kind == "half":
            m[i, s // 2 + int(torch.randint(0, 70, (1,), generator=g, device="cuda")):] = -math.inf
        elif kind == "runs":
            m[i, (at // 128) % 2 == 0] = torch.finfo(torch.float32).min
    return m


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("buckets", [0, 32])
@pytest.mark.parametrize("b,s,n,d,order", [
    # three buffers of scores (head dims up to 64, more than 1024 tokens), several items to a block
    (7, 1025, 4, 64, ("few", "all", "none", "runs", "half")),
    (6, 1100, 5, 48, ("half", "none", "few", "none", "all", "none")),
    (3, 2048, 12, 64, ("half", "runs", "none")),
    (4, 2090, 6, 64, ("none", "few", "half", "none")),
    # two buffers
    (9, 520, 10, 64, ("few", "none", "half", "runs", "all", "none")),
    (5, 1100, 7, 128, ("few", "all", "none", "runs", "half")),
])
def test_items_with_and_without_keys(dtype, buckets, b, s, n, d, order):
    g = torch.Generator(device="cuda").manual_seed(s + d)
    dt = DT[dtype]
    q, k, v, do = (torch.randn(b, s, n, d, generator=g, device="cuda").to(dt) for _ in range(4))
    table = torch.randn(buckets, n, generator=g, device="cuda").to(dt) if buckets else None
    m = _padded(b, s, order, g)
    o, lse = tlp.attention_forward(q, k, v, m, table)
    first = tlp.attention_backward(q, k, v, o, lse, do, m, table)
    for _ in range(8):
        again = tlp.attention_backward(q, k, v, o, lse, do, m, table)
        assert all(x is y or torch.equal(x, y) for x, y in zip(first, again))
    tlp.device_check()
    for i in range(b):                      # one sequence at a time: the reference holds (heads, s, s) in float64
        one = [t[i:i + 1] for t in (q, k, v, o, lse, do, m)]
        want, tol = ref.forward(*one[:3], one[6], table)
        _check("o", one[3], want["o"], tol["o"])
        _check("lse", one[4], want["lse"], tol["lse"])
        want, tol = ref.backward(*one[:6], one[6], table)
        for name, t in zip(("dq", "dk", "dv"), first):
            _check(name, t[i:i + 1], want[name], tol[name])
        if buckets:
            total = (want["dtable"], tol["dtable"]) if i == 0 else (total[0] + want["dtable"], total[1] + tol["dtable"])
    if buckets:
        # the sum over the sequences is float64, rounded once
        _check("dtable", first[3], total[0], total[1] + ref.W * total[0].abs())
