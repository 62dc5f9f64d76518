"""The float64 reference of the attention calls: its gradients against central
differences and against autograd, and its buckets against the closed form."""
import math

import pytest
import torch

import attention_ref as ref


def _inputs(mask_kind):
    g = torch.Generator().manual_seed(3)
    b, s, n, d, u = 2, 6, 2, 8, 8
    q, k, v, do = (torch.randn(b, s, n, d, generator=g, dtype=torch.float64) for _ in range(4))
    table = torch.randn(u, n, generator=g, dtype=torch.float64)
    mask = None
    if mask_kind == "holes":
        mask = torch.zeros(b, s, dtype=torch.float32)
        mask[0, 2] = -math.inf
        mask[1, 4:] = torch.finfo(torch.float32).min
        mask[1, 0] = 0.5
    elif mask_kind == "empty":
        mask = torch.zeros(b, s, dtype=torch.float32)
        mask[0] = -math.inf
    return q, k, v, do, table, mask


@pytest.mark.parametrize("mask_kind", ["none", "holes", "empty"])
def test_gradients_against_differences(mask_kind):
    q, k, v, do, table, mask = _inputs(mask_kind)

    def loss(q, k, v, table):
        return float((ref.forward(q, k, v, mask, table, 4)[0]["o"] * do).sum())

    out = ref.forward(q, k, v, mask, table, 4)[0]
    got, _ = ref.backward(q, k, v, out["o"], out["lse"], do, mask, table, 4)
    g = torch.Generator().manual_seed(5)
    h = 1e-5
    for i, name in enumerate(("dq", "dk", "dv", "dtable")):
        args = [q, k, v, table]
        step = torch.randn(args[i].shape, generator=g, dtype=torch.float64)
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + h * step, args[i] - h * step
        diff = (loss(*hi) - loss(*lo)) / (2 * h)
        want = float((got[name] * step).sum())
        # central differences: O(h^2) = 1e-10 of third derivatives of order 10, and 1e-16 / h of rounding
        assert abs(diff - want) <= 1e-7 * max(1.0, abs(want)), name


@pytest.mark.parametrize("buckets,distance", [(4, 2), (8, 64), (32, 128), (64, 300), (256, 1024)])
def test_buckets_against_the_closed_form(buckets, distance):
    half, first = buckets // 2, buckets // 4
    for rel in range(-2 * distance, 2 * distance + 1):
        n = abs(rel)
        far = first + math.floor(math.log(max(n, 1) / first) / math.log(distance / first) * (half - first) + 1e-9)
        want = (n if n < first else min(far, half - 1)) + (half if rel > 0 else 0)
        assert ref.bucket(rel, buckets, distance) == want, rel
