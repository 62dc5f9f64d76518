"""Long rows in which one key outweighs each of the others, which together weigh about as much: their probabilities are
float16 subnormals relative to the row's maximum."""
import math

import pytest
import torch

import attention_ref as ref
import transformer_layer_pre_b200 as tlp
from test_gpu_attention import DT, _check

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


def _finite_masks(dtype, value, s, d):
    """Masks that remove nothing: over a whole sequence, over its first half (the running reference starts there), and in
    steps of a quarter of the value (it climbs)."""
    g = torch.Generator(device="cuda").manual_seed(s)
    q, k, v, do = (torch.randn(3, s, 2, d, generator=g, device="cuda").to(DT[dtype]) for _ in range(4))
    table = torch.randn(32, 2, generator=g, device="cuda").to(DT[dtype])
    m = torch.zeros(3, s, device="cuda")
    m[0] = value
    m[1, : s // 2] = value
    m[2] = value * (1 - (4 * torch.arange(s, device="cuda") // s) / 4)
    return q, k, v, do, m, table


FINITE = [(dt, x, s, d) for dt in ("f32", "f16", "bf16") for x in (-1e4, -1e6, -3e7, -1e8, -1e9, -1e29)
          for s, d in ((100, 64), (600, 64), (300, 128))]


@pytest.mark.parametrize("dtype,value,s,d", FINITE)
def test_forward_under_finite_masks(dtype, value, s, d):
    """Within the bounds, which grow with |mask|, and finite."""
    q, k, v, _, m, table = _finite_masks(dtype, value, s, d)
    for t in (None, table):
        o, lse = tlp.attention_forward(q, k, v, m, t)
        tlp.device_check()
        assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(lse).all())
        want, tol = ref.forward(q, k, v, m, t)
        _check("o", o, want["o"], tol["o"])
        _check("lse", lse, want["lse"], tol["lse"])
        # a float32 lse holds log2 of the sum to half a last place of its own size, whatever the reference was
        whole = lse[0].double() - value
        assert float((whole - (want["lse"][0] - value)).abs().max()) <= 16 * 2.0 ** -24 * abs(value) + 2.0 ** -17


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_that_float32_rounds_by_whole_units(dtype, d):
    """Scores of 2^21 to 2^27 with steps between the keys, and a bias: P stays finite in float16."""
    g = torch.Generator(device="cuda").manual_seed(d)
    s = 520
    for size in (2.0 ** 21, 2.0 ** 24, 2.0 ** 27):
        q = torch.full((1, s, 2, d), 64.0, device="cuda")
        k = (size / (64 * d)) * (1 + torch.arange(s, device="cuda") / s * 2.0 ** -9)[None, :, None, None].expand(1, s, 2, d)
        v = torch.randn(1, s, 2, d, generator=g, device="cuda")
        table = 3 * torch.randn(32, 2, generator=g, device="cuda")
        q, k, v, table = (t.to(DT[dtype]).contiguous() for t in (q, k, v, table))
        for t in (None, table):
            o, lse = tlp.attention_forward(q, k, v, None, t, scale=1.0)
            tlp.device_check()
            assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(lse).all())
            assert float(o.abs().max()) <= float(v.abs().max()) * (1 + 2.0 ** -6)


@pytest.mark.parametrize("dtype,value,s,d", FINITE)
def test_backward_under_finite_masks(dtype, value, s, d):
    """Finite, and within the bounds, which grow with |mask| and |lse|: where a place of lse is worth more than a factor
    of the probabilities they bound nothing else."""
    q, k, v, do, m, table = _finite_masks(dtype, value, s, d)
    for t in (None, table):
        o, lse = tlp.attention_forward(q, k, v, m, t)
        grads = dict(zip(("dq", "dk", "dv", "dtable"), tlp.attention_backward(q, k, v, o, lse, do, m, t)))
        tlp.device_check()
        if t is None:
            assert grads.pop("dtable") is None
        for name, x in grads.items():
            assert bool(torch.isfinite(x).all()), name
        want, tol = ref.backward(q, k, v, o, lse, do, m, t)
        for name, x in grads.items():
            _check(name, x, torch.nan_to_num(want[name], 0.0, 0.0, 0.0), torch.nan_to_num(tol[name], math.inf, math.inf))
        # the sequence that masks only its first half (and its gradients) is as if those keys were removed
        if value <= -1e6:
            gone = m[1:2].clone()
            gone[gone < 0] = -math.inf
            one = [x[1:2].contiguous() for x in (q, k, v)]
            o1, lse1 = tlp.attention_forward(*one, gone, t)
            want = tlp.attention_backward(*one, o1, lse1, do[1:2].contiguous(), gone, t)
            tlp.device_check()
            assert float((o[1:2] - o1).abs().max()) <= 2 * torch.finfo(o1.dtype).eps * float(o1.abs().max())
            for name, y in zip(("dq", "dk", "dv"), want):
                assert float((grads[name][1:2].double() - y.double()).abs().max()) <= 2.0 ** -6 * float(y.double().abs().max())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("s,d", [(100, 64), (300, 128)])
def test_gradients_are_finite_under_any_finite_mask(dtype, s, d):
    """A whole row masked by a finite value: among them ones whose lse, rounded, lies a place below the scores."""
    g = torch.Generator(device="cuda").manual_seed(s)
    q, k, v, do = (torch.randn(1, s, 2, d, generator=g, device="cuda").to(DT[dtype]) for _ in range(4))
    for value in [-1.36e8, -1.41e8] + [-10.0 ** (4 + 0.1 * i + 0.001 * j) for i in range(259) for j in (0, 37)]:
        m = torch.full((1, s), value, device="cuda")
        o, lse = tlp.attention_forward(q, k, v, m)
        grads = tlp.attention_backward(q, k, v, o, lse, do, m)[:3]
        assert all(bool(torch.isfinite(x).all()) for x in (o, *grads)), value
    tlp.device_check()
