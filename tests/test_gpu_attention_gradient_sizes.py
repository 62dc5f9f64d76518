"""The 16-bit attention backward on gradients of any size: dS is as small as the gradient that comes in times a
probability, and float16 has 11 bits only between 2^-14 and 65504.  u is half a step of one rounding of the type,
2^-25 half of float16's smallest step."""
import math

import pytest
import torch

import attention_ref as ref
import transformer_layer_pre_b200 as tlp
from test_gpu_attention import DT, _check, _mask

pytestmark = pytest.mark.gpu

SIZES = [(2, 128, 2, 64), (2, 90, 3, 40), (2, 256, 2, 64), (1, 200, 2, 24), (1, 512, 2, 128), (1, 1536, 1, 128), (1, 2048, 2, 64)]


@pytest.mark.parametrize("s,d", [(128, 64), (256, 64), (1024, 64), (2048, 64), (4096, 32), (512, 128), (2048, 128)])
def test_equal_small_entries(s, d):
    """Scores 0, P = 1/s; keys and values of alternating sign make every dS +-14.5 of float16's smallest steps and all of
    their roundings the same: dQ = c d x y on the first half of the dims, dK = +-c d x y on the other.
    Bound: dS and the result rounded, u each; float32 terms below 2^-12 (the exponential of lse = log s, at most 8.4: 80
    last places of 2^-23 of it, 2^-14; a sum of s / 16 products, 2^-15; the d products of dP, 2^-16); 2^-25 where the
    result is subnormal itself."""
    x = float(torch.tensor(14.5 / 128).half())
    y = 2.0 ** -13 * s / 1024 * 64 / d                    # d x y / s = 14.5 * 2^-24
    sign = torch.ones(1, s, 1, 1, device="cuda")
    sign[:, 1::2] = -1
    lower = (torch.arange(d, device="cuda") < d // 2).float()
    q = (1 - lower).expand(1, s, 1, d).half().contiguous()
    k = (sign * lower).half().contiguous()
    v = (sign * x).expand(1, s, 1, d).half().contiguous()
    do = torch.full((1, s, 1, d), y, device="cuda").half()
    assert float(do[0, 0, 0, 0]) == y
    o, lse = tlp.attention_forward(q, k, v)
    dq, dk, dv, _ = tlp.attention_backward(q, k, v, o, lse, do)
    tlp.device_check()
    want = d ** -0.5 * d * x * y
    tol = want * (2 * 2.0 ** -11 + 2.0 ** -12) + 2.0 ** -25
    assert float((dq.double() - want * lower.double()).abs().max()) <= tol
    assert float((dk.double() - want * (sign * (1 - lower)).double()).abs().max()) <= tol
    assert float((dv.double() - y).abs().max()) <= y * (2 * 2.0 ** -11 + 2.0 ** -12) + 2.0 ** -25


def _expected_rms(dtype, ds, p, q, k, do, c, val):
    """Root mean square of the roundings' sum: each is uniform within half a step, at most u of its value, so of a variance
    of at most u^2 / 3 of its square; signs do not depend on one another."""
    u2 = (torch.finfo(dtype).eps / 2) ** 2 / 3
    sub = (2.0 ** -25) ** 2 / 3 if dtype == torch.float16 else 0.0
    var = {"dq": c * c * (ds ** 2) @ k ** 2, "dk": c * c * (ds ** 2).transpose(2, 3) @ q ** 2, "dv": (p ** 2).transpose(2, 3) @ do ** 2}
    return {n: (u2 * (var[n].transpose(1, 2) + val[n] ** 2) + sub).mean((1, 3)).sqrt() for n in var}


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", [100.0, 1e-2, 1e-3, 1e-4])
@pytest.mark.parametrize("b,s,n,d", SIZES)
def test_relative_error_at_any_size(dtype, size, b, s, n, d):
    """Random tensors: the error of every sequence and head within twice the expected root mean square, which the mean of
    thousands of roundings does not leave.  Padded keys hold large values, a second sequence gradients 1000 times smaller,
    a second head values 30 times larger."""
    dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(s + d)
    q, k, v, do = (torch.randn(b, s, n, d, generator=g, device="cuda") for _ in range(4))
    m = torch.zeros(b, s, device="cuda")
    m[:, s - s // 7:] = -math.inf
    do *= size
    do[1:] *= 1e-3
    v[:, :, 1:] *= 30
    v[:, s - s // 7:] = 5e4
    q, k, v, do = (t.to(dt) for t in (q, k, v, do))
    table = torch.randn(32, n, generator=g, device="cuda").to(dt)
    o, lse = tlp.attention_forward(q, k, v, m, table)
    got = dict(zip(("dq", "dk", "dv", "dtable"), tlp.attention_backward(q, k, v, o, lse, do, m, table)))
    tlp.device_check()
    val, tol = ref.backward(q, k, v, o, lse, do, m, table)
    c = d ** -0.5
    x, _ = ref.scores(q, k, m, table, 128, c)
    p = torch.exp(x - lse.double()[..., None])
    qq, kk, vv, oo, dd = (t.double().transpose(1, 2) for t in (q, k, v, o, do))
    ds = p * (dd @ vv.transpose(2, 3) - (dd * oo).sum(-1, keepdim=True))
    rms = _expected_rms(dt, ds, p, qq, kk, dd, c, val)
    for name in ("dq", "dk", "dv"):
        err = ((got[name].double() - val[name]) ** 2).mean((1, 3)).sqrt()
        assert bool((err <= 2 * rms[name]).all()), (name, (err / rms[name]).tolist())
    _check("dtable", got["dtable"], val["dtable"], tol["dtable"])


@pytest.mark.parametrize("b,s,n,d,size", [(2, 16, 2, 64, 40.0), (1, 300, 2, 128, 400.0), (1, 1200, 1, 64, 2000.0)])
def test_entries_beyond_the_largest_float16(b, s, n, d, size):
    """dS up to several times 65504, gradients that float16 holds: small queries and keys."""
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v, do = (torch.randn(b, s, n, d, generator=g, device="cuda") for _ in range(4))
    q, k, v, do = (0.02 * q).half(), (0.02 * k).half(), (size * v).half(), (4000 * do).clamp(-16000, 16000).half()
    o, lse = tlp.attention_forward(q, k, v)
    got = tlp.attention_backward(q, k, v, o, lse, do)
    tlp.device_check()
    val, tol = ref.backward(q, k, v, o, lse, do)
    for name, t in zip(("dq", "dk", "dv"), got):
        assert float(val[name].abs().max()) < 60000
        _check(name, t, val[name], tol[name])


@pytest.mark.parametrize("s,d", [(100, 64), (300, 64), (200, 128)])
def test_no_gradient(s, d):
    """dO = 0, and one sequence of it among others: zero gradients, no NaN."""
    g = torch.Generator(device="cuda").manual_seed(4)
    q, k, v, do = (torch.randn(2, s, 2, d, generator=g, device="cuda").half() for _ in range(4))
    table = torch.randn(32, 2, generator=g, device="cuda").half()
    do[0] = 0
    m = _mask("empty", 2, s, g)
    for mask in (None, m):
        o, lse = tlp.attention_forward(q, k, v, mask, table)
        out = tlp.attention_backward(q, k, v, o, lse, do, mask, table)
        tlp.device_check()
        assert all(bool(torch.isfinite(t).all()) and bool((t[0] == 0).all()) for t in out[:3])
        assert bool(torch.isfinite(out[3]).all()) and (mask is None or bool((out[3] == 0).all()))
