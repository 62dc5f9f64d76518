"""A bias table that shuts buckets out (-inf): causal attention by the table alone, and rows that it leaves no key."""
import math

import pytest
import torch

import attention_ref as ref
import transformer_layer_pre_b200 as tlp
from test_gpu_attention import DT
from test_gpu_attention_gradient_sizes import _expected_rms

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("side", ["behind", "ahead"])
@pytest.mark.parametrize("s,d", [(2, 64), (100, 64), (128, 32), (700, 64), (1300, 40), (300, 128), (600, 128)])
def test_one_side_shut(dtype, side, s, d):
    """side: the keys that are left, the query's own among those behind it.  Error within twice the roundings' expected
    root mean square (float32: 1e-5 of the largest value); rows without a key: zeros, lse = +inf, zero gradients."""
    dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(s + d)
    b, n, c = 2, 3, d ** -0.5
    q, k, v, do = (torch.randn(b, s, n, d, generator=g, device="cuda").to(dt) for _ in range(4))
    table = torch.randn(32, n, generator=g, device="cuda")
    table[16:] = table[16:] if side == "ahead" else -math.inf
    table[:16] = table[:16] if side == "behind" else -math.inf
    table = table.to(dt)
    o, lse = tlp.attention_forward(q, k, v, None, table)
    got = dict(zip(("dq", "dk", "dv", "dtable"), tlp.attention_backward(q, k, v, o, lse, do, None, table)))
    tlp.device_check()
    ids = ref.bucket_matrix(s, 32, 128, "cuda")
    qq, kk, vv, oo, dd = (t.double().transpose(1, 2) for t in (q, k, v, o, do))
    x = c * qq @ kk.transpose(2, 3) + table.double().t()[:, ids]
    want_lse = torch.logsumexp(x, -1)
    empty = want_lse == -math.inf
    assert bool(empty.any()) == (side == "ahead")
    p = torch.where(empty[..., None], 0.0, torch.exp(x - torch.where(empty, 0.0, want_lse)[..., None]))
    assert torch.equal(lse == math.inf, empty)
    assert float((lse.double() - want_lse)[~empty].abs().max()) <= 2.0 ** -23 * (s / 64 + 80 * float(want_lse[~empty].abs().max() + 8))
    ds = p * (dd @ vv.transpose(2, 3) - (dd * oo).sum(-1, keepdim=True))
    val = {"o": (p @ vv).transpose(1, 2), "dq": (c * ds @ kk).transpose(1, 2),
           "dk": (c * ds.transpose(2, 3) @ qq).transpose(1, 2), "dv": (p.transpose(2, 3) @ dd).transpose(1, 2)}
    got["o"] = o
    u2 = ref.half_step(dt) ** 2 / 3
    rms = _expected_rms(dt, ds, p, qq, kk, dd, c, val)
    rms["o"] = (u2 * (((p ** 2) @ vv ** 2).transpose(1, 2) + val["o"] ** 2)).mean((1, 3)).sqrt()
    for name in ("o", "dq", "dk", "dv"):
        err = got[name].double() - val[name]
        if dtype == "f32":
            assert float(err.abs().max()) <= 1e-5 * float(val[name].abs().max()) + 1e-6, name
        else:
            # two keys at most: dS = P (dP - D) is a difference that D's own rounding of O reaches
            few = 2.0 * c * float(dd.abs().max()) * 2.0 ** -20
            assert bool(((err ** 2).mean((1, 3)).sqrt() <= 2 * rms[name] + few).all()), (name, (err ** 2).mean((1, 3)).sqrt(), rms[name])
    rows = empty.transpose(1, 2)
    assert bool((o[rows] == 0).all()) and bool((got["dq"][rows] == 0).all())
    want = torch.zeros(32, n, dtype=torch.float64, device="cuda").index_add_(0, ids.reshape(-1), ds.sum(0).reshape(n, -1).t())
    shut = torch.isinf(table)
    assert bool((got["dtable"][shut] == 0).all())
    size = torch.zeros(32, n, dtype=torch.float64, device="cuda").index_add_(
        0, ids.reshape(-1), (p * (dd.abs() @ vv.abs().transpose(2, 3) + (dd * oo).abs().sum(-1, keepdim=True))).sum(0).reshape(n, -1).t())
    assert bool((got["dtable"].double() - want).abs().le(size * 2.0 ** -23 * (2 * d + s * b + 80 * (float(x[x > -math.inf].abs().max()) + 8)) + 1e-30).all())
