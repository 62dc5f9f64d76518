"""The attention calls at the ends of what they take: the longest sequence, the most sequences, offsets beyond 32 bits."""
import math

import pytest
import torch

import attention_ref as ref
import transformer_layer_pre_b200 as tlp
from test_gpu_attention import DT, _check

pytestmark = pytest.mark.gpu


def test_longest_sequence():
    """2^20 tokens of 8 dims, float16, with a bias: sampled rows and keys, first and last among them, in float64.
    Bounds as in attention_ref, with its sums over 2^20 terms: u for P, dS and the results (half a step), 2^-23 for each of
    seq / 16 accumulated products (the unit adds 16 at a time) and seq / 64 tile sums, e for the exponent."""
    s, d, c = 1 << 20, 8, 8 ** -0.5
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, do = (torch.randn(1, s, 1, d, generator=g, device="cuda").half() for _ in range(4))
    table = torch.randn(32, 1, generator=g, device="cuda").half()
    o, lse = tlp.attention_forward(q, k, v, None, table)
    dq, dk, dv, dtable = tlp.attention_backward(q, k, v, o, lse, do, None, table)
    tlp.device_check()
    Q, K, V, O, G = (t[0, :, 0].double() for t in (q, k, v, o, do))
    L, T = lse[0, 0].double(), table[:, 0].double()
    near = torch.tensor([ref.bucket(r, 32, 128) for r in range(-200, 201)], device="cuda")
    pick = torch.cat([torch.tensor([0, 1, 127, 128, s // 2, s - 129, s - 2, s - 1], device="cuda"),
                      torch.randint(0, s, (24,), generator=g, device="cuda")])
    pos = torch.arange(s, device="cuda")
    u, w = 2.0 ** -11, 2.0 ** -23
    D = (G * O).sum(1)
    for i in pick.tolist():
        bias = T[near[(pos - i).clamp(-200, 200) + 200]]
        x = c * (K @ Q[i]) + bias
        total = torch.logsumexp(x, 0)
        assert abs(float(L[i] - total)) <= (s / 64 + 200) * w + 32 * w
        p = torch.exp(x - L[i])
        e = 16 * w * (c * K.abs() @ Q[i].abs() + bias.abs() + 14) + (s / 64) * w
        tol = ((u + e + (s / 16) * w) * p) @ V.abs() + u * O[i].abs() + 2.0 ** -25
        assert bool(((p @ V) - O[i]).abs().le(tol).all()), i
        ds = p * (V @ G[i] - D[i])
        size = p * (V.abs() @ G[i].abs() + (G[i] * O[i]).abs().sum())
        want = c * (ds @ K)
        tol = c * (((u + (s / 16) * w) * ds.abs() + (e + 12 * w) * size) @ K.abs()) + u * want.abs() + 2.0 ** -25
        assert bool((want - dq[0, i, 0].double()).abs().le(tol).all()), i
        # key i: the queries are the others
        bias = T[near[(i - pos).clamp(-200, 200) + 200]]
        x = c * (Q @ K[i]) + bias
        p = torch.exp(x - L)
        e = 16 * w * (c * Q.abs() @ K[i].abs() + bias.abs() + 14) + (s / 64) * w
        ds = p * (G @ V[i] - D)
        size = p * (G.abs() @ V[i].abs() + (G * O).abs().sum(1))
        want = c * (ds @ Q)
        tol = c * (((u + (s / 16) * w) * ds.abs() + (e + 12 * w) * size) @ Q.abs()) + u * want.abs() + 2.0 ** -25
        assert bool((want - dk[0, i, 0].double()).abs().le(tol).all()), i
        want = p @ G
        tol = ((u + e + (s / 16) * w) * p) @ G.abs() + u * want.abs() + 2.0 ** -25
        assert bool((want - dv[0, i, 0].double()).abs().le(tol).all()), i
    assert bool(torch.isfinite(dtable).all())


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_most_sequences(dtype):
    """2^23 sequences and heads of one token: P = 1, so O = V, dV = dO (exactly but for the rounding of 2^-x to 1), and
    dS = 0 but for the rounding of dP - D: d products of each, their bound |dO||V| times (d + 4) places."""
    b, n, d = 1 << 19, 16, 8
    g = torch.Generator(device="cuda").manual_seed(2)
    dt = DT[dtype]
    q, k, v, do = (torch.randn(b, 1, n, d, generator=g, device="cuda").to(dt) for _ in range(4))
    table = torch.randn(32, n, generator=g, device="cuda").to(dt)
    o, lse = tlp.attention_forward(q, k, v, None, table)
    dq, dk, dv, dtable = tlp.attention_backward(q, k, v, o, lse, do, None, table)
    tlp.device_check()
    w = 2.0 ** -23
    u = ref.half_step(dt)
    qf, kf, vf, gf = (t.float() for t in (q, k, v, do))
    x = d ** -0.5 * (qf * kf).sum(-1) + table[0].float()
    size = d ** -0.5 * (qf * kf).abs().sum(-1) + table[0].float().abs() + 1
    assert bool((lse[:, :, 0] - x[:, 0]).abs().le(16 * w * size[:, 0]).all())
    close = (2 * u + 24 * w * size + 8 * w)[..., None]
    assert bool((o.float() - vf).abs().le(close * vf.abs() + 2.0 ** -24).all())
    assert bool((dv.float() - gf).abs().le(close * gf.abs() + 2.0 ** -24).all())
    off = (gf * vf).abs().sum(-1) * ((d + 4) * w + 1.01 * u + 24 * w * size)     # O = V rounded once more
    for got, other in ((dq, kf), (dk, qf)):
        assert bool(got.float().abs().le((1 + 2 * u) * d ** -0.5 * off[..., None] * other.abs() + 2.0 ** -24).all())
    # the float64 sum of every |dS| bounds bucket 0's gradient; no other bucket has an entry
    assert bool(dtable[1:].eq(0).all()) and bool(dtable[0].abs().double().le(off[:, 0].double().sum(0) + 1e-6).all())


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_offsets_beyond_32_bits(dtype):
    """Sequences 2^31 + 64 elements apart, and heads 2^31 + 64 apart: as dense."""
    b, s, n, d = 2, 200, 2, 64
    far = (1 << 31) + 64
    dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v, do = (torch.randn(b, s, n, d, generator=g, device="cuda").to(dt) for _ in range(4))
    table = torch.randn(32, n, generator=g, device="cuda").to(dt)
    o, lse = tlp.attention_forward(q, k, v, None, table)
    want = tlp.attention_backward(q, k, v, o, lse, do, None, table)
    base = torch.empty(far + 8 * s * n * d, dtype=dt, device="cuda")
    places = iter(range(8))

    def spread(t, strides):
        x = base.as_strided((b, s, n, d), strides, next(places) * s * n * d)
        if t is not None:
            x.copy_(t)
        return x

    for strides in ((far, n * d, d, 1), (s * d, d, far, 1)):
        places = iter(range(8))
        x = [spread(t, strides) for t in (q, k, v, None, do, None, None, None)]
        _, lse1 = tlp.attention_forward(x[0], x[1], x[2], None, table, o=x[3])
        got = tlp.attention_backward(*x[:4], lse1, x[4], None, table, dq=x[5], dk=x[6], dv=x[7])
        tlp.device_check()
        assert torch.equal(x[3], o) and torch.equal(lse1, lse)
        assert all(torch.equal(i, j) for i, j in zip(got, want))
