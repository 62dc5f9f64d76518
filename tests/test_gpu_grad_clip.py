"""clip_grad_norm on the GPU against the formula in float64."""
import math

import pytest
import torch

import transformer_layer_pre_b200 as tlp

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _make(dtype, sizes, seed=0, std=0.02, offset=0):
    """Views of one flat buffer that start `offset` elements into it."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    flat = (std * torch.randn(sum(sizes) + offset, generator=g, device="cuda")).to(DT[dtype])
    return list(flat[offset:].split(sizes)), flat


def _verify(grads, limit, norm, outs, dtype):
    """norm: float64 sums and root, one float32 rounding (and the last places of a reordered float64 sum): 2^-23.
    out: one rounded factor (2^-24) and product (2^-24 more in float32), then the storage rounding, half a step."""
    total = math.sqrt(sum(float(t.double().square().sum()) for t in grads))
    assert abs(float(norm) - total) <= 2.0 ** -23 * total
    coef = min(1.0, limit / (total + 1e-6))
    u = torch.finfo(DT[dtype]).eps / 2
    for t, o in zip(grads, outs):
        want = t.double() * coef
        tol = want.abs() * (u + 2.0 ** -22) + (2.0 ** -25 if dtype == "f16" else 1e-45)
        assert bool(((o.double() - want).abs() <= tol).all())
        if coef == 1.0:
            assert torch.equal(o, t)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("sizes", [[1], [7], [8, 0, 3], [5, 1, 1, 33, 127], [8192], [8191, 8193, 4097], [100000, 3, 250001],
                                   [3] * 25, [70] * 321, [11] * 1001, [2] * 2003, [3_000_000, 12345]])
@pytest.mark.parametrize("limit", [1e-3, 1e9])
def test_sizes_and_alignments(dtype, sizes, limit):
    for offset in (0, 1, 5):
        grads, flat = _make(dtype, sizes, offset=offset)
        outs, oflat = _make(dtype, sizes, seed=1, offset=offset)
        keep = flat.clone()
        norm = tlp.clip_grad_norm(grads, limit, out=outs)
        assert torch.equal(flat, keep)
        _verify(grads, limit, norm, outs, dtype)
        other, _ = _make(dtype, sizes, seed=2, offset=offset + 1)      # aligned differently
        tlp.clip_grad_norm(grads, limit, out=other)
        assert all(torch.equal(a, b) for a, b in zip(outs, other))
        again = tlp.clip_grad_norm(grads, limit)                          # in place
        assert torch.equal(again, norm) and all(torch.equal(a, b) for a, b in zip(outs, grads))
    tlp.device_check()


@pytest.mark.parametrize("std", [1e-30, 1e-20, 1e18, 1e30])
def test_squares_outside_float32(std):
    grads, _ = _make("f32", [1000, 4097], std=std)
    outs, _ = _make("f32", [1000, 4097])
    limit = 0.5 * std
    norm = tlp.clip_grad_norm(grads, limit, out=outs)
    _verify(grads, limit, norm, outs, "f32")


def test_limits():
    grads, flat = _make("f32", [5000, 77])
    keep = flat.clone()
    norm = tlp.clip_grad_norm(grads, math.inf)
    assert torch.equal(flat, keep) and float(norm) > 0
    tlp.clip_grad_norm(grads, 0.0)
    assert bool((flat == 0).all())
    assert float(tlp.clip_grad_norm(grads, 1.0)) == 0.0 and bool((flat == 0).all())


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_not_finite(bad):
    grads, flat = _make("f32", [5000, 77])
    flat[4321] = bad
    norm = tlp.clip_grad_norm(grads, 1.0)
    assert not math.isfinite(float(norm))
    if math.isnan(bad):
        assert bool(torch.isnan(flat).all())
    else:                                   # factor 0: 0 * inf is the one NaN
        assert math.isnan(float(flat[4321])) and int((flat == 0).sum()) == flat.numel() - 1


@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_measuring_only_changes_nothing(bad):
    grads, flat = _make("f32", [5000, 77])
    flat[4321] = bad
    keep = flat.clone()
    norm = tlp.clip_grad_norm(grads, math.inf)
    assert not math.isfinite(float(norm)) and torch.equal(flat.view(torch.int32), keep.view(torch.int32))


def test_graph_and_streams_repeat_bitwise():
    sets = [_make("f32", [200001, 5, 64], seed=s) for s in range(2)]
    want = []
    for grads, _ in sets:
        outs = [torch.empty_like(t) for t in grads]
        want.append((tlp.clip_grad_norm(grads, 0.1, out=outs), outs))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for st, (grads, _) in zip(streams, sets):
            with torch.cuda.stream(st):
                outs = [torch.empty_like(t) for t in grads]
                got.append((tlp.clip_grad_norm(grads, 0.1, out=outs), outs))
        torch.cuda.synchronize()
        for (n0, o0), (n1, o1) in zip(want, got):
            assert torch.equal(n0, n1) and all(torch.equal(a, b) for a, b in zip(o0, o1))
    static, flat = _make("f32", [200001, 5, 64])
    outs = [torch.empty_like(t) for t in static]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = tlp.clip_grad_norm(static, 0.1, out=outs)
    for (_, src), (n0, o0) in list(zip(sets, want)) * 2:
        flat.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, n0) and all(torch.equal(a, b) for a, b in zip(outs, o0))


def test_python_refusals():
    t = torch.zeros(8, 8, device="cuda")
    bad = [
        lambda: tlp.clip_grad_norm([t, t.half()], 1.0),
        lambda: tlp.clip_grad_norm([t, t.cpu()], 1.0),
        lambda: tlp.clip_grad_norm([t.t()[:4]], 1.0),
        lambda: tlp.clip_grad_norm([t.int()], 1.0),
        lambda: tlp.clip_grad_norm([t], -1.0),
        lambda: tlp.clip_grad_norm([t], math.nan),
        lambda: tlp.clip_grad_norm([t], 1.0, out=[]),
        lambda: tlp.clip_grad_norm([t], 1.0, out=[torch.zeros(8, device="cuda")]),
        lambda: tlp.clip_grad_norm([t], 1.0, out=[t.half()]),
    ]
    for f in bad:
        with pytest.raises(tlp.TlError):
            f()
