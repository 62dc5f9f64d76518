"""Outputs of the attention calls that share memory with another tensor are refused, wherever they begin; views that
interleave within one buffer are not."""
import itertools
import random

import pytest
import torch

import transformer_layer_pre_b200 as tlp
from test_attention_abi import AT, EINVAL, _desc

ES, D, N, S, B = 2, 64, 3, 33, 2
TOKEN, BATCH = N * D, S * N * D
SIZE = B * BATCH * ES


@pytest.fixture(scope="module")
def lib():
    return tlp.load_library()


def _call(lib, desc, at, strides, lse, ws, dtable=None, backward=True):
    """at: address of q, k, v, o, dO, dQ, dK, dV; strides: (batch, token, head) of each."""
    need = lib.tl_attention_workspace_bytes(desc, 1)
    v = [tlp._Heads(a, *s) for a, s in zip(at, strides)]
    if backward:
        return lib.tl_attention_backward(desc, *v[:5], lse, *v[5:], dtable, 0, ws, need, None)
    return lib.tl_attention_forward(desc, *v[:4], lse, ws, need, None)


def _far():
    return [AT * (16 + i) for i in range(8)], [(BATCH, TOKEN, D)] * 8, 40 * AT, 64 * AT


@pytest.mark.parametrize("move", [0, D * ES, -D * ES, TOKEN * ES, 5 * TOKEN * ES + D * ES, BATCH * ES, -BATCH * ES, SIZE - 16, 16 - SIZE])
@pytest.mark.parametrize("other", range(8))
def test_outputs_within_another_tensor(lib, move, other):
    """One head, token or sequence off, and the last 16 bytes of one over the first of the other."""
    for out in (5, 6, 7):
        if out == other:
            continue
        at, strides, lse, ws = _far()
        at[out] = at[other] + move
        assert _call(lib, _desc(), at, strides, lse, ws) == EINVAL
    if other < 3:
        at, strides, lse, ws = _far()
        at[3] = at[other] + move
        assert _call(lib, _desc(), at, strides, lse, ws, backward=False) == EINVAL


@pytest.mark.parametrize("other", range(8))
def test_statistics_table_and_workspace_within_a_tensor(lib, other):
    at, strides, lse, ws = _far()
    inside = at[other] + 7 * TOKEN * ES + 16
    if other < 4:
        assert _call(lib, _desc(), at, strides, inside, ws, backward=False) == EINVAL
    if other >= 5:                                          # lse is an input of the backward
        assert _call(lib, _desc(), at, strides, inside, ws) == EINVAL
    assert _call(lib, _desc(), at, strides, lse, ws, dtable=inside) == EINVAL
    assert _call(lib, _desc(), at, strides, lse, at[other] + 256) == EINVAL
    assert _call(lib, _desc(), at, strides, lse, lse - 256) == EINVAL
    assert _call(lib, _desc(bias_table=lse + 8), at, strides, lse, ws, backward=False) == EINVAL
    assert _call(lib, _desc(mask=lse + 8), at, strides, lse, ws, backward=False) == EINVAL
    assert _call(lib, _desc(mask=at[6] + 8), at, strides, lse, ws) == EINVAL
    assert _call(lib, _desc(bias_table=lse - 512), at, strides, lse, ws, dtable=lse - 512 + 4) == EINVAL


def _bytes(at, strides, shape, d):
    sb, st, sh = strides
    out = set()
    for b, s, n in itertools.product(*(range(x) for x in shape)):
        first = at + (b * sb + s * st + n * sh) * ES
        out.update(range(first, first + d * ES, 16))        # everything steps by 16 bytes
    return out


@pytest.mark.skipif(torch.cuda.is_available(), reason="calls that are taken would run on made-up addresses")
def test_random_views(lib):
    """Against the addresses themselves: o refused where it shares one with q, k or v, and only there."""
    rng = random.Random(5)
    refused = 0
    for _ in range(1500):
        shape = (rng.randint(1, 3), rng.randint(1, 4), rng.randint(1, 3))
        d = 8 * rng.randint(1, 3)
        desc = _desc(batch=shape[0], seq=shape[1], heads=shape[2], head_dim=d, bias_table=None)
        order = rng.sample(range(3), 3)
        step, strides = d * rng.randint(1, 4), [0, 0, 0]
        for i in order:                                     # an output steps over its inner dimensions
            strides[i] = step
            step = 8 * ((step * shape[i] + 8 * rng.randint(0, 9)) // 8)
        views = []
        for _ in range(3):
            same = rng.random() < 0.6
            views.append((AT * 16 + 16 * rng.randint(-60, 60),
                          tuple(strides) if same else tuple(8 * rng.randint(d // 8, 30) for _ in range(3))))
        o = _bytes(AT * 16, strides, shape, d)
        want = any(o & _bytes(a, s, shape, d) for a, s in views)
        at = [a for a, _ in views] + [AT * 16]
        got = _call(lib, desc, at, [s for _, s in views] + [tuple(strides)], 40 * AT, 64 * AT, backward=False)
        assert (got == EINVAL) == want
        refused += want
    assert 200 < refused < 1300


@pytest.mark.parametrize("odd", [0, -1, 3, (1 << 63) - 1, -(1 << 63)])
def test_strides_of_single_entries_mean_nothing(lib, odd):
    desc = _desc(batch=1, heads=1)
    at, _, lse, ws = _far()
    strides = [(odd, D, odd)] * 8
    at[3] = at[0] + 5 * D * ES
    assert _call(lib, desc, at, strides, lse, ws, backward=False) == EINVAL
    if not torch.cuda.is_available():          # else it would run on made-up addresses
        at[3] = at[0] + S * D * ES
        assert _call(lib, desc, at, strides, lse, ws, backward=False) != EINVAL


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("form", ["tokens", "heads", "sequences"])
def test_one_buffer_for_everything(dtype, form):
    """q, k, v, o, dO, dQ, dK and dV as views of one buffer: as results in tensors of their own."""
    b, s, n, d = 2, 150, 3, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    if form == "tokens":                                    # side by side in each token
        base = torch.randn(b, s, 8, n, d, generator=g, device="cuda").to(dtype)
        t = list(base.unbind(2))
    elif form == "heads":                                   # side by side in each head
        base = torch.randn(b, n, s, 8 * d, generator=g, device="cuda").to(dtype)
        t = [x.transpose(1, 2) for x in base.split(d, 3)]
    else:                                                   # a packed q, k, v and then the rest, for each sequence
        base = torch.randn(b, 8 * s * n * d, generator=g, device="cuda").to(dtype)
        t = list(base[:, :3 * s * n * d].unflatten(1, (s, 3, n, d)).unbind(2))
        t += list(base[:, 3 * s * n * d:].unflatten(1, (5, s, n, d)).unbind(1))
    assert all(x.shape == (b, s, n, d) and x.untyped_storage().data_ptr() == base.untyped_storage().data_ptr() for x in t)
    q, k, v, o, do, dq, dk, dv = t
    table = torch.randn(32, n, generator=g, device="cuda").to(dtype)
    o1, lse1 = tlp.attention_forward(q.contiguous(), k.contiguous(), v.contiguous(), None, table)
    want = tlp.attention_backward(q.contiguous(), k.contiguous(), v.contiguous(), o1, lse1, do.contiguous(), None, table)
    _, lse = tlp.attention_forward(q, k, v, None, table, o=o)
    got = tlp.attention_backward(q, k, v, o, lse, do, None, table, dq=dq, dk=dk, dv=dv)
    tlp.device_check()
    assert torch.equal(o, o1) and torch.equal(lse, lse1)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    with pytest.raises(tlp.TlError):
        tlp.attention_backward(q, k, v, o, lse, do, None, table, dq=dq, dk=dk, dv=dk)
