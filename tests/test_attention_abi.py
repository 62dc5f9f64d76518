"""Refusals of the attention and clipping entry points (no GPU: every argument
error is reported before anything is enqueued), and of their Python calls."""
import ctypes

import pytest
import torch

import transformer_layer_pre_b200 as tlp

OK, EINVAL, EUNSUPPORTED = 0, 1, 6
AT = 1 << 20     # an address that is never read: the calls below are refused


@pytest.fixture(scope="module")
def lib():
    return tlp.load_library()


def _desc(**kw):
    d = dict(dtype=2, batch=2, seq=33, heads=3, head_dim=64, scale=0.0, mask=None, bias_table=AT, buckets=32, max_distance=128)
    d.update(kw)
    return tlp._Attention(*[d[n] for n, _ in tlp._Attention._fields_])


def _view(data=AT, batch=33 * 192, token=192, head=64):
    return tlp._Heads(data, batch, token, head)


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(dtype=-1), dict(batch=0), dict(seq=0), dict(heads=-1), dict(head_dim=0), dict(head_dim=12),
    dict(head_dim=136), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(mask=AT + 2),
    dict(buckets=2), dict(buckets=7), dict(buckets=258), dict(buckets=0), dict(max_distance=8), dict(max_distance=0),
    dict(max_distance=(1 << 20) + 1), dict(bias_table=AT + 1),
])
def test_description_refused(lib, bad):
    d = _desc(**bad)
    assert lib.tl_attention_workspace_bytes(d, 0) == 0 and lib.tl_attention_workspace_bytes(d, 1) == 0
    o = _view(2 * AT)
    assert lib.tl_attention_forward(d, _view(), _view(), _view(), o, AT, AT, 1 << 40, None) == EINVAL


@pytest.mark.parametrize("big", [dict(seq=(1 << 20) + 1), dict(batch=1 << 12, seq=1 << 10, heads=1 << 10)])
def test_sizes_beyond_the_limits(lib, big):
    assert lib.tl_attention_forward(_desc(**big), _view(), _view(), _view(), _view(2 * AT), AT, AT, 1 << 40, None) == EUNSUPPORTED
    assert lib.tl_attention_workspace_bytes(_desc(**big), 1) == 0


def test_null_description(lib):
    assert lib.tl_attention_workspace_bytes(None, 0) == 0
    v = _view()
    assert lib.tl_attention_forward(None, v, v, v, _view(2 * AT), AT, AT, 1 << 40, None) == EINVAL


@pytest.mark.parametrize("bad", [
    dict(data=None), dict(data=AT + 8), dict(token=0), dict(token=-192), dict(token=63), dict(token=196), dict(batch=4),
    dict(head=60), dict(head=0), dict(batch=1 << 36),
])
@pytest.mark.parametrize("which", range(8))
def test_views_refused(lib, bad, which):
    d = _desc()
    need = lib.tl_attention_workspace_bytes(d, 1)
    assert need > 0
    views = [_view(AT * (i + 1)) for i in range(8)]
    kw = dict(data=AT * (which + 1))
    kw.update(bad)
    views[which] = _view(**kw)
    q, k, v, o, do, dq, dk, dv = views
    if which < 4:
        assert lib.tl_attention_forward(d, q, k, v, o, AT, AT, need, None) == EINVAL
    assert lib.tl_attention_backward(d, q, k, v, o, do, AT, dq, dk, dv, AT, 0, AT, need, None) == EINVAL


def test_other_pointers_refused(lib):
    d = _desc()
    need = lib.tl_attention_workspace_bytes(d, 1)
    q, k, v, o, do, dq, dk, dv = (_view(AT * (i + 1)) for i in range(8))
    f = lib.tl_attention_forward
    b = lib.tl_attention_backward
    assert f(d, q, k, v, o, None, AT, need, None) == EINVAL            # no lse
    assert f(d, q, k, v, o, AT + 2, AT, need, None) == EINVAL
    assert f(d, q, k, v, o, AT, None, need, None) == EINVAL            # no workspace
    assert f(d, q, k, v, o, AT, AT + 128, need, None) == EINVAL        # unaligned workspace
    assert f(d, q, k, v, o, AT, AT, lib.tl_attention_workspace_bytes(d, 0) - 1, None) == EINVAL
    assert f(d, q, k, v, q, AT, AT, need, None) == EINVAL              # output is an input
    assert f(d, None, k, v, o, AT, AT, need, None) == EINVAL
    assert b(d, q, k, v, o, do, AT, dq, dq, dv, AT, 0, AT, need, None) == EINVAL
    assert b(d, q, k, v, o, do, AT, do, dk, dv, AT, 0, AT, need, None) == EINVAL
    assert b(d, q, k, v, o, do, AT, dq, dk, dv, AT + 1, 0, AT, need, None) == EINVAL
    assert b(d, q, k, v, o, do, AT, dq, dk, dv, AT, 0, AT, need - 1, None) == EINVAL
    none = _desc(bias_table=None)
    assert b(none, q, k, v, o, do, AT, dq, dk, dv, AT, 0, AT, need, None) == EINVAL   # a table gradient without a table


@pytest.mark.parametrize("shared", [
    dict(token=64),                      # rows over the heads of their neighbours
    dict(batch=192),                     # sequences over one another
    dict(head=33 * 192 - 128, token=192),
])
def test_outputs_over_themselves_refused(lib, shared):
    d = _desc()
    need = lib.tl_attention_workspace_bytes(d, 1)
    q, k, v, o, do, dq, dk, dv = (_view(AT * (i + 1)) for i in range(8))
    assert lib.tl_attention_forward(d, q, k, v, _view(AT * 4, **shared), AT, AT, need, None) == EINVAL
    for i in range(3):
        outs = [dq, dk, dv]
        outs[i] = _view(AT * (6 + i), **shared)
        assert lib.tl_attention_backward(d, q, k, v, o, do, AT, *outs, AT, 0, AT, need, None) == EINVAL


def test_workspace_grows_with_the_call(lib):
    n = lib.tl_attention_workspace_bytes(_desc(), 0)
    assert 0 < n < lib.tl_attention_workspace_bytes(_desc(), 1)
    assert lib.tl_attention_workspace_bytes(_desc(bias_table=None, buckets=0, max_distance=0), 0) > 0
    assert n % 256 == 0


def _clip(lib, dtype=0, count=1, src=(AT,), dst=(AT,), n=(8,), limit=1.0, norm=AT, ws=AT, bytes_=1 << 30):
    p = (ctypes.c_void_p * max(1, len(src)))(*src)
    q = (ctypes.c_void_p * max(1, len(dst)))(*dst)
    s = (ctypes.c_uint64 * max(1, len(n)))(*n)
    return lib.tl_clip_grad_norm(dtype, count, p, q, s, limit, norm, ws, bytes_, None)


@pytest.mark.parametrize("bad", [
    dict(dtype=5), dict(count=-1), dict(src=(None,)), dict(dst=(None,)), dict(src=(AT + 2,)), dict(dst=(AT + 1,)),
    dict(n=(1 << 60,)), dict(limit=-1.0), dict(limit=float("nan")), dict(norm=None), dict(norm=AT + 1), dict(ws=None),
    dict(ws=AT + 4), dict(bytes_=8),
])
def test_clip_refusals(lib, bad):
    assert _clip(lib, **bad) == EINVAL


@pytest.mark.parametrize("many", [2, 300])
@pytest.mark.parametrize("dst", [
    (AT, AT),                            # one gradient twice
    (AT, AT + 28),                       # the last value of one is the first of the other
    (3 * AT, AT),                        # over another input
    (3 * AT, AT + 32 - 4), (AT + 4, 3 * AT), (3 * AT, 3 * AT),
])
def test_clip_outputs_that_overlap_refused(lib, dst, many):
    src = (AT, dst[1] if dst[0] == AT else 2 * AT)
    far = tuple((5 + i) * AT for i in range(many - 2))
    assert _clip(lib, count=many, src=src + far, dst=dst + far, n=(8,) * many) == EINVAL
    assert _clip(lib, count=many, src=far + src, dst=far + dst, n=(8,) * many) == EINVAL


def test_clip_workspace(lib):
    assert lib.tl_clip_workspace_bytes(-1) == 0
    assert 0 < lib.tl_clip_workspace_bytes(1) <= lib.tl_clip_workspace_bytes(5000)


def test_python_calls_refuse_cpu_tensors():
    q = torch.zeros(1, 8, 2, 16)
    with pytest.raises(tlp.TlError):
        tlp.attention_forward(q, q, q)
    with pytest.raises(tlp.TlError):
        tlp.attention_backward(q, q, q, q, torch.zeros(1, 2, 8), q)
    with pytest.raises(tlp.TlError):
        tlp.clip_grad_norm([q], 1.0)
    with pytest.raises(tlp.TlError):
        tlp.clip_grad_norm([], 1.0)


def test_position_bias_arguments(lib):
    """Refusals that need no device: a null layer, bad buckets and distances."""
    h = ctypes.c_void_p()
    assert lib.layer_create(2, 16, 64, 4, 0, 0.0, 0.0, 1, 1, ctypes.byref(h)) == OK
    f = lib.layer_set_position_bias
    try:
        assert f(None, AT, 32, 128, None, 0) == EINVAL
        assert f(h, None, 0, 0, None, 0) == OK           # nothing to take away
        for buckets, distance in ((31, 128), (2, 128), (258, 1000), (32, 8), (32, 1 << 21)):
            assert f(h, AT, buckets, distance, None, 0) == EINVAL
            assert lib.layer_last_error(h)
        assert f(h, AT, 32, 128, AT + 1, 0) == EINVAL
    finally:
        lib.layer_destroy(h)
