"""A layer that cannot have a position bias says why (no GPU: nothing is enqueued)."""
import ctypes

import pytest

import transformer_layer_pre_b200 as tlp

OK, EINVAL, EUNSUPPORTED = 0, 1, 6
AT = 1 << 20


@pytest.mark.parametrize("batch,seq,hidden,heads,buckets,status,word", [
    (1 << 17, 8, 2048, 128, 32, EUNSUPPORTED, "2^30"),
    (1, (1 << 20) + 8, 64, 4, 32, EUNSUPPORTED, "2^20"),
    (2, 16, 64, 4, 31, EINVAL, "buckets"),
])
def test_the_reason_is_the_layers(batch, seq, hidden, heads, buckets, status, word):
    lib = tlp.load_library()
    h = ctypes.c_void_p()
    assert lib.layer_create(batch, seq, hidden, heads, 8, 0.0, 0.0, 1, 1, ctypes.byref(h)) == OK
    try:
        assert lib.layer_set_position_bias(h, AT, buckets, 128, None, 0) == status
        assert word in lib.layer_last_error(h).decode()
    finally:
        lib.layer_destroy(h)
