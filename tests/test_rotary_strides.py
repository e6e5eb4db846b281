"""Strides of a projection whose extents no integer holds. No GPU: every call is refused before a launch."""
import pytest

from test_rotary import FAKE, h2o, qkv  # noqa: F401

BIG = 1 << 37  # the largest stride of heads of 128: 2^30 of them


@pytest.mark.parametrize("x,n,T", [
    (dict(q=(FAKE, BIG, 128, 128), q_heads=1), (1 << 27) + 1, 1),       # 2^64 elements: the extent would be a head's
    (dict(q=(FAKE, BIG, 128, 128), q_heads=1), (1 << 31) - 1, 1),
    (dict(q=(FAKE, BIG, 128, 128), q_heads=1), (1 << 26) + 1, 1),       # 2^63
])
def test_extents_that_no_integer_holds_are_refused(h2o, x, n, T):  # noqa: F811
    """In the place of a size that wrapped, with which an output on the input's first head was let through, or
    one far from it was not."""
    lib = h2o.load_library()
    for out in (FAKE * 2, FAKE):
        assert lib.h2o_rotate_qkv(qkv(d=128, **x), None, n, T, None, out, None, None) == -1
        if out != FAKE:
            assert b"strides" in lib.h2o_last_error(), lib.h2o_last_error()


@pytest.mark.parametrize("x,n,T", [(dict(q=(FAKE, BIG, 128, 128), q_heads=1), 1 << 10, 1),
                                   (dict(q=(FAKE, 128, BIG, 128), q_heads=1), 1, 1 << 20)])
def test_extents_within_64_bits_count_for_the_overlap(h2o, x, n, T):  # noqa: F811
    lib = h2o.load_library()
    assert lib.h2o_rotate_qkv(qkv(d=128, **x), None, n, T, None, FAKE + (1 << 40), None, None) == -1
    assert b"overlap" in lib.h2o_last_error()
