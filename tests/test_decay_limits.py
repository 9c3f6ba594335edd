"""Strides and sizes whose byte counts do not fit 64 bits are refused: no GPU needed (the addresses are made up and never
read)."""

import pytest

from test_decay_refusals import NAN, arr, at, fwd, lib, rope, slots_call  # noqa: F401

BIG = 1 << 62
WRAPS = ((1 << 64) // 3 + 8) // 8 * 8  # three times this is a small number in 64 bits


@pytest.mark.parametrize("strides", [
    [256, 128, 256, 128, 512, BIG],               # (heads - 1) x stride wraps round to a negative number
    [256, 128, 256, 128, 512, WRAPS],  # and to a small one
    [256, 128, 256, 128, BIG, 128],
    [256, BIG, 256, 128, 512, 128],
])
@pytest.mark.parametrize("what", ["forward", "decode"])
def test_strides(lib, what, strides):  # noqa: F811
    if what == "forward":
        rc, _ = fwd(lib, strides=strides)
    else:
        rc = lib.kda_decay_attn_decode(at(0), at(1), at(2), at(3), 1, at(5), 1, None, None, 4, 2, 2, 4, 128, NAN, arr(strides), at(7),
                                       None)
    assert rc in (1, 2), lib.kda_last_error_message()


def test_many_tokens_far_apart(lib):  # noqa: F811
    """Each stride is accepted for few tokens; all tokens together reach past 2^64 bytes."""
    far = 1 << 38
    assert fwd(lib, T=(1 << 31) - 2, hqk=1, hv=1, strides=[far, 128] * 3)[0] == 2
    assert rope(lib, n=1 << 30, hq=1, hk=1, strides=[1 << 40, 128] * 4) == 2


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("i", range(6))
def test_rope_strides(lib, bwd, i):  # noqa: F811
    strides = [512, 128, 256, 128] * (3 if bwd else 2)
    if 2 * i + 1 >= len(strides):
        pytest.skip("the forward has four tensors")
    for at_, value in ((2 * i + 1, BIG), (2 * i + 1, WRAPS), (2 * i, BIG)):
        strides_ = list(strides)
        strides_[at_] = value
        assert rope(lib, bwd=bwd, strides=strides_) in (1, 2), (at_, value, lib.kda_last_error_message())


@pytest.mark.parametrize("what", ["decode", "prefill"])
def test_pools(lib, what):  # noqa: F811
    """2^31 slots of 2^20 heads."""
    args = (at(5), 1, None, None, 1 << 31)
    if what == "decode":
        rc = lib.kda_decay_attn_decode(at(0), at(1), at(2), at(3), 1, *args, 1, 1, 1 << 20, 128, NAN, None, at(7), None)
    else:
        rc = lib.kda_decay_attn_prefill(at(0), at(1), at(2), at(3), 1, None, None, 0, 1, 1, 1, 1 << 20, 128, NAN, None, *args, at(7),
                                        at(9), 1 << 30, None, None)
    assert rc == 2, lib.kda_last_error_message()


def test_backward_too_large_for_its_sums(lib):  # noqa: F811
    """More (token, head) rows than the grid of the heads' sums takes: refused before the first launch."""
    rc = lib.kda_decay_attn_bwd(at(0), at(1), at(2), at(3), 1, None, None, None, 0, 1, 1 << 30, 128, 128, 128, NAN, None, at(17),
                                at(9), None, at(10), at(11), at(12), at(13), None, at(16), 1 << 62, None, None)
    assert rc == 2, lib.kda_last_error_message()
