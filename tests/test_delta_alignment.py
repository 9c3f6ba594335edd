"""Addresses that are not aligned to their elements are refused by the gated delta rule, and by the checks that it shares with
the decay attention: no GPU needed (the addresses are made up and never read)."""

import ctypes

import pytest

from test_decay_refusals import NAN, arr, at, lib  # noqa: F401

CU = [0, 20, 64]


def call(lib, what, **kw):  # noqa: F811
    """One valid call of a kind, but for what kw says."""
    a = dict(g=at(3), beta=at(4), cu=at(5), status=at(6), idx=at(7), dg=at(8), db=at(9), per_token=1)
    a.update(kw)
    packed = (a["cu"], arr(CU), 2, 1, 64)
    heads = (2, 4, 128, NAN, None)
    pool = (at(10), 1, a["idx"], arr((0, 1), ctypes.c_int32), 4)
    ws = (at(16), 1 << 30)
    q, k, v = at(0), at(1), at(2)
    if what == "fwd":
        return lib.kda_gated_delta_fwd(q, k, v, a["g"], a["beta"], None, *packed, *heads, at(11), at(12), *ws, a["status"], None)
    if what == "bwd":
        return lib.kda_gated_delta_bwd(q, k, v, a["g"], a["beta"], *packed, *heads, at(11), None, at(12), at(13), at(14), a["dg"], a["db"],
                                       None, *ws, a["status"], None)
    if what == "prefill":
        return lib.kda_gated_delta_prefill(q, k, v, a["g"], a["beta"], *packed, *heads, *pool, at(11), *ws, a["status"], None)
    if what == "decode":
        return lib.kda_gated_delta_decode(q, k, v, a["g"], a["beta"], *pool, 2, *heads, at(11), None)
    gate = (a["g"], a["per_token"])
    if what == "decay fwd":
        return lib.kda_decay_attn_fwd(q, k, v, *gate, None, *packed, *heads, at(11), at(12), *ws, a["status"], None)
    if what == "decay bwd":
        return lib.kda_decay_attn_bwd(q, k, v, *gate, None, *packed, *heads, None, at(11), None, at(12), at(13), at(14), a["dg"], None,
                                      *ws, a["status"], None)
    if what == "decay prefill":
        return lib.kda_decay_attn_prefill(q, k, v, *gate, *packed, *heads, *pool, at(11), *ws, a["status"], None)
    return lib.kda_decay_attn_decode(q, k, v, *gate, *pool, 2, *heads, at(11), None)


OFFSETS = dict(g=1, beta=1, cu=4, status=2, idx=2, dg=1, db=1)
TAKES = {"fwd": ("g", "beta", "cu", "status"), "bwd": ("g", "beta", "cu", "status", "dg", "db"),
         "prefill": ("g", "beta", "cu", "status", "idx"), "decode": ("g", "beta", "idx"),
         "decay fwd": ("g", "cu", "status"), "decay bwd": ("g", "cu", "status", "dg"), "decay prefill": ("g", "cu", "status", "idx"),
         "decay decode": ("g", "idx")}


@pytest.mark.parametrize("what,name", [(w, n) for w, names in TAKES.items() for n in names])
def test_refused(lib, what, name):  # noqa: F811
    assert call(lib, what) in (2, 5)  # (the device check: there is none here)
    good = {"g": at(3), "beta": at(4), "cu": at(5), "status": at(6), "idx": at(7), "dg": at(8), "db": at(9)}[name]
    assert call(lib, what, **{name: good + 2 * OFFSETS[name]}) in (2, 5)
    assert call(lib, what, **{name: good + OFFSETS[name]}) == 1
    assert "aligned" in lib.kda_last_error_message().decode()


@pytest.mark.parametrize("what", [w for w in TAKES if w.startswith("decay") and w != "decay bwd"])
def test_fixed_decays(lib, what):  # noqa: F811
    """FP32 numbers, one for each head."""
    assert call(lib, what, per_token=0) in (2, 5)
    assert call(lib, what, per_token=0, g=at(3) + 2) == 1
    assert "aligned" in lib.kda_last_error_message().decode()
