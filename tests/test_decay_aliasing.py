"""Overlaps that kda_qk_norm_rope_bwd refuses among its weights' gradients, its workspace and the other buffers: no GPU
needed (the addresses are made up and never read)."""

import pytest

from test_decay_refusals import at, lib, rope  # noqa: F401

DIM, ROWS = 128, 8 * 4 * 128 * 2  # bytes of a query tensor


@pytest.mark.parametrize("kw", [
    dict(dqw=at(11)), dict(dkw=at(10) + 256),                     # each other
    dict(ws=at(10)), dict(ws=at(11) - 1024), dict(dqw=at(12) + 4096),  # the workspace
    dict(ws=at(0)), dict(ws=at(1)), dict(ws=at(8)), dict(ws=at(9)),    # over inputs
    dict(ws=at(6)), dict(ws=at(7) - 64), dict(ws=at(2)), dict(ws=at(3)), dict(ws=at(4)), dict(ws=at(5)),
    dict(dqw=at(2)), dict(dkw=at(3) + 16), dict(dqw=at(3)),       # over weights
    dict(dqw=at(0) + ROWS - 16), dict(dkw=at(1)), dict(dqw=at(8)), dict(dkw=at(9)), dict(dqw=at(6)), dict(dkw=at(7)),
    dict(dqw=at(4)), dict(dkw=at(5)),
])
def test_rope_backward_refuses(lib, kw):  # noqa: F811
    assert rope(lib, bwd=True, **kw) == 3, lib.kda_last_error_message()


def test_rope_backward_accepts(lib):  # noqa: F811
    """Buffers next to each other, weights that are not there, an empty batch, and no positions."""
    for kw in (dict(dqw=at(0) + ROWS, dkw=at(0) + ROWS + 4 * DIM, ws=at(0) + ROWS + 8 * DIM), dict(qw=None, dqw=None),
               dict(qw=None, kw=None, dqw=None, dkw=None, ws=None, wsb=0), dict(n=0, pos=at(10)), dict(rot=0, pos=at(10), freq=at(12)),
               dict(qw=at(3))):
        assert rope(lib, bwd=True, **kw) in (2, 5), (kw, lib.kda_last_error_message())
