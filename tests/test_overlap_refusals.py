"""Outputs whose rows share elements are refused, layouts whose rows lie apart are not (CPU only).

No call reaches a kernel: each has an unaligned pointer too, which is refused after the layout."""
import ctypes
import itertools

import pytest

from tests.test_prefill_abi import ARG, _plan, _rope, lib  # noqa: F401

UNALIGNED = ctypes.c_void_p(4098)


def _apart(sizes, strides, extent):
    """By listing every row: whether the rows [start, start + extent) are disjoint."""
    starts = sorted(sum(i * s for i, s in zip(at, strides)) for at in itertools.product(*map(range, sizes)))
    return all(b - a >= extent for a, b in zip(starts, starts[1:]))


@pytest.mark.parametrize("sizes, strides", [
    ((2, 3, 4), (768, 256, 64)), ((2, 3, 4), (64 * 4, 64 * 8, 64)), ((2, 3, 4), (64, 128, 384)), ((1, 3, 4), (0, 256, 64)),
    ((1, 1, 1), (0, 0, 0)), ((2, 1, 4), (256, 7, 64)), ((2, 3, 4), (1000, 300, 70)), ((2, 3, 4), (2 ** 62, 2 ** 61, 2 ** 40)),
    ((2, 3, 4), (768, 256, 63)), ((2, 3, 4), (768, 255, 64)), ((2, 3, 4), (767, 256, 64)), ((2, 3, 4), (768, 64, 64)),
    ((2, 3, 4), (256, 256, 64)), ((2, 1, 1), (1, 0, 0)), ((1, 1, 2), (0, 0, 63)), ((1, 3, 1), (0, 8, 0))])
def test_rope_out(lib, sizes, strides):  # noqa: F811
    _, plan = _plan(lib, dim=32)
    b, t, h = sizes
    assert ARG == _rope(lib, plan, batch=b, tokens=t, heads=h, head_dim=64, rope_offset=0, strides=(4096, 1024, 128),
                        out_strides=strides, pos=UNALIGNED)
    message = lib.mla_last_error()
    assert (b"overlap" if not _apart(sizes, strides, 64) else b"aligned") in message, message


def test_rope_in_place_writes_the_rotated_dims_alone(lib):  # noqa: F811
    _, plan = _plan(lib, dim=32)
    x = ctypes.c_void_p(1 << 30)
    for step, fine in ((64, True), (40, True), (32, True), (31, False), (1, False)):
        assert ARG == _rope(lib, plan, x=x, out=x, batch=1, tokens=1, heads=5, head_dim=64, rope_offset=0, strides=(0, 0, step),
                            pos=UNALIGNED)
        assert (b"aligned" if fine else b"overlap") in lib.mla_last_error(), step
