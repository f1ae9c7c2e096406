"""Outputs whose rows share elements are refused, layouts whose rows lie apart are not (CPU only).

No call reaches a kernel: each has an unaligned pointer too, which is refused after the layout."""
import ctypes
import itertools

import pytest

from tests.test_prefill_abi import ARG, DUMMY, _append, _plan, _rope, _shape, lib  # noqa: F401

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


@pytest.mark.parametrize("heads, blocks, strides", [
    (2, 3, (64 * 1152, 1152, 576)), (2, 3, (64 * 576, 576, 3 * 64 * 576)), (2, 3, (576, 2 * 3 * 576, 3 * 576)),
    (1, 3, (64 * 640, 640, 576)), (1, 1, (576, 576, 576)), (2, 3, (64 * 1152, 576, 576)), (2, 3, (1152, 1152, 576)),
    (2, 3, (64 * 1152 - 8, 1152, 576)), (2, 3, (64 * 1152, 1144, 576)), (1, 2, (576 * 63, 576, 576))])
def test_append_caches(lib, heads, blocks, strides):  # noqa: F811
    _, plan = _plan(lib)
    fine = _apart((blocks, 64, heads), strides, 576)
    assert ARG == _append(lib, plan, h_k=heads, num_blocks=blocks, k=strides, latent=UNALIGNED)
    assert (b"aligned" if fine else b"overlap") in lib.mla_last_error(), lib.mla_last_error()
    # the rotary cache of two, with the same layout in rows of 64
    fine = _apart((blocks, 64, heads), [s // 9 // 8 * 8 for s in strides], 64)
    assert ARG == _append(lib, plan, h_k=heads, num_blocks=blocks, kr=DUMMY, k=(64 * heads * 512, heads * 512, 512),
                          krs=[s // 9 // 8 * 8 for s in strides], latent=UNALIGNED)
    assert (b"aligned" if fine else b"overlap") in lib.mla_last_error(), lib.mla_last_error()


@pytest.mark.parametrize("tokens, heads, strides", [
    (6, 16, (16 * 512, 512)), (6, 16, (512, 6 * 512)), (1, 16, (8, 520)), (6, 1, (512, 8)), (6, 16, (16 * 520, 520)),
    (6, 16, (512, 512)), (6, 16, (15 * 512, 512)), (6, 16, (1024, 512)), (6, 16, (512, 5 * 512)), (2, 2, (512, 512))])
def test_chunk_out(lib, tokens, heads, strides):  # noqa: F811
    n = ctypes.c_size_t(0)
    rc = lib.mla_chunk_workspace_size(ctypes.byref(_shape(total_q=tokens, h_q=heads, o=strides)), ctypes.byref(n))
    assert rc == (0 if _apart((tokens, heads), strides, 512) else ARG)
