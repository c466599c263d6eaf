"""Sizes and scales at which the attention's calls end, on the host (CPU)."""

import ctypes

import pytest

import context_packed_sequence_amd as thd
from test_train_refusals import _attention, _shape, lib  # noqa: F401  (fixture)


@pytest.mark.parametrize("bad", [dict(scale=2.0 ** -100.1), dict(scale=1e-38), dict(scale=2.0 ** 100.1), dict(scale=1e38),
                                 dict(cap=2.0 ** -64.1), dict(cap=1e-39), dict(cap=3e38), dict(scale=2.0 ** -90, cap=1e30),
                                 dict(scale=2.0 ** 100, cap=2.0 ** -28)])
def test_scales_without_room(lib, bad):
    # scale 1e-38: lse / scale of 4 is past 32 bits; 1e38: products that end at 2^-126 are off by
    # 1 in the score; cap 1e-39: its reciprocal is past 32 bits
    for backward in (0, 1):
        assert lib.thd_attention_workspace_bytes(ctypes.byref(_shape(**bad)), backward) == -1
        assert _attention(lib, _shape(**bad), backward=bool(backward)) == thd.THD_ERR_ARG


@pytest.mark.parametrize("good", [dict(scale=2.0 ** -100), dict(scale=2.0 ** 100), dict(cap=2.0 ** -64), dict(cap=2e38),
                                  dict(scale=2.0 ** -100, cap=2.0 ** 49), dict(scale=2.0 ** 100, cap=2.0 ** -27)])
def test_scales_with_room(lib, good):
    for backward in (0, 1):
        assert lib.thd_attention_workspace_bytes(ctypes.byref(_shape(**good)), backward) > 0


def test_longest_stream(lib):
    # a key position passes the last token by up to a tile, and a row's window starts before the
    # first: both have to fit 32 bits
    how = dict(heads=1, kv_heads=1, dim=8, cp_size=2, window=64)
    shape = lambda n: ctypes.byref(_shape(total_tokens=n, **how))  # noqa: E731
    assert lib.thd_attention_workspace_bytes(shape(thd.THD_MAX_STREAM), 0) > 0
    for n in (thd.THD_MAX_STREAM + 2, 2 ** 31 - 64, 2 ** 31 - 4):
        assert lib.thd_attention_workspace_bytes(shape(n), 0) == -1
        assert _attention(lib, _shape(total_tokens=n, **how)) == thd.THD_ERR_ARG
