"""Sizes whose products leave 64 bits are refused like any other size out of range (no GPU needed)."""

from __future__ import annotations

import pytest

from channel_wise_gated_b200 import _native, build

FAKE = 0x10000  # 16-byte aligned, never dereferenced: every case fails validation first


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.load()


@pytest.mark.parametrize("n,t,H", [(1 << 30, 16, 1 << 30), ((1 << 31) - 1, 16, (1 << 31) - 1),
                                   (1, 16, (1 << 31) - 1), (1 << 30, 2, 1 << 30), ((1 << 31) - 1, 1, 1),
                                   (1, 1, (1 << 31) - 1), (1, 16, 1 << 27), (1 << 27, 16, 1)])
def test_decode_rows(lib, n, t, H):
    assert lib.kda_mla_decode(FAKE, FAKE, 4, 64, FAKE, 2, FAKE, None, n, t, H, 0.07, FAKE, FAKE, FAKE, 1 << 30,
                              None) == _native.KDA_ERR_SHAPE


@pytest.mark.parametrize("n,T,H", [((1 << 31) - 1, 1 << 30, (1 << 31) - 1), (1 << 20, 256, 1 << 12)])
def test_prefill_grid(lib, n, T, H):
    assert lib.kda_mla_prefill(FAKE, 1 << 20, 192, FAKE, 1 << 20, 128, FAKE, 64, FAKE, 1 << 20, 128, FAKE, FAKE, n, T, T,
                               H, 0.07, 1, FAKE, None, None) == _native.KDA_ERR_SHAPE


@pytest.mark.parametrize("n,H", [((1 << 31) - 1, (1 << 31) - 1), (1 << 24, 2)])
def test_tree_states(lib, n, H):
    assert lib.kda_decode_tree(*[FAKE] * 8, n, 16, H, _native.KDA_BF16, _native.KDA_BF16, None) == \
        _native.KDA_ERR_SHAPE
