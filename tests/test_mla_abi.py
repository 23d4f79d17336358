"""Refusals of the latent-attention entry points and of kda_decode_tree: bad arguments return
their status on the host, before any CUDA call (no GPU needed)."""

from __future__ import annotations

import pytest

from channel_wise_gated_b200 import _native, build

FAKE = 0x10000  # 16-byte aligned, never dereferenced: every case fails validation first
BF, F32 = _native.KDA_BF16, _native.KDA_F32


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.load()


def test_status_strings_of_the_device_errors(lib):
    assert "page" in _native.status_string(_native.KDA_ERR_PAGE)
    assert "path" in _native.status_string(_native.KDA_ERR_TREE)


def test_decode_tree_validation(lib):
    def f(**a):
        g = lambda n: a.get(n, FAKE)
        return lib.kda_decode_tree(g("q"), g("k"), g("v"), g("la"), g("b"), g("s"),
                                   a.get("tree", FAKE), g("o"), a.get("n", 4), a.get("t", 2),
                                   a.get("H", 2), a.get("dt", BF), a.get("gt", BF), None)
    for p in ("q", "k", "v", "la", "b", "s", "o"):
        assert f(**{p: None}) == _native.KDA_ERR_NULL
    for p in ("q", "k", "v", "la", "s", "o"):
        assert f(**{p: FAKE + 8}) == _native.KDA_ERR_ALIGN
    assert f(tree=FAKE + 2) == _native.KDA_ERR_ALIGN
    for bad in (dict(n=0), dict(H=0), dict(t=0), dict(t=_native.KDA_DECODE_MAX_TOKENS + 1),
                dict(n=1 << 20, H=1 << 12)):
        assert f(**bad) == _native.KDA_ERR_SHAPE
    assert f(dt=5) == _native.KDA_ERR_DTYPE and f(gt=5) == _native.KDA_ERR_DTYPE


def test_append_validation(lib):
    def f(**a):
        return lib.kda_mla_append(a.get("x", FAKE), a.get("stride", 576), a.get("w", FAKE),
                                  a.get("eps", 1e-6), a.get("cache", FAKE), a.get("pages", 4),
                                  a.get("page", 64), a.get("table", FAKE), a.get("most", 2),
                                  a.get("lens", FAKE), a.get("cu", FAKE), a.get("n", 2),
                                  a.get("T", 8), a.get("lat", FAKE), None)
    for p in ("x", "cache", "table", "lens"):
        assert f(**{p: None}) == _native.KDA_ERR_NULL
    for p in ("x", "w", "cache", "lat"):
        assert f(**{p: FAKE + 8}) == _native.KDA_ERR_ALIGN
    for p in ("table", "lens", "cu"):
        assert f(**{p: FAKE + 2}) == _native.KDA_ERR_ALIGN
    for bad in (dict(stride=575), dict(stride=580), dict(eps=-1.0), dict(eps=float("nan")),
                dict(pages=0), dict(page=0), dict(most=0), dict(n=0), dict(T=-1),
                dict(most=1 << 26, page=64)):
        assert f(**bad) == _native.KDA_ERR_SHAPE
    assert f(cu=None, T=7) == _native.KDA_ERR_SEQLENS      # no equal runs
    assert f(T=0, x=None) == _native.KDA_OK                # nothing to do
