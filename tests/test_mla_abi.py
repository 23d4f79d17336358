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


def test_prefill_validation(lib):
    def f(**a):
        g = lambda n, d=FAKE: a.get(n, d)
        return lib.kda_mla_prefill(
            g("q"), g("qt", 384), g("qh", 192), g("k"), g("kt", 256), g("kh", 128), g("ks"),
            g("kst", 64), g("v"), g("vt", 256), g("vh", 128), g("cq", None), g("ck", None),
            g("n", 1), g("Tq", 64), g("Tk", 64), g("H", 2), g("scale", 0.07), g("causal", 1),
            g("o"), g("lse"), None)
    for p in ("q", "k", "ks", "v", "o"):
        assert f(**{p: None}) == _native.KDA_ERR_NULL
        assert f(**{p: FAKE + 8}) == _native.KDA_ERR_ALIGN
    assert f(lse=FAKE + 2) == _native.KDA_ERR_ALIGN
    assert f(cq=FAKE + 2, ck=FAKE) == _native.KDA_ERR_ALIGN
    for bad in (dict(n=0), dict(H=0), dict(Tq=-1), dict(Tk=-1), dict(Tq=1 << 31), dict(Tk=1 << 31),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(qh=191), dict(qt=388), dict(kh=120), dict(kt=260), dict(kst=60), dict(vh=4),
                dict(vt=1 << 40), dict(H=1 << 20, Tq=1 << 30, qt=1 << 30)):
        assert f(**bad) == _native.KDA_ERR_SHAPE
    assert f(n=2) == _native.KDA_ERR_SEQLENS               # several sequences need cu_seqlens
    assert f(cq=FAKE) == _native.KDA_ERR_SEQLENS           # both or none
    assert f(ck=FAKE) == _native.KDA_ERR_SEQLENS
    assert f(Tq=0, q=None, o=None) == _native.KDA_OK       # nothing to do


def test_decode_validation(lib):
    def f(**a):
        g = lambda n, d=FAKE: a.get(n, d)
        return lib.kda_mla_decode(g("q"), g("cache"), g("pages", 4), g("page", 64), g("table"),
                                  g("most", 2), g("lens"), g("tree", None), g("n", 2), g("t", 1),
                                  g("H", 4), g("scale", 0.07), g("o"), g("lse"), g("ws"),
                                  g("bytes", 1 << 30), None)
    for p in ("q", "cache", "table", "lens", "o", "ws"):
        assert f(**{p: None}) == _native.KDA_ERR_NULL
    for p in ("q", "cache", "o", "ws"):
        assert f(**{p: FAKE + 8}) == _native.KDA_ERR_ALIGN
    for p in ("table", "lens", "tree", "lse"):
        assert f(**{p: FAKE + 2}) == _native.KDA_ERR_ALIGN
    for bad in (dict(n=0), dict(t=0), dict(t=_native.KDA_DECODE_MAX_TOKENS + 1), dict(H=0),
                dict(n=1 << 20, t=16, H=1 << 8), dict(page=0), dict(page=12), dict(pages=0),
                dict(pages=1 << 31), dict(most=0), dict(most=(1 << 24) + 1), dict(scale=0.0),
                dict(scale=float("nan"))):
        assert f(**bad) == _native.KDA_ERR_SHAPE


def test_workspace_size_of_bad_sizes(lib):
    size = lib.kda_mla_decode_workspace_size
    assert size(0, 4) == 0 and size(17, 4) == 0 and size(1, 0) == 0


def test_python_refusals_need_no_gpu():
    """The binding names what is wrong before it looks for the library or a device."""
    import torch

    import channel_wise_gated_b200 as kda
    bf = torch.bfloat16
    z = lambda *s, dtype=bf: torch.zeros(s, dtype=dtype)
    lens = z(2, dtype=torch.int32)
    with pytest.raises(ValueError):                       # not on a GPU
        kda.mla_append(z(4, 576), None, z(2, 16, 576), z(2, 1, dtype=torch.int32), lens)
    with pytest.raises(ValueError):                       # not [T, 576]
        kda.mla_append(z(4), None, z(2, 16, 576), z(2, 1, dtype=torch.int32), lens)
    with pytest.raises(ValueError):
        kda.mla_prefill(z(4, 2), z(4, 2, 128), z(4, 64), z(4, 2, 128))
    with pytest.raises(ValueError):
        kda.mla_prefill(z(4, 2, 192), z(4, 2), z(4, 64), z(4, 2, 128))
    with pytest.raises(ValueError):
        kda.mla_decode(z(2, 1, 4, 512), z(2, 16, 576), z(2, 1, dtype=torch.int32), lens)
    with pytest.raises(ValueError):                       # 17 tokens
        kda.mla_decode(z(2, 17, 4, 576), z(2, 16, 576), z(2, 1, dtype=torch.int32), lens)
    with pytest.raises(ValueError):
        kda.decode_tree(z(2, 17, 4, 128), z(2, 17, 4, 128), z(2, 17, 4, 128), z(2, 17, 4, 128),
                        z(2, 17, 4), z(2, 4, 128, 128))
