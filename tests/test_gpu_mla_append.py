"""kda_mla_append against its definition in 64 bits, through the Python binding.

Tolerance, before any run: fp32 arithmetic (a sum of 512 squares, one square root, one division,
two products: under 512 * 2^-24 / 2 + 4 * 2^-24 = 1.6e-5 relative), then one rounding to bf16.
Values that are copied, and every row that is not written, must be equal bit for bit.
"""

from __future__ import annotations

import pytest
import torch

from refs import latent as ref

pytestmark = pytest.mark.gpu

W = ref.LATENT + ref.SHARED
REL = 1.6e-5


@pytest.fixture(scope="module")
def kda():
    from channel_wise_gated_b200 import build
    build.build()
    import channel_wise_gated_b200 as m
    return m


@pytest.fixture(autouse=True)
def _no_device_error(kda):
    yield
    assert kda.device_status() == 0


def setup(new, lens, page, seed, max_extra=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-x // page) for x in lens]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(need) + max_extra), -1, dtype=torch.int32, device="cuda")
    at = 0
    for n, k in enumerate(need):
        table[n, :k] = order[at:at + k]
        at += k
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    return dict(x=torch.randn((cu[-1], W), generator=g, device="cuda").bfloat16(),
                w=0.5 + torch.rand(ref.LATENT, generator=g, device="cuda"),
                cache=torch.randn((pool, page, W), generator=g, device="cuda").bfloat16(),
                table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                cu=torch.tensor(cu, dtype=torch.int32, device="cuda"))


def expect(s, new, lens, page, normed):
    """(64-bit value of every written row, their flat slots)."""
    y = ref.rmsnorm(s["x"][:, :512].cpu(), s["w"].cpu(), 1e-6) if normed else s["x"][:, :512].cpu().double()
    table, slots = s["table"].cpu(), []
    for n, (t, L) in enumerate(zip(new, lens)):
        for p in range(L - t, L):
            slots.append(int(table[n, p // page]) * page + p % page)
    return y, slots


def check_rows(got, y):
    err = (got.cpu().double() - y).abs()
    assert bool((err <= (ref.half_step(torch.bfloat16) + REL) * y.abs()).all())


@pytest.mark.parametrize("new,lens,page", [
    ([1], [1], 16), ([1], [65], 64), ([5], [5], 8), ([3, 0, 1, 17], [64, 30, 1, 17], 16),
    ([7] * 40, list(range(7, 47)), 32), ([129, 1, 70], [200, 4097, 70], 64), ([2, 9], [11, 9], 1),
    ([4] * 33, [100] * 33, 24)])
@pytest.mark.parametrize("normed", [True, False])
def test_append(kda, new, lens, page, normed):
    s = setup(new, lens, page, seed=len(new) + page)
    before = s["cache"].clone()
    lat = kda.mla_append(s["x"], s["w"] if normed else None, s["cache"], s["table"], s["lens"],
                         cu_seqlens=s["cu"], output_latent=True)
    y, slots = expect(s, new, lens, page, normed)
    flat = s["cache"].view(-1, W)
    rows = flat[slots]
    check_rows(rows[:, :512], y)
    assert torch.equal(rows[:, 512:], s["x"][:, 512:])
    assert torch.equal(lat, rows[:, :512])
    if not normed:
        assert torch.equal(rows, s["x"])
    untouched = torch.ones(flat.shape[0], dtype=torch.bool)
    untouched[slots] = False
    assert torch.equal(flat.cpu()[untouched], before.view(-1, W).cpu()[untouched])


def test_equal_runs_strided_rows_and_no_latent(kda):
    """Without cu_seqlens every sequence appends T / N tokens; x is a slice of a wider row."""
    new, lens, page = [4] * 6, [4, 9, 64, 65, 63, 130], 64
    s = setup(new, lens, page, seed=5)
    wide = torch.randn(24, 2000, device="cuda").bfloat16()
    wide[:, 1000:1000 + W] = s["x"]
    a, b = s["cache"].clone(), s["cache"].clone()
    assert kda.mla_append(s["x"], s["w"], a, s["table"], s["lens"], cu_seqlens=s["cu"]) is None
    kda.mla_append(wide[:, 1000:1000 + W], s["w"], b, s["table"], s["lens"])
    assert torch.equal(a, b)


def test_zero_rows_and_extreme_values(kda):
    """An all-zero latent stays zero (eps guards it); large values scale without overflow."""
    s = setup([3], [3], 16, seed=6)
    s["x"][0] = 0
    s["x"][1, :512] = 1e18
    kda.mla_append(s["x"], s["w"], s["cache"], s["table"], s["lens"])
    rows = s["cache"].view(-1, W)[expect(s, [3], [3], 16, True)[1]]
    assert bool((rows[0] == 0).all())
    assert bool(torch.isfinite(rows).all())
    check_rows(rows[:, :512], ref.rmsnorm(s["x"][:, :512].cpu(), s["w"].cpu(), 1e-6))


def test_bad_pages_and_lengths_are_skipped_and_flagged(kda):
    """A page out of range, a negative row and a length past the table: those tokens are left
    out, the others land, and the device reports it."""
    from channel_wise_gated_b200 import _native
    new, lens, page = [2, 2, 2, 2], [2, 2, 2, 2], 16
    s = setup(new, lens, page, seed=7, max_extra=0)
    good = expect(s, new, lens, page, True)
    for seq, what in ((0, "page"), (1, "high"), (2, "negative"), (3, "length")):
        table, ln = s["table"].clone(), s["lens"].clone()
        if what == "page":
            table[seq, 0] = -1
        elif what == "high":
            table[seq, 0] = s["cache"].shape[0]
        elif what == "negative":
            ln[seq] = 0
        else:
            ln[seq] = 1000
        cache = s["cache"].clone()
        kda.mla_append(s["x"], s["w"], cache, table, ln, cu_seqlens=s["cu"])
        assert kda.device_status() == _native.KDA_ERR_PAGE
        for i, slot in enumerate(good[1]):
            if i // 2 == seq:
                assert torch.equal(cache.view(-1, W)[slot], s["cache"].view(-1, W)[slot])
            else:
                check_rows(cache.view(-1, W)[slot][:512][None], good[0][i][None])


def test_bad_cu_seqlens_flagged(kda):
    from channel_wise_gated_b200 import _native
    s = setup([4, 4], [4, 4], 16, seed=8)
    cu = torch.tensor([0, 9, 8], dtype=torch.int32, device="cuda")
    kda.mla_append(s["x"], s["w"], s["cache"], s["table"], s["lens"], cu_seqlens=cu)
    assert kda.device_status() != 0


def test_large_offsets(kda):
    """A cache past 2^31 values: the row's offset takes 64 bits."""
    page = 128
    pages = (1 << 31) // (page * W) + 40
    cache = torch.zeros((pages, page, W), dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[pages - 1], [pages - 2]], dtype=torch.int32, device="cuda")
    x = torch.randn(4, W, device="cuda").bfloat16()
    kda.mla_append(x, None, cache, table, torch.tensor([128, 2], dtype=torch.int32, device="cuda"))
    assert torch.equal(cache[-1, 126:], x[:2]) and torch.equal(cache[-2, :2], x[2:])
    assert int((cache != 0).any(-1).sum()) == 4


def test_rows_behind_the_last_sequence_are_left(kda):
    """A batch padded behind its last sequence: the padding (NaN here) is written nowhere, the
    latent output's rows there stay, and the device reports the lengths."""
    from channel_wise_gated_b200 import _native
    new, lens, page = [3, 5], [20, 5], 16
    s = setup(new, lens, page, seed=8)
    a, b = s["cache"].clone(), s["cache"].clone()
    want = kda.mla_append(s["x"], s["w"], a, s["table"], s["lens"], cu_seqlens=s["cu"], output_latent=True)
    x = torch.cat([s["x"], torch.full((4, W), float("nan"), device="cuda").bfloat16()])
    lat = torch.full((12, ref.LATENT), 7.0, device="cuda").bfloat16()
    kda.mla_append(x, s["w"], b, s["table"], s["lens"], cu_seqlens=s["cu"], latent=lat)
    assert kda.device_status() == _native.KDA_ERR_SEQLENS
    assert torch.equal(a, b) and torch.equal(lat[:8], want) and bool((lat[8:] == 7).all())
