"""kda_mla_decode against softmax attention in 64 bits over the rows each token sees.

Tolerances, before any run. Scores: fp32 sums of 576 exact products, off by at most 576 * 2^-24 =
3.5e-5 of the terms' absolute sum, which for these draws is about 210 before the scale of 0.072:
5e-4, and lse no more. Output: a weight is off by 5e-4 from its score, 2^-8 from its rounding to
bf16 and 2^-22 from the exponential, relative, so o by at most (2^-8 + 1e-3) sum_j w_j |c_j| and
its own rounding, 2^-8 |o|.
"""

from __future__ import annotations

import math

import pytest
import torch

from refs import latent as ref

pytestmark = pytest.mark.gpu

W = ref.LATENT + ref.SHARED
SCALE = (ref.D + ref.SHARED) ** -0.5


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


def setup(lens, t, H, page, seed, garbage=True):
    """Queries, a shuffled pool, its table. Rows that belong to no length hold NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-x // page) for x in lens]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(max(need), 1) + 1), -1, dtype=torch.int32, device="cuda")
    cache = torch.full((pool, page, W), float("nan") if garbage else 0.0, device="cuda").bfloat16()
    at = 0
    for n, k in enumerate(need):
        table[n, :k] = order[at:at + k]
        at += k
        if lens[n]:
            p = torch.arange(lens[n], device="cuda")
            cache[table[n, p // page].long(), p % page] = \
                torch.randn((lens[n], W), generator=g, device="cuda").bfloat16()
    q = (torch.randn((len(lens), t, H, W), generator=g, device="cuda") * 0.577).bfloat16()
    return q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


def check(o, lse, q, cache, table, lens, tree=None, scale=SCALE):
    c = [x.cpu() for x in (q, cache, table, lens)]
    tr = None if tree is None else tree.cpu()
    o_ref, lse_ref = ref.mla_decode(*c, tr, scale)
    big = c[1].clone()
    spread = torch.zeros_like(o_ref)
    N, t, H, _ = q.shape
    for n in range(N):     # sum of weights times |value|, from the same weights
        L = int(lens[n])
        rows = ref.cached_rows(big, c[2], n, 0, L)
        for j in range(t):
            bits = (2 << j) - 1 if tr is None else int(tr[n, j])
            seen = [p for p in range(L) if p < L - t or (bits >> (p - (L - t))) & 1]
            for h in range(H):
                spread[n, j, h], _ = ref.attend(c[0][n, j, h].double(), rows[seen],
                                                rows[seen][:, :512].abs(), scale)
    h = ref.half_step(torch.bfloat16)
    err = (o.cpu().double() - o_ref).abs()
    assert bool((err <= (h + 1e-3) * spread + h * o_ref.abs()).all()), float(err.max())
    if lse is not None:
        inf = torch.isinf(lse_ref)
        assert torch.equal(torch.isinf(lse.cpu()), inf)
        d = (lse.cpu().double() - lse_ref)[~inf].abs()
        assert d.numel() == 0 or float(d.max()) <= 5e-4


@pytest.mark.parametrize("L", [1, 2, 8, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 1000])
@pytest.mark.parametrize("H", [1, 4, 32])
def test_one_sequence_one_token(kda, L, H):
    s = setup([L], 1, H, 64, seed=L + H)
    o, lse = kda.mla_decode(*s, output_lse=True)
    check(o, lse, *s)


@pytest.mark.parametrize("page", [8, 16, 24, 32, 40, 64, 128, 192, 256])
def test_page_sizes(kda, page):
    s = setup([300, 77, 256], 1, 8, page, seed=page)
    o, lse = kda.mla_decode(*s, output_lse=True)
    check(o, lse, *s)


@pytest.mark.parametrize("t,H", [(1, 5), (2, 16), (3, 11), (4, 32), (16, 1), (1, 64), (1, 65), (1, 128), (7, 20),
                                 (16, 8)])
def test_rows_and_chains(kda, t, H):
    """Rows of one to several groups, padded and not; lengths shorter than the tokens, none."""
    s = setup([200, t, 0, 66, max(1, t - 1), 64], t, H, 16, seed=t * 100 + H)
    o, lse = kda.mla_decode(*s, output_lse=True)
    check(o, lse, *s)
    assert bool((o[2] == 0).all()) and bool((lse[2] == -math.inf).all())


@pytest.mark.parametrize("t,H", [(2, 4), (5, 3), (8, 8), (16, 2)])
def test_trees(kda, t, H):
    s = setup([130, t, 64 + t, 63, 65], t, H, 32, seed=t * 7 + H)
    tree = ref.random_tree(5, t, seed=t).cuda()
    o, lse = kda.mla_decode(*s, tree=tree, output_lse=True)
    check(o, lse, *s, tree=tree)


def test_a_token_that_sees_nothing(kda):
    """No bits and no prefix: zeros and -inf; its neighbours are not touched by it."""
    s = setup([4, 4], 4, 3, 16, seed=3)
    tree = torch.tensor([[1, 0, 4, 8], [0, 0, 0, 0]], dtype=torch.int32, device="cuda")
    o, lse = kda.mla_decode(*s, tree=tree, output_lse=True)
    check(o, lse, *s, tree=tree)
    assert bool((o[0, 1] == 0).all()) and bool((lse[0, 1] == -math.inf).all())
    assert bool((o[1] == 0).all())


@pytest.mark.parametrize("lens", [[3000], [1, 2000, 1, 1500], [0, 0, 900, 0], [65] * 200, [700] * 40])
@pytest.mark.parametrize("t,H", [(1, 2), (1, 70)])
def test_runs_that_cut_sequences(kda, lens, t, H):
    """Long sequences over many CTAs, many short ones in one CTA, and empty slots between."""
    s = setup(lens, t, H, 64, seed=len(lens))
    o, lse = kda.mla_decode(*s, output_lse=True)
    pick = [0, len(lens) // 2, len(lens) - 1]
    check(o[pick], lse[pick], s[0][pick], s[1], s[2][pick], s[3][pick])
    # every sequence alone gives the same up to how it is cut
    n = max(range(len(lens)), key=lambda i: lens[i])
    o1, l1 = kda.mla_decode(s[0][n:n + 1].contiguous(), s[1], s[2][n:n + 1].contiguous(),
                            s[3][n:n + 1].contiguous(), output_lse=True)
    assert float((l1[0] - lse[n]).abs().max()) <= 1e-5 * max(1.0, float(lse[n].abs().max()))
    again, _ = kda.mla_decode(*s)
    assert torch.equal(again, o)


def test_rising_scores_move_the_reference(kda):
    """Scores that grow along the sequence by some hundreds: sums of terms up to 400 / scale in
    one product are exact to 576 * 2^-24 of it: 400 * 3.5e-5 = 1.4e-2 in lse."""
    L, H = 900, 3
    q, cache, table, lens = setup([L], 1, H, 64, seed=4, garbage=False)
    q = (q * 0.2).bfloat16()
    q[..., 0] = 6.0
    p = torch.arange(L, device="cuda")
    cache[table[0, p // 64].long(), p % 64, 0] = p.bfloat16()
    o, lse = kda.mla_decode(q, cache, table, lens, output_lse=True)
    o_ref, lse_ref = ref.mla_decode(q.cpu(), cache.cpu(), table.cpu(), lens.cpu(), None, SCALE)
    assert float((lse.cpu().double() - lse_ref).abs().max()) <= 1.4e-2
    assert float((o.cpu().double() - o_ref).abs().max()) <= 0.04 * float(o_ref.abs().max())


def test_shared_pages_and_the_last_page(kda):
    """Two sequences over the same prefix pages; a cache past 2^31 values, read at its end."""
    page = 128
    pages = (1 << 31) // (page * W) + 40
    cache = torch.zeros((pages, page, W), dtype=torch.bfloat16, device="cuda")
    cache[-3:] = torch.randn(3, page, W, device="cuda").bfloat16()
    table = torch.tensor([[pages - 1, pages - 2], [pages - 1, pages - 3]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([200, 256], dtype=torch.int32, device="cuda")
    q = (torch.randn(2, 2, 4, W, device="cuda") * 0.577).bfloat16()
    o, lse = kda.mla_decode(q, cache, table, lens, output_lse=True)
    small = cache[-3:].contiguous()
    t2 = torch.tensor([[2, 1], [2, 0]], dtype=torch.int32, device="cuda")
    o2, lse2 = kda.mla_decode(q, small, t2, lens, output_lse=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check(o, lse, q, small, t2, lens)


def test_bad_pages_and_lengths_are_flagged(kda):
    """A page out of range reads page 0 instead, a length past the table ends with it; both are
    reported, and the other sequences keep their results (up to where the runs cut them)."""
    from channel_wise_gated_b200 import _native
    s = setup([100, 100, 100], 1, 4, 16, seed=9, garbage=False)
    want, _ = kda.mla_decode(*s)
    for what in ("low", "high", "length", "negative"):
        table, lens = s[2].clone(), s[3].clone()
        if what == "low":
            table[1, 2] = -5
        elif what == "high":
            table[1, 2] = s[1].shape[0]
        elif what == "length":
            table[1] = 0
            lens[1] = 100000
        else:
            lens[1] = -3
        o, _ = kda.mla_decode(s[0], s[1], table, lens)
        assert kda.device_status() == _native.KDA_ERR_PAGE
        keep = [0, 2]
        err = (o[keep].float() - want[keep].float()).abs().max()
        assert float(err) <= 2 ** -7 * float(want[keep].float().abs().max())


def test_scale_workspace_other_stream_and_capture(kda):
    s = setup([500, 20, 333], 2, 8, 32, seed=12)
    from channel_wise_gated_b200 import _native
    n = _native.load().kda_mla_decode_workspace_size(2, 8)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")       # NaN everywhere
    want, lw = kda.mla_decode(*s, scale=0.1, output_lse=True, workspace=ws)
    check(want, lw, *s, scale=0.1)
    with pytest.raises(kda.KdaError):
        kda.mla_decode(*s, workspace=ws[:n - 16])
    out, lse = torch.zeros_like(want), torch.zeros_like(lw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kda.mla_decode(*s, scale=0.1, o=out, lse=lse)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, lw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.mla_decode(*s, scale=0.1, o=out, lse=lse, workspace=ws)
    for lens in ([500, 20, 333], [1, 24, 352], [0, 0, 7]):
        cache = torch.nan_to_num(s[1])
        s[1].copy_(cache)
        s[3].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        keep = [i for i, L in enumerate(lens) if L <= [500, 20, 333][i]]
        check(out[keep], lse[keep], s[0][keep], s[1], s[2][keep], s[3][keep], scale=0.1)
