"""The latent-attention kernels over the lengths that people run, against softmax attention in 64 bits:
prefills on both sides of the 40 key tiles from which the second query tile starts late, decodes of many
parts per sequence and of long runs per CTA, up to 1,048,576 rows.

Tolerances, before any run. With K values per score (192 or 576), a score is off by at most K *
2^-24 of its terms' absolute sum, times the scale, and its exponent by 3 roundings of it (2^-24 |z|
each); e is the sum of the two, taken from the inputs. A weight is then off by e, 2^-8 from its rounding
to bf16 and 2^-22 from the exponential, relative, the sum it is divided by by e, and both sums are
fp32 ones of n terms in a row (n * 2^-23: matrix units may cut instead of rounding): o within
(2^-8 + 2 e + 2^-22 + n 2^-22) sum_j w_j |v_j| + 2^-8 |o|, lse within e + 2^-22 + n 2^-23 + 2^-23 |lse|.
n: a run of keys adds 8 products a tile to an accumulator (prefill: 8 of 16 keys each; decode: 2)
and at most 34 values a tile to a thread's sum; below, 34 per tile is taken for both, and a join adds
its parts.
"""

from __future__ import annotations

import math

import pytest
import torch

from refs import latent as ref

pytestmark = pytest.mark.gpu

D, SH, LAT = ref.D, ref.SHARED, ref.LATENT
W = LAT + SH
SCALE = (D + SH) ** -0.5
H8 = ref.half_step(torch.bfloat16)


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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def attend(q, keys, values):
    """One query [K], keys [L, K], values [L, C] in 64 bits on the GPU: (o, lse, sum_j w_j |v_j|, e)."""
    q = q.double()
    z = torch.cat([k.double() @ q for k in keys.split(1 << 17)]) * SCALE
    terms = max(float((k.double().abs() @ q.abs()).max()) for k in keys.split(1 << 17))
    m = z.max()
    p = torch.exp(z - m)
    l = p.sum()
    o = sum((a @ b.double()) for a, b in zip(p.split(1 << 17), values.split(1 << 17))) / l
    spread = sum((a @ b.double().abs()) for a, b in zip(p.split(1 << 17), values.split(1 << 17))) / l
    e = q.numel() * 2.0 ** -24 * terms * SCALE + 3 * 2.0 ** -24 * float(z.abs().max()) / math.log(2)
    return o, float(m + torch.log(l)), spread, e


def check_row(o, lse, q, keys, values, n):
    w, wl, spread, e = attend(q, keys, values)
    tol = (H8 + 2 * e + 2.0 ** -22 + n * 2.0 ** -22) * spread + H8 * w.abs()
    err = (o.double() - w).abs()
    assert bool((err <= tol).all()), (float((err / tol).max()), e, n)
    d = abs(float(lse) - wl)
    assert d <= e + 2.0 ** -22 + n * 2.0 ** -23 + 2.0 ** -23 * abs(wl), (d, e, n)


# ---------------------------------------------------------------------------- prefill
def heads(Tq, Tk, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    return r(Tq, H, D + SH), r(Tk, H, D), r(Tk, SH), r(Tk, H, D)


def check_prefill(o, lse, q, k, ks, v, cq, ck, causal, rows):
    """The given rows of every sequence (positions within it, those that exist)."""
    for a, b, c, d in zip(cq, cq[1:], ck, ck[1:]):
        for i in sorted({r if r >= 0 else b - a + r for r in rows}):
            if not 0 <= i < b - a:
                continue
            last = min(d, c + i + (d - c) - (b - a) + 1) if causal else d
            for h in range(q.shape[1]):
                if last <= c:
                    assert bool((o[a + i, h] == 0).all()) and float(lse[a + i, h]) == -math.inf
                    continue
                keys = torch.cat([k[c:last, h], ks[c:last]], 1)
                check_row(o[a + i, h], lse[a + i, h], q[a + i, h], keys, v[c:last, h],
                          34 * ((last - c + 127) // 128))


ROWS = [0, 1, 31, 63, 64, 127, 128, 129, 200, 255, 256, 299, -1]


@pytest.mark.parametrize("lq", [1, 128, 129, 300])
@pytest.mark.parametrize("lk", [4992, 4993, 5101, 5120, 5121, 5300, 8192])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_around_the_late_start(kda, lq, lk, causal):
    """39 to 64 key tiles; a second query tile with all rows, one, and none."""
    q, k, ks, v = heads(lq, lk, 1, lq + lk)
    o, lse = kda.mla_prefill(q, k, ks, v, causal=causal, output_lse=True)
    check_prefill(o, lse, q, k, ks, v, [0, lq], [0, lk], causal, ROWS)
    again, l2 = kda.mla_prefill(q, k, ks, v, causal=causal, output_lse=True)
    assert torch.equal(o, again) and torch.equal(lse, l2)


def test_prefill_packed_over_the_late_start(kda):
    """Sequences on both sides of it in one batch, one without keys."""
    lq, lk = [130, 1, 300, 64, 5, 257], [5200, 300, 5000, 64, 0, 7777]
    cq, ck = [0], [0]
    for a, b in zip(lq, lk):
        cq.append(cq[-1] + a)
        ck.append(ck[-1] + b)
    q, k, ks, v = heads(cq[-1], ck[-1], 2, 5)
    o, lse = kda.mla_prefill(q, k, ks, v, cu_seqlens=i32(cq), cu_seqlens_k=i32(ck), output_lse=True)
    check_prefill(o, lse, q, k, ks, v, cq, ck, True, ROWS)


def test_prefill_whole_prompt(kda):
    """6,000 tokens and 2 heads: pairs of query tiles below and above the late start."""
    T = 6000
    q, k, ks, v = heads(T, T, 2, 6)
    o, lse = kda.mla_prefill(q, k, ks, v, output_lse=True)
    check_prefill(o, lse, q, k, ks, v, [0, T], [0, T], True,
                  [0, 1, 127, 128, 4863, 4864, 4991, 4992, 5000, 5119, 5120, 5375, 5376, 5999])


def test_prefill_rising_scores_over_the_late_start(kda):
    """The reference moves in every other tile of 45, late start included."""
    lq, lk = 200, 5700
    q, k, ks, v = heads(lq, lk, 1, 7)
    q[..., 0] = 8.0
    k[..., 0] = (torch.arange(lk, device="cuda") // 32)[:, None].bfloat16()     # to 178, exact in bf16
    o, lse = kda.mla_prefill(q, k, ks, v, output_lse=True)
    check_prefill(o, lse, q, k, ks, v, [0, lq], [0, lk], True, ROWS)


@pytest.mark.parametrize("lk", [131072, 1048576 - 5])
def test_prefill_behind_a_long_context(kda, lk):
    lq = 3
    q, k, ks, v = heads(lq, lk, 1, 8)
    o, lse = kda.mla_prefill(q, k, ks, v, output_lse=True)
    check_prefill(o, lse, q, k, ks, v, [0, lq], [0, lk], True, [0, 1, 2])


# ---------------------------------------------------------------------------- decode
def cached(lens, t, H, page, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-x // page) for x in lens]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32, device="cuda")
    cache = torch.randn((pool, page, W), generator=g, device="cuda", dtype=torch.bfloat16)
    at = 0
    for n, k in enumerate(need):
        table[n, :k] = order[at:at + k]
        at += k
        if lens[n] % page:
            cache[table[n, k - 1].long(), lens[n] % page:] = float("nan")     # rows behind the last
    q = (torch.randn((len(lens), t, H, W), generator=g, device="cuda") * 0.577).bfloat16()
    return q, cache, table, i32(lens)


def rows_of(cache, table, n, L):
    page = cache.shape[1]
    return cache[table[n, :-(-L // page)].long()].reshape(-1, W)[:L]


def check_decode(o, lse, q, cache, table, lens, which, tree=None, tokens=None):
    L_all, t = lens.tolist(), q.shape[1]
    tiles = sum(-(-x // 32) for x in L_all) * -(-t * q.shape[2] // 16)
    for n in which:
        L = L_all[n]
        rows = rows_of(cache, table, n, L)
        for j in range(t) if tokens is None else tokens:
            bits = (2 << j) - 1 if tree is None else int(tree[n, j])
            seen = torch.ones(L, dtype=torch.bool, device="cuda")
            for i in range(t):
                if not (bits >> i) & 1 and L - t + i >= 0:
                    seen[L - t + i] = False
            r = rows[seen]
            for h in range(q.shape[2]):
                if r.shape[0] == 0:
                    assert bool((o[n, j, h] == 0).all()) and float(lse[n, j, h]) == -math.inf
                    continue
                # (a run is no longer than the sequence, nor than the line's share of one of 100 CTAs and more)
                n_add = 34 * min(-(-L // 32), -(-tiles // 100) + 3) + 160
                check_row(o[n, j, h], lse[n, j, h], q[n, j, h], r, r[:, :LAT], n_add)


@pytest.mark.parametrize("L", [3071, 3100, 5003, 20000, 40001])
@pytest.mark.parametrize("t,H", [(1, 1), (2, 2), (1, 40), (3, 40)])
def test_decode_many_parts_per_row(kda, L, t, H):
    """One sequence over 32 to 148 CTAs: the split join's later rounds of parts."""
    s = cached([L], t, H, 64, L + H)
    o, lse = kda.mla_decode(*s, output_lse=True)
    check_decode(o, lse, *s, [0])
    again, l2 = kda.mla_decode(*s, output_lse=True)
    assert torch.equal(o, again) and torch.equal(lse, l2)


@pytest.mark.parametrize("page", [8, 48, 64])
@pytest.mark.parametrize("long_at", [0, 5, 11])
def test_decode_one_long_among_short(kda, page, long_at):
    """12 sequences, one of 12,001 rows: the join that gives a row to one warp, with 90 and more parts."""
    lens = [37, 1, 200, 64, 0, 33, 5, 90, 128, 300, 31, 2]
    lens[long_at] = 12001
    s = cached(lens, 1, 3, page, page + long_at)
    o, lse = kda.mla_decode(*s, output_lse=True)
    check_decode(o, lse, *s, range(12))


@pytest.mark.parametrize("t,H", [(1, 2), (2, 24), (1, 64), (5, 20)])
def test_decode_long_runs_with_rising_scores(kda, t, H):
    """24 sequences of some 20,000 rows: 100 tiles per CTA and group of rows, a reference that moves
    about every 16 tiles."""
    lens = [20000 - 13 * i for i in range(24)]
    q, cache, table, ln = cached(lens, t, H, 64, H)
    q[..., 0] = 12.0
    for n, L in enumerate(lens):
        p = torch.arange(L, device="cuda")
        cache[table[n, p // 64].long(), p % 64, 0] = (p // 80).bfloat16()       # to 249, exact in bf16
    o, lse = kda.mla_decode(q, cache, table, ln, output_lse=True)
    few = torch.arange(0, H, max(1, H // 3), device="cuda")
    for n in (0, 7, 12, 23):
        check_decode(o[n:n + 1, :, few], lse[n:n + 1, :, few], q[n:n + 1, :, few], cache, table[n:n + 1], ln[n:n + 1],
                     [0], tokens=[0, t - 1])


@pytest.mark.parametrize("L", [131072, 1048576])
def test_decode_long_context(kda, L):
    s = cached([L, 100], 2, 2, 64, 9)
    o, lse = kda.mla_decode(*s, output_lse=True)
    check_decode(o, lse, *s, [0, 1])


@pytest.mark.parametrize("tree", [False, True])
def test_decode_most_rows(kda, tree):
    """16 tokens x 128 heads: 2,048 rows a sequence in 32 groups; an empty slot, a prefix shorter than
    the tokens."""
    lens, t, H = [70, 16, 0, 9, 333], 16, 128
    s = cached(lens, t, H, 16, 10)
    bits = ref.random_tree(len(lens), t, seed=4).cuda() if tree else None
    o, lse = kda.mla_decode(*s, tree=bits, output_lse=True)
    hs = torch.tensor([0, 3, 64, 127], device="cuda")
    check_decode(o[:, :, hs], lse[:, :, hs], s[0][:, :, hs], *s[1:], [0, 1, 3, 4], tree=bits)
    assert bool((o[2] == 0).all()) and bool((lse[2] == -math.inf).all())
    # the other heads: each the same as in a call of its own few
    part = torch.arange(40, 48, device="cuda")
    o1, l1 = kda.mla_decode(s[0][:, :, part].contiguous(), *s[1:], tree=bits, output_lse=True)
    fin = torch.isfinite(l1)
    assert torch.equal(fin, torch.isfinite(lse[:, :, part]))
    assert float((l1 - lse[:, :, part])[fin].abs().max()) <= 1e-4
    assert float((o1.float() - o[:, :, part].float()).abs().max()) <= 2 * H8 * float(o1.float().abs().max())


@pytest.mark.parametrize("page,most", [(1 << 15, 1 << 15), (8, 1 << 20)])
def test_widest_page_table(kda, page, most):
    """A table for 2^30 rows a sequence (or of a million pages), of which a few are there; the rest of its
    entries are -1 and never read."""
    L = 1000
    used = -(-L // page)
    table = torch.full((2, most), -1, dtype=torch.int32, device="cuda")
    table[0, :used] = torch.arange(used, device="cuda", dtype=torch.int32)
    table[1, :used] = torch.arange(used, 2 * used, device="cuda", dtype=torch.int32)
    cache = torch.full((2 * used, page, W), float("nan"), device="cuda", dtype=torch.bfloat16)
    x = torch.randn(2 * L, W, device="cuda").bfloat16()
    lens = i32([L, L])
    kda.mla_append(x, None, cache, table, lens)
    q = (torch.randn(2, 1, 4, W, device="cuda") * 0.577).bfloat16()
    o, lse = kda.mla_decode(q, cache, table, lens, output_lse=True)
    check_decode(o, lse, q, cache, table, lens, [0, 1])
