"""kda_mla_prefill against softmax attention in 64 bits.

Tolerances, before any run. Scores: fp32 sums of 192 exact products of bf16 values, relative
error of the terms' absolute sum under 192 * 2^-24 = 1.2e-5; for unit-normal inputs that sum is
about 120 before the scale of 0.072, so a score, and with it lse, is off by at most 1e-4 (the
exponential's and the logarithm's own errors, 2^-22, are below that). Output: every weight is
off by 1e-4 from its score and 2^-8 from its rounding to bf16, relative, so o is off by at
most (2^-8 + 2e-4) sum_j w_j |v_j|, plus the output's rounding, 2^-8 |o|. sum_j w_j |v_j| is
computed along with the reference.
"""

from __future__ import annotations

import math

import pytest
import torch

from refs import latent as ref

pytestmark = pytest.mark.gpu

D, SH = ref.D, ref.SHARED
SCALE = (D + SH) ** -0.5


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


def draw(Tq, Tk, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    return r(Tq, H, D + SH), r(Tk, H, D), r(Tk, SH), r(Tk, H, D)


def cu(lens):
    c = [0]
    for x in lens:
        c.append(c[-1] + x)
    return c


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(o, lse, q, k, ks, v, cq, ck, causal=True, scale=SCALE):
    c = [t.cpu() for t in (q, k, ks, v)]
    o_ref, lse_ref = ref.mla_prefill(*c, cq, ck, causal, scale)
    spread, _ = ref.mla_prefill(*c[:3], c[3].abs(), cq, ck, causal, scale)
    h = ref.half_step(torch.bfloat16)
    err = (o.cpu().double() - o_ref).abs()
    assert bool((err <= (h + 2e-4) * spread + h * o_ref.abs()).all()), float((err - h * o_ref.abs()).max())
    if lse is not None:
        inf = torch.isinf(lse_ref)
        assert torch.equal(torch.isinf(lse.cpu()), inf)
        assert bool((lse.cpu()[inf] < 0).all())
        assert float((lse.cpu().double() - lse_ref)[~inf].abs().max() if (~inf).any() else 0.0) <= 1e-4


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 384, 500, 770])
@pytest.mark.parametrize("H", [1, 3])
def test_one_sequence(kda, T, H):
    q, k, ks, v = draw(T, T, H, T)
    o, lse = kda.mla_prefill(q, k, ks, v, output_lse=True)
    check(o, lse, q, k, ks, v, [0, T], [0, T])


@pytest.mark.parametrize("lens", [[1, 1, 1], [5, 0, 130, 256, 1], [257, 255, 3], [64] * 40, [300]])
def test_packed(kda, lens):
    c = cu(lens)
    q, k, ks, v = draw(c[-1], c[-1], 2, 7)
    o, lse = kda.mla_prefill(q, k, ks, v, cu_seqlens=i32(c), output_lse=True)
    check(o, lse, q, k, ks, v, c, c)


@pytest.mark.parametrize("lq,lk", [([1], [300]), ([130], [131]), ([17, 200, 1], [400, 200, 129]),
                                   ([200, 90, 5], [100, 0, 3]), ([300], [40])])
@pytest.mark.parametrize("causal", [True, False])
def test_queries_and_keys_of_different_number(kda, lq, lk, causal):
    """A prefix before the queries; fewer keys than queries (the first rows see none); no keys."""
    cq, ck = cu(lq), cu(lk)
    q, k, ks, v = draw(cq[-1], ck[-1], 2, 11)
    o, lse = kda.mla_prefill(q, k, ks, v, cu_seqlens=i32(cq), cu_seqlens_k=i32(ck), causal=causal,
                             output_lse=True)
    check(o, lse, q, k, ks, v, cq, ck, causal)
    if len(lq) == 1:
        o1, lse1 = kda.mla_prefill(q, k, ks, v, causal=causal, output_lse=True)
        assert torch.equal(o, o1) and torch.equal(lse, lse1)


def test_no_keys_and_no_queries(kda):
    q, k, ks, v = draw(5, 0, 2, 3)
    o, lse = kda.mla_prefill(q, k, ks, v, output_lse=True)
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())
    q, k, ks, v = draw(0, 5, 2, 3)
    o, lse = kda.mla_prefill(q, k, ks, v, output_lse=True)
    assert o.shape == (0, 2, D) and lse.shape == (0, 2)


def test_strided_views(kda):
    """k and v as halves of one projection, q a slice, the shared part out of a latent row."""
    T, H = 200, 3
    q, k, ks, v = draw(T, T, H, 21)
    kv = torch.cat([k, v], -1)
    wide = torch.zeros(T, H, 256, device="cuda", dtype=torch.bfloat16)
    wide[..., 64:256] = q
    rows = torch.zeros(T, 576, device="cuda", dtype=torch.bfloat16)
    rows[:, 512:] = ks
    a, _ = kda.mla_prefill(q, k, ks, v)
    b, _ = kda.mla_prefill(wide[..., 64:], kv[..., :D], rows[:, 512:], kv[..., D:])
    assert torch.equal(a, b)
    qh = q.transpose(0, 1).contiguous().transpose(0, 1)     # head-major storage
    c, _ = kda.mla_prefill(qh, k, ks, v)
    assert torch.equal(a, c)


@pytest.mark.parametrize("lens", [[100, 60], [1, 31], [129, 127]])
def test_other_sequences_values_never_matter(kda, lens):
    """NaN and infinities in one sequence's keys and values leave the others bit for bit."""
    c = cu(lens)
    q, k, ks, v = draw(c[-1], c[-1], 2, 31)
    a, la = kda.mla_prefill(q, k, ks, v, cu_seqlens=i32(c), output_lse=True)
    b0 = c[1]
    k[b0:], ks[b0:], v[b0:], q[b0:] = float("nan"), float("inf"), float("nan"), float("nan")
    b, lb = kda.mla_prefill(q, k, ks, v, cu_seqlens=i32(c), output_lse=True)
    assert torch.equal(a[:b0], b[:b0]) and torch.equal(la[:b0], lb[:b0])
    assert bool(torch.isnan(b[b0:]).all())


def test_rising_scores_and_large_ones(kda):
    """Keys whose scores grow along the sequence, so the running maximum moves in every tile,
    and scores of some hundreds. lse: scores up to 400 in fp32 sums whose terms reach 400 / scale
    in one product are exact to 192 * 2^-24 of it, 5e-3."""
    T, H = 700, 1
    q, k, ks, v = draw(T, T, H, 41)
    q = (q * 0.1).bfloat16()
    q[..., 0] = 8.0
    k[..., 0] = (torch.arange(T, device="cuda")[:, None] * 1.0).bfloat16()
    o, lse = kda.mla_prefill(q, k, ks, v, output_lse=True)
    o_ref, lse_ref = ref.mla_prefill(*[t.cpu() for t in (q, k, ks, v)], [0, T], [0, T], True, SCALE)
    assert float((lse.cpu().double() - lse_ref).abs().max()) <= 5e-3
    spread, _ = ref.mla_prefill(*[t.cpu() for t in (q, k, ks, v.abs())], [0, T], [0, T], True, SCALE)
    h = ref.half_step(torch.bfloat16)
    assert bool(((o.cpu().double() - o_ref).abs() <= (h + 1e-2) * spread + h * o_ref.abs()).all())
    # falling scores: the first tile's maximum stays
    k2 = k.flip(0).contiguous()
    o, lse = kda.mla_prefill(q, k2, ks, v, output_lse=True)
    o_ref, lse_ref = ref.mla_prefill(*[t.cpu() for t in (q, k2, ks, v)], [0, T], [0, T], True, SCALE)
    assert float((lse.cpu().double() - lse_ref).abs().max()) <= 5e-3


def test_parts_join_by_their_lse(kda):
    """A prefix without causal and the rest with it, joined, are the whole."""
    T, P, H = 300, 170, 2
    q, k, ks, v = draw(T, T, H, 51)
    n = T - P
    whole, lw = kda.mla_prefill(q[P:], k, ks, v, output_lse=True)
    a, la = kda.mla_prefill(q[P:], k[:P], ks[:P], v[:P], causal=False, output_lse=True)
    b, lb = kda.mla_prefill(q[P:], k[P:], ks[P:], v[P:], output_lse=True)
    l = torch.logaddexp(la, lb)
    assert float((l - lw).abs().max()) <= 2e-4
    j = torch.exp(la - l)[..., None] * a.float() + torch.exp(lb - l)[..., None] * b.float()
    h = ref.half_step(torch.bfloat16)
    # three roundings of outputs, and the weights' roundings of both ways
    spread = ref.mla_prefill(*[t.cpu() for t in (q[P:], k, ks, v.abs())], [0, n], [0, T], True, SCALE)[0]
    assert bool(((j - whole.float()).abs().cpu() <= 4 * (h + 2e-4) * spread).all())


def test_scale_other_stream_and_capture(kda):
    q, k, ks, v = draw(333, 333, 4, 61)
    c = i32([0, 100, 333])
    want, lw = kda.mla_prefill(q, k, ks, v, cu_seqlens=c, scale=0.2, output_lse=True)
    check(want, lw, q, k, ks, v, [0, 100, 333], [0, 100, 333], scale=0.2)
    out, lse = torch.zeros_like(want), torch.zeros_like(lw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kda.mla_prefill(q, k, ks, v, cu_seqlens=c, scale=0.2, o=out, lse=lse)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, lw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.mla_prefill(q, k, ks, v, cu_seqlens=c, scale=0.2, o=out, lse=lse)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    c.copy_(i32([0, 200, 333]))      # the graph reads the present lengths
    graph.replay()
    check(out, lse, q, k, ks, v, [0, 200, 333], [0, 200, 333], scale=0.2)


def test_bad_cu_seqlens_stay_in_bounds(kda):
    from channel_wise_gated_b200 import _native
    q, k, ks, v = draw(100, 100, 1, 71)
    for bad in ([0, 60, 50, 100], [0, 40, 300, 100], [5, 40, 60, 90], [0, -7, 60, 100]):
        kda.mla_prefill(q, k, ks, v, cu_seqlens=i32(bad))
        assert kda.device_status() == _native.KDA_ERR_SEQLENS


@pytest.mark.parametrize("n_seqs", [2, 40])
def test_rows_behind_the_last_sequence_are_left(kda, n_seqs):
    """A batch padded behind its last sequence: outputs there stay, the device reports it."""
    from channel_wise_gated_b200 import _native
    cu = [9 * n for n in range(n_seqs + 1)]
    real, total = cu[-1], cu[-1] + 21
    q, k, ks, v = draw(total, total, 2, 73)
    want, lw = kda.mla_prefill(q[:real], k[:real], ks[:real], v[:real], cu_seqlens=i32(cu), output_lse=True)
    out = torch.full((total, 2, 128), 7.0, device="cuda").bfloat16()
    lse = torch.full((total, 2), 7.0, device="cuda")
    kda.mla_prefill(q, k, ks, v, cu_seqlens=i32(cu), o=out, lse=lse)
    assert kda.device_status() == _native.KDA_ERR_SEQLENS
    assert torch.equal(out[:real], want) and torch.equal(lse[:real], lw)
    assert bool((out[real:] == 7).all()) and bool((lse[real:] == 7).all())
