"""The operators of a hybrid model's step together, as a serving loop calls them.

* A prompt: latents appended, the expanded form over the up-projected keys and values; then the
  absorbed form of a new token equals the expanded one over all tokens (the same mathematics with
  the up-projections moved), within the roundings that each way makes.
* A tree of drafted tokens through both kinds of layer: outputs of every node; then the accepted
  path is applied (decode_tokens on the state, append over the drafted rows) and must leave what
  the plain token-by-token path leaves.
"""

from __future__ import annotations

import pytest
import torch

import kda_inputs
from refs import latent as ref

pytestmark = pytest.mark.gpu

D, LAT, SH, W = ref.D, ref.LATENT, ref.SHARED, 576


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


def test_expanded_and_absorbed_agree(kda):
    """Tolerance: the expanded way rounds k, v (2^-8 each, scores of spread 1 from 192 products:
    about 2^-8 / sqrt(192) * a few of their spread) and the weights; the absorbed way the query in
    the latent space, the weights and the latent output, 2^-8 each, then a plain projection.
    Each of these 2^-8 errors is a random one over hundreds of terms, so 3 * 2^-8 of the largest
    output bounds their sum with room; a wrong mask or position is off by its whole size."""
    torch.manual_seed(0)
    H, T, page = 8, 333, 64
    x = torch.randn(T, W, device="cuda").bfloat16()
    w = 0.5 + torch.rand(LAT, device="cuda")
    uk = (torch.randn(H, LAT, D, device="cuda") / LAT ** 0.5).bfloat16()
    uv = (torch.randn(H, LAT, D, device="cuda") / LAT ** 0.5).bfloat16()
    q = torch.randn(T, H, D + SH, device="cuda").bfloat16()
    pages = -(-T // page)
    table = torch.randperm(pages + 2, device="cuda")[:pages].to(torch.int32)[None]
    cache = torch.zeros(pages + 2, page, W, device="cuda", dtype=torch.bfloat16)
    lat = kda.mla_append(x, w, cache, table, i32([T]), output_latent=True)
    k = torch.einsum("tl,hld->thd", lat.float(), uk.float()).bfloat16()
    v = torch.einsum("tl,hld->thd", lat.float(), uv.float()).bfloat16()
    o, lse = kda.mla_prefill(q, k, x[:, LAT:], v, output_lse=True)
    # the last four tokens through the cache
    t = 4
    qa = torch.cat([torch.einsum("thd,hld->thl", q[-t:, :, :D].float(), uk.float()),
                    q[-t:, :, D:].float()], -1).bfloat16()[None]
    oa, la = kda.mla_decode(qa, cache, table, i32([T]), output_lse=True)
    back = torch.einsum("thl,hld->thd", oa[0].float(), uv.float())
    tol = 3 * ref.half_step(torch.bfloat16)
    assert float((back - o[-t:].float()).abs().max()) <= tol * float(o.float().abs().max())
    assert float((la[0] - lse[-t:]).abs().max()) <= 3 * ref.half_step(torch.bfloat16)


def test_tree_step_and_its_commit(kda):
    """Verify trees of drafted tokens in a latent-attention layer and a KDA layer, then apply one
    accepted path per sequence: caches and states equal those of the tokens taken one by one."""
    torch.manual_seed(1)
    N, H, t, page = 3, 2, 6, 16
    prefix = [37, 16, 5]
    tree = ref.random_tree(N, t, seed=5).cuda()
    dec = kda_inputs.make_decode(N, H, t, torch.float32, torch.float32, seed=9, device="cuda")
    kx = {n: dec[n].transpose(0, 1).contiguous() for n in ("q", "k", "v", "log_alpha", "beta")}
    state = dec["state"]
    # the latent layer's cache: prefixes, then the drafted rows behind them
    most = max(-(-(p + t) // page) for p in prefix)
    table = torch.randperm(N * most, device="cuda").view(N, most).to(torch.int32)
    cache = torch.zeros(N * most, page, W, device="cuda", dtype=torch.bfloat16)
    w = 0.5 + torch.rand(LAT, device="cuda")
    first = torch.randn(sum(prefix), W, device="cuda").bfloat16()
    cu = [0]
    for p in prefix:
        cu.append(cu[-1] + p)
    kda.mla_append(first, w, cache, table, i32(prefix), cu_seqlens=i32(cu))
    draft = torch.randn(N, t, W, device="cuda").bfloat16()
    lens = i32([p + t for p in prefix])
    kda.mla_append(draft.view(N * t, W), w, cache, table, lens)
    q = (torch.randn(N, t, H, W, device="cuda") * 0.577).bfloat16()
    o, _ = kda.mla_decode(q, cache, table, lens, tree=tree)
    ok = kda.decode_tree(kx["q"], kx["k"], kx["v"], kx["log_alpha"], kx["beta"], state, tree)
    o_ref, _ = ref.mla_decode(q.cpu(), cache.cpu(), table.cpu(), lens.cpu(), tree.cpu(), (D + SH) ** -0.5)
    assert float((o.cpu().double() - o_ref).abs().max()) <= 2 ** -6 * float(o_ref.abs().max())
    # the longest path of every tree is accepted
    for n in range(N):
        bits = tree[n].tolist()
        last = max(range(t), key=lambda j: bin(bits[j]).count("1"))
        path = [j for j in range(t) if (bits[last] >> j) & 1]
        m = len(path)
        # KDA layer: the tokens of the path in place; the outputs are those the tree gave
        s1 = state[n:n + 1].clone()
        part = [kx[x][n:n + 1, path].contiguous() for x in ("q", "k", "v", "log_alpha", "beta")]
        op = kda.decode_tokens(*part, s1)
        assert float((op[0] - ok[n, path]).abs().max()) <= 2e-4 * float(op.abs().max())
        # latent layer: the accepted rows over the drafted ones
        one = i32([prefix[n] + m])
        kda.mla_append(draft[n, path].contiguous(), w, cache, table[n:n + 1].contiguous(), one)
        qp = q[n:n + 1, path].contiguous()
        oc, _ = kda.mla_decode(qp, cache, table[n:n + 1].contiguous(), one)
        # the chain over the compacted rows is the path through the tree (rounded twice: 2 * 2^-8)
        assert float((oc[0].float() - o[n, path].float()).abs().max()) <= \
            2 ** -6 * float(oc.float().abs().max())


def test_two_graphs_one_workspace(kda):
    """Two captured calls that share a workspace, replayed in turn on one stream, and once more
    with other lengths: each keeps its own results."""
    torch.manual_seed(2)
    page, H = 32, 8
    cache = torch.randn(80, page, W, device="cuda").bfloat16()
    ta = torch.arange(40, device="cuda", dtype=torch.int32)[None]
    tb = torch.arange(40, 80, device="cuda", dtype=torch.int32).view(2, 20)
    la, lb = i32([1200]), i32([600, 37])
    qa = (torch.randn(1, 1, H, W, device="cuda") * 0.577).bfloat16()
    qb = (torch.randn(2, 2, H, W, device="cuda") * 0.577).bfloat16()
    ws = torch.empty(max(kda.mla_decode_workspace_size(1, H), kda.mla_decode_workspace_size(2, H)),
                     dtype=torch.uint8, device="cuda")
    oa, ob = torch.zeros(1, 1, H, LAT, device="cuda", dtype=torch.bfloat16), \
        torch.zeros(2, 2, H, LAT, device="cuda", dtype=torch.bfloat16)
    kda.mla_decode(qa, cache, ta, la, o=oa, workspace=ws)       # (warm)
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        kda.mla_decode(qa, cache, ta, la, o=oa, workspace=ws)
    with torch.cuda.graph(gb):
        kda.mla_decode(qb, cache, tb, lb, o=ob, workspace=ws)
    for lens_a, lens_b in (([1200], [600, 37]), ([77], [2, 640])):
        la.copy_(i32(lens_a))
        lb.copy_(i32(lens_b))
        wa, _ = kda.mla_decode(qa, cache, ta, la)
        wb, _ = kda.mla_decode(qb, cache, tb, lb)
        for _ in range(3):
            ga.replay()
            gb.replay()
        torch.cuda.synchronize()
        assert torch.equal(oa, wa) and torch.equal(ob, wb)


def test_calls_on_two_streams_at_once(kda):
    """The same operators from two streams at the same time, each with its own workspace."""
    torch.manual_seed(3)
    page, H = 64, 16
    cache = torch.randn(64, page, W, device="cuda").bfloat16()
    table = torch.arange(64, device="cuda", dtype=torch.int32).view(4, 16)
    lens = i32([1000, 700, 300, 1024])
    q = [(torch.randn(4, 1, H, W, device="cuda") * 0.577).bfloat16() for _ in range(2)]
    want = [kda.mla_decode(x, cache, table, lens)[0] for x in q]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(kda.mla_decode(q[i], cache, table, lens)[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


@pytest.mark.parametrize("N", [33, 700, 3001])
def test_many_short_sequences(kda, N):
    """Packed batches of thousands of sequences, some empty: appended, attended in both forms. Every
    sequence's result is that of a small batch of it and its neighbours."""
    torch.manual_seed(4)
    page, H = 8, 2
    g = torch.Generator().manual_seed(N)
    lens = torch.randint(0, 6, (N,), generator=g).tolist()
    lens[5], lens[N - 1] = 300, 270
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    T = cu[-1]
    need = [-(-x // page) for x in lens]
    table = torch.zeros(N, max(need), dtype=torch.int32)
    at = 0
    for n, k in enumerate(need):
        table[n, :k] = torch.arange(at, at + k)
        at += k
    table = table.cuda()
    cache = torch.zeros(at, page, W, device="cuda", dtype=torch.bfloat16)
    x = torch.randn(T, W, device="cuda").bfloat16()
    kda.mla_append(x, None, cache, table, i32(lens), cu_seqlens=i32(cu))
    for n in (0, 5, N // 2, N - 1):
        rows = cache[table[n, :need[n]].long()].reshape(-1, W)[:lens[n]]
        assert torch.equal(rows, x[cu[n]:cu[n + 1]])
    q = torch.randn(T, H, D + SH, device="cuda").bfloat16()
    k, v = torch.randn(T, H, D, device="cuda").bfloat16(), torch.randn(T, H, D, device="cuda").bfloat16()
    o, lse = kda.mla_prefill(q, k, x[:, LAT:], v, cu_seqlens=i32(cu), output_lse=True)
    qd = (torch.randn(N, 1, H, W, device="cuda") * 0.577).bfloat16()
    od, ld = kda.mla_decode(qd, cache, table, i32(lens), output_lse=True)
    for a in (0, N // 2 - 3, N - 9):
        b = a + 9
        s, e = cu[a], cu[b]
        part = i32([c - s for c in cu[a:b + 1]])
        o1, l1 = kda.mla_prefill(q[s:e], k[s:e], x[s:e, LAT:], v[s:e], cu_seqlens=part, output_lse=True)
        assert torch.equal(o[s:e], o1) and torch.equal(lse[s:e], l1)
        od1, ld1 = kda.mla_decode(qd[a:b].contiguous(), cache, table[a:b].contiguous(), i32(lens[a:b]), output_lse=True)
        # (a run's border may cut a long one elsewhere: fp32 sums in another order)
        fin = torch.isfinite(ld1)
        assert torch.equal(fin, torch.isfinite(ld[a:b]))
        assert float((ld[a:b] - ld1)[fin].abs().max()) <= 1e-5 * 10
        assert float((od[a:b].float() - od1.float()).abs().max()) <= 2 ** -7 * float(od1.float().abs().max())
