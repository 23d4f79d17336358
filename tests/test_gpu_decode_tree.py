"""kda_decode_tree against the recurrence run along every token's path in 64 bits.

Tolerances, before any run. The kernel computes in fp32 from exact inputs: dot products of 128
terms (relative error at most 128 * 2^-24 of the terms' absolute sum) carried through at most 16
substitution steps whose factors are at most about 1 for unit keys: 16 * 2 * 128 * 2^-24 = 2.4e-4
in the worst case, and about its square root's share in practice; 1e-4 of the largest output is
required, as everywhere for fp32 in this library. A bf16 output adds one rounding, 2^-8 of the
value itself.
"""

from __future__ import annotations

import pytest
import torch

import kda_inputs
from refs import latent as ref

pytestmark = pytest.mark.gpu

TOL_F32 = 1e-4


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


def draw(N, H, t, dtype, gates, seed):
    d = kda_inputs.make_decode(N, H, t, dtype, gates, seed=seed, device="cuda")
    x = {n: d[n].transpose(0, 1).contiguous() for n in ("q", "k", "v", "log_alpha", "beta")}
    return x, d["state"]


def check(o, o_ref):
    o_ref = o_ref.to(o.device)
    slack = TOL_F32 * o_ref.abs().max()
    if o.dtype != torch.float32:
        slack = slack + ref.half_step(o.dtype) * o_ref.abs()
    assert bool(((o.double() - o_ref).abs() <= slack).all())


def run_ref(x, state, tree):
    c = {n: t.cpu() for n, t in x.items()}
    return ref.kda_tree(c["q"], c["k"], c["v"], c["log_alpha"], c["beta"], state.cpu(),
                        None if tree is None else tree.cpu())


@pytest.mark.parametrize("N,H,t", [(1, 1, 1), (3, 2, 2), (2, 3, 5), (5, 1, 8), (2, 2, 16)])
@pytest.mark.parametrize("dtype,gates", [(torch.float32, torch.float32),
                                         (torch.bfloat16, torch.bfloat16),
                                         (torch.bfloat16, torch.float32),
                                         (torch.float32, torch.bfloat16)])
def test_tree_vs_recurrence(kda, N, H, t, dtype, gates):
    x, state = draw(N, H, t, dtype, gates, seed=300 + t)
    before = state.clone()
    tree = ref.random_tree(N, t, seed=t).cuda()
    o = kda.decode_tree(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], state, tree)
    assert torch.equal(state, before)
    check(o, run_ref(x, state, tree)[0])


@pytest.mark.parametrize("t", [1, 4, 16])
def test_chain_without_a_tree(kda, t):
    """tree None is a chain: decode_tokens' outputs up to the order of its sums."""
    x, state = draw(3, 2, t, torch.float32, torch.float32, seed=320 + t)
    o = kda.decode_tree(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], state)
    check(o, run_ref(x, state, None)[0])
    chain = torch.tensor([[(2 << j) - 1 for j in range(t)]] * 3, dtype=torch.int32, device="cuda")
    assert torch.equal(o, kda.decode_tree(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], state, chain))
    o_tok = kda.decode_tokens(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], state.clone())
    assert float((o - o_tok).abs().max()) <= 2 * TOL_F32 * float(o_tok.abs().max())


def test_siblings_do_not_see_each_other(kda):
    """Every token a root: each output is a single step's from the state; NaN in one token's
    inputs stays in its own output."""
    x, state = draw(2, 2, 6, torch.float32, torch.float32, seed=331)
    roots = torch.tensor([[1 << j for j in range(6)]] * 2, dtype=torch.int32, device="cuda")
    x["v"][:, 2] = float("nan")
    x["k"][:, 2] = float("nan")
    o = kda.decode_tree(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], state, roots)
    for j in range(6):
        if j == 2:
            assert bool(torch.isnan(o[:, j]).all())
            continue
        one = [x[n][:, j].contiguous() for n in ("q", "k", "v", "log_alpha", "beta")]
        o1 = kda.decode_step(*one, state.clone())
        assert float((o[:, j] - o1).abs().max()) <= 2 * TOL_F32 * float(o1.abs().max())


def test_strong_decay_and_none(kda):
    """log alpha of -200 (the state is forgotten: e^G underflows to 0) and of 0, in one path."""
    x, state = draw(2, 1, 4, torch.float32, torch.float32, seed=341)
    x["log_alpha"][:, 1, :, ::2] = -200.0
    x["log_alpha"][:, 2] = 0.0
    x["beta"][:, 3] = 1.0
    tree = torch.tensor([[1, 3, 7, 15], [1, 3, 5, 11]], dtype=torch.int32, device="cuda")
    o = kda.decode_tree(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], state, tree)
    check(o, run_ref(x, state, tree)[0])


def test_decay_between_tokens_behind_a_strong_one(kda):
    """log alpha of -3e4 on the first token: the decay between later tokens is not lost in the
    difference of two sums of that size (which fp32 holds to 2e-3 only)."""
    x, state = draw(2, 2, 5, torch.float32, torch.float32, seed=345)
    x["log_alpha"][:, 0] = -3e4
    tree = torch.tensor([[1, 3, 7, 11, 23], [1, 3, 5, 13, 17]], dtype=torch.int32, device="cuda")
    o = kda.decode_tree(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], state, tree)
    check(o, run_ref(x, state, tree)[0])


@pytest.mark.parametrize("t,dtype", [(3, torch.bfloat16), (8, torch.bfloat16), (12, torch.float32), (16, torch.bfloat16),
                                     (16, torch.float32)])
def test_more_states_than_resident_ctas(kda, t, dtype):
    """Every CTA walks several states (the next one's inputs and state in flight): the batch equals
    its parts, each small enough for one state per CTA."""
    x, state = draw(40, 16, t, dtype, dtype, seed=347)
    tree = ref.random_tree(40, t, seed=t + 1).cuda()
    o = kda.decode_tree(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], state, tree)
    for a in range(0, 40, 8):
        part = [x[n][a:a + 8] for n in ("q", "k", "v", "log_alpha", "beta")]
        assert torch.equal(o[a:a + 8], kda.decode_tree(*part, state[a:a + 8], tree[a:a + 8]))
    check(o[38:], run_ref({n: y[38:] for n, y in x.items()}, state[38:], tree[38:])[0])


def test_rows_that_are_no_path_are_flagged(kda):
    """A row with bits that are no path is taken by its parent (the highest bit below its own)
    and reported; the rest of the batch is untouched by it."""
    from channel_wise_gated_b200 import _native
    x, state = draw(3, 1, 4, torch.float32, torch.float32, seed=351)
    good = torch.tensor([[1, 3, 5, 13]] * 3, dtype=torch.int32, device="cuda")
    want = kda.decode_tree(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], state, good)
    bad = good.clone()
    bad[1] = torch.tensor([1, 3, 5 | 8, 4 | 2 | 8], dtype=torch.int32)   # a bit above itself; two branches
    o = kda.decode_tree(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], state, bad)
    assert kda.device_status() == _native.KDA_ERR_TREE
    assert torch.equal(o, want)


def test_captured_and_on_another_stream(kda):
    x, state = draw(4, 3, 5, torch.bfloat16, torch.bfloat16, seed=361)
    tree = ref.random_tree(4, 5, seed=9).cuda()
    args = (x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], state, tree)
    want = kda.decode_tree(*args)
    out = torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kda.decode_tree(*args, o=out)
    side.synchronize()
    assert torch.equal(out, want)
    graph, out2 = torch.cuda.CUDAGraph(), torch.zeros_like(want)
    with torch.cuda.graph(graph):
        kda.decode_tree(*args, o=out2)
    for _ in range(2):
        out2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out2, want)
    # the graph reads the tree's and the inputs' present values
    x["v"].mul_(2)
    graph.replay()
    assert torch.equal(out2, kda.decode_tree(*args))
