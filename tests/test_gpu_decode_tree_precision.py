"""The precision that kda_decode_tree states, where it shows: products with the state that cancel.

Tolerance, before any run, from the parts that the kernel takes of each factor. A rounding to p bits
leaves 2^-p of the value (bf16 p = 8, tf32 p = 11), so a = a1 + a2 + r with |a2| <= 2^-p |a| and |r| <=
2^-2p |a|; without a2 b2 a product is off by at most 3 * 2^-2p |a b|. The rows x = k e^G, q e^G are
themselves rounded to fp32 after an exponential (4 * 2^-24), and the sums are of fp32 (128 terms
and three partial sums: 132 * 2^-24): together eps_p = 3 * 2^-2p + 136 * 2^-24 of sum_c |x_c S_c|.
These go through the substitution with the coefficients A and P: a delta is off by beta times its
product's error plus the sum over its ancestors of |A| times theirs, an output by its product's plus the
sum of |P| times the deltas'. A and P are themselves fp32 sums of 128 terms (136 * 2^-24 of their
terms' absolute sum), and the substitution adds 16 * 2^-24 of its terms. A bf16 output is rounded
once (2^-8).
"""

from __future__ import annotations

import pytest
import torch

from refs import latent as ref

pytestmark = pytest.mark.gpu

D, U = 128, 2.0 ** -24


@pytest.fixture(scope="module")
def kda():
    from channel_wise_gated_b200 import build
    build.build()
    import channel_wise_gated_b200 as m
    return m


def bound(x, state, tree, o_ref, p, dtype):
    """The tolerance above for every output, [N, t, H, 128]."""
    q, k, v, la, be = (x[n].double() for n in ("q", "k", "v", "log_alpha", "beta"))
    S = state.double()
    N, t, H, _ = q.shape
    eps = 3 * 2.0 ** (-2 * p) + 136 * U
    tol = torch.zeros(N, t, H, D, dtype=torch.float64)
    for n in range(N):
        bits = [(2 << j) - 1 for j in range(t)] if tree is None else [int(b) for b in tree[n]]
        delta, err = [None] * t, [None] * t
        for r in range(t):
            path = [i for i in range(r + 1) if (bits[r] >> i) & 1]
            g = {}                      # decay from each ancestor to r
            acc = torch.zeros(H, D, dtype=torch.float64)
            for i in reversed(path):
                g[i] = acc.exp()
                acc = acc + la[n, i]
            xk, xq = k[n, r] * acc.exp(), q[n, r] * acc.exp()
            beta = be[n, r][:, None]
            uk = torch.einsum("hc,hcv->hv", xk, S[n])
            d, e = beta * (v[n, r] - uk), beta * eps * torch.einsum("hc,hcv->hv", xk.abs(), S[n].abs())
            mag = beta * (v[n, r].abs() + uk.abs())
            y = eps * torch.einsum("hc,hcv->hv", xq.abs(), S[n].abs())
            for i in path[:-1]:
                A = beta[:, 0] * (k[n, r] * k[n, i] * g[i]).sum(-1)
                Aa = beta[:, 0] * (k[n, r] * k[n, i] * g[i]).abs().sum(-1)
                d = d - A[:, None] * delta[i]
                e = e + A.abs()[:, None] * err[i] + 136 * U * Aa[:, None] * (delta[i].abs() + err[i])
                mag = mag + A.abs()[:, None] * delta[i].abs()
            delta[r], err[r] = d, e + 16 * U * mag
            for i in path:
                Pa = (q[n, r] * k[n, i] * g[i]).abs().sum(-1)
                P = (q[n, r] * k[n, i] * g[i]).sum(-1).abs()
                y = y + P[:, None] * err[i] + (136 + 16) * U * Pa[:, None] * (delta[i].abs() + err[i])
            tol[n, r] = y
    if dtype != torch.float32:
        tol = tol * (1 + ref.half_step(dtype)) + ref.half_step(dtype) * o_ref.abs()
    return tol


def draw(N, H, t, dtype, seed, cancel):
    g = torch.Generator().manual_seed(seed)
    unit = lambda a: torch.nn.functional.normalize(a, dim=-1)
    k = unit(torch.randn(N, t, H, D, generator=g)).to(dtype)
    q = unit(torch.randn(N, t, H, D, generator=g)).to(dtype)
    S = 64.0 * torch.randn(N, H, D, D, generator=g)
    la = torch.nn.functional.logsigmoid(torch.randn(N, t, H, D, generator=g) + 3.0)
    be = torch.sigmoid(torch.randn(N, t, H, generator=g))
    v = torch.randn(N, t, H, D, generator=g).to(dtype)
    if cancel:
        # one query for all tokens and no decay, the state without its share along the query: q^T S is
        # a rounding of sums of |q||S|, about 500, and what is read out the tokens' own deltas
        q = q[:, :1].expand(N, t, H, D).contiguous()
        la.zero_()
        u = q[:, 0].double()
        S = S.double()
        for _ in range(2):
            S = S - torch.einsum("nhc,nhv->nhcv", u, torch.einsum("nhc,nhcv->nhv", u, S)) / \
                (u * u).sum(-1)[..., None, None]
        S = S.float()
        k = unit(k.double() - torch.einsum("nthc,nthc->nth", k.double(), q.double())[..., None] * q.double()).to(dtype)
    return {"q": q, "k": k, "v": v, "log_alpha": la.to(dtype), "beta": be.to(dtype)}, S


@pytest.mark.parametrize("t", [1, 4, 8, 16])
@pytest.mark.parametrize("dtype,p", [(torch.bfloat16, 8), (torch.float32, 11)])
@pytest.mark.parametrize("cancel", [False, True])
def test_large_state(kda, t, dtype, p, cancel):
    x, state = draw(2, 2, t, dtype, 500 + t, cancel)
    tree = ref.random_tree(2, t, seed=t + 3)
    o_ref, _ = ref.kda_tree(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], state, tree)
    tol = bound(x, state, tree, o_ref, p, dtype)
    c = {n: a.cuda() for n, a in x.items()}
    args = (c["q"], c["k"], c["v"], c["log_alpha"], c["beta"])
    o = kda.decode_tree(*args, state.cuda(), tree.cuda()).cpu().double()
    err = (o - o_ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    # a chain against the token-by-token step, which keeps fp32: both within their own bounds of the formula
    chain, _ = ref.kda_tree(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], state, None)
    both = bound(x, state, None, chain, p, dtype)
    a = kda.decode_tree(*args, state.cuda()).cpu().double()
    b = kda.decode_tokens(*args, state.cuda()).cpu().double()
    assert bool(((a - chain).abs() <= both).all())
    assert bool(((a - b).abs() <= 2 * both).all())
    assert kda.device_status() == 0
