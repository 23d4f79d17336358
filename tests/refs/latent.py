"""Plain 64-bit forms of the latent-attention operators and of the drafted-tree KDA step.

Written from the definitions, one sequence, one token and one page at a time, on the CPU. They
share no code with the kernels; scores of unseen keys never enter (they are left out, not masked),
so whatever an unused cache row holds cannot reach a result.
"""

from __future__ import annotations

import math

import torch

LATENT, SHARED, D = 512, 64, 128


def half_step(dtype) -> float:
    """The largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def rmsnorm(x, w, eps):
    x = x.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return y if w is None else y * w.double()


def cached_rows(cache, page_table, n, first, last):
    """Rows first .. last-1 of sequence n, [last - first, 576] in 64 bits."""
    ps = cache.shape[1]
    p = torch.arange(first, max(first, last))
    return cache[page_table[n, p // ps].long(), p % ps].double()


def attend(q, keys, values, scale):
    """One query against the keys it sees: (output, log of the sum of exponentials)."""
    if keys.shape[0] == 0:
        return torch.zeros(values.shape[1], dtype=torch.float64), -math.inf
    z = (keys @ q) * scale
    m = z.max()
    e = torch.exp(z - m)
    return (e / e.sum()) @ values, float(m + torch.log(e.sum()))


def mla_decode(q, cache, page_table, cache_lens, tree, scale):
    """q [N, t, H, 576]; token j sees the rows before the t newest and, of those, its bits of
    tree[n, j] (None: 0 .. j)."""
    N, t, H, _ = q.shape
    o = torch.zeros(N, t, H, LATENT, dtype=torch.float64)
    lse = torch.full((N, t, H), -math.inf, dtype=torch.float64)
    for n in range(N):
        L = int(cache_lens[n])
        rows = cached_rows(cache, page_table, n, 0, L)
        for j in range(t):
            bits = (2 << j) - 1 if tree is None else int(tree[n, j])
            seen = [p for p in range(L) if p < L - t or (bits >> (p - (L - t))) & 1]
            r = rows[seen]
            for h in range(H):
                o[n, j, h], lse[n, j, h] = attend(q[n, j, h].double(), r, r[:, :LATENT], scale)
    return o, lse


def mla_prefill(q, k, k_shared, v, cu_q, cu_k, causal, scale):
    """Packed sequences; with causal a sequence's last query sees its last key."""
    o = torch.zeros(q.shape[0], q.shape[1], D, dtype=torch.float64)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    for a, b, c, d in zip(cu_q, cu_q[1:], cu_k, cu_k[1:]):
        if b == a or d == c:
            continue
        ks = k_shared[c:d].double()
        for h in range(q.shape[1]):
            kk = torch.cat([k[c:d, h].double(), ks], 1)
            z = q[a:b, h].double() @ kk.t() * scale
            if causal:
                i, j = torch.arange(b - a)[:, None] + (d - c) - (b - a), torch.arange(d - c)
                z = torch.where(j <= i, z, torch.tensor(-math.inf, dtype=torch.float64))
            m = z.amax(1, keepdim=True)
            e = torch.exp(z - torch.where(torch.isinf(m), torch.zeros_like(m), m))
            s = e.sum(1, keepdim=True)
            o[a:b, h] = (e / torch.where(s == 0, torch.ones_like(s), s)) @ v[c:d, h].double()
            lse[a:b, h] = (m + torch.log(s)).squeeze(1)
    return o, lse


def parents(bits):
    """Parent of every token of one tree (-1: the root state), from its ancestor bits."""
    return [max((i for i in range(j) if (b >> i) & 1), default=-1) for j, b in enumerate(bits)]


def random_tree(n, t, seed):
    """Ancestor bits [n, t] int32 of random trees; token 0 is a root, others may be too."""
    g = torch.Generator().manual_seed(seed)
    out = torch.zeros(n, t, dtype=torch.int32)
    for i in range(n):
        for j in range(t):
            p = int(torch.randint(-1, j, (1,), generator=g)) if j else -1
            out[i, j] = (int(out[i, p]) if p >= 0 else 0) | (1 << j)
    return out


def kda_tree(q, k, v, log_alpha, beta, state, tree):
    """The KDA recurrence from every token's parent's state. q.. [N, t, H, 128], state [N, H, 128, 128];
    tree None: a chain. Returns (outputs, the state after every token [N, t, H, 128, 128])."""
    N, t, H, _ = q.shape
    q, k, v = q.double(), k.double(), v.double()
    al, be, S0 = log_alpha.double().exp(), beta.double(), state.double()
    o = torch.zeros_like(q)
    after = torch.zeros(N, t, H, D, D, dtype=torch.float64)
    for n in range(N):
        par = [j - 1 for j in range(t)] if tree is None else parents(tree[n].tolist())
        for j in range(t):
            S = (S0[n] if par[j] < 0 else after[n, par[j]]) * al[n, j].unsqueeze(-1)
            miss = v[n, j] - torch.einsum("hcv,hc->hv", S, k[n, j])
            S = S + be[n, j][:, None, None] * k[n, j].unsqueeze(-1) * miss.unsqueeze(-2)
            after[n, j] = S
            o[n, j] = torch.einsum("hcv,hc->hv", S, q[n, j])
    return o, after
