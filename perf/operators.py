"""Operators of the hybrid model's latent-attention layers and of drafted trees, case by case.

Three KDA layers alternate with one layer of latent attention (MLA, no positional encoding): a
token's keys and values come from one vector of 512 values that all heads share, cached beside 64
key values that are shared as they are (576 per token and layer). The operators:

* ``mla_append``: RMSNorm of the down-projection's 512 latent values, and the write of the 576 values
  into a paged cache;
* ``mla_prefill``: the expanded form. Causal softmax attention of packed sequences, 128 key
  values per head and the 64 shared ones, 128 value channels per head;
* ``mla_decode``: the absorbed form over the paged cache. 1 to 16 new tokens per sequence, a
  chain or a tree of drafted tokens, queries already multiplied into the latent space;
* ``decode_tree``: the KDA recurrence's outputs for such a tree, the state read and left as it is.

``run`` computes them in plain torch operations, or calls ``channel_wise_gated_b200`` where ``own`` is true.
"""

from __future__ import annotations

import math

import torch

own = False

LATENT, SHARED, D = 512, 64, 128
WIDTH = LATENT + SHARED          # values cached per token
EPS = 1e-6
SCALE = 1.0 / math.sqrt(D + SHARED)


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of one sequence, the smallest call between two projections: latency
        dict(name="append_1", op="append", n=1, lo=3001, hi=3001, t=1, page=64, plan=1),
        # a packed prefill batch of 16 ragged prompts, normalised latents returned for the up-projection
        dict(name="append_varlen16", op="append", n=16, lo=512, hi=8192, t=0, page=64, plan=2),
        # a short chat turn: three prompts, the shortest of one token
        dict(name="prefill_short", op="prefill", heads=32, n=3, lo=1, hi=211, prefix=0, causal=True, plan=5),
        # one prompt of 4096 tokens and 32 heads, the length of the KDA prefill workload
        dict(name="prefill_4k", op="prefill", heads=32, n=1, lo=4096, hi=4096, prefix=0, causal=True, plan=1),
        # a packed batch of ragged prompts, odd lengths
        dict(name="prefill_varlen8", op="prefill", heads=32, n=8, lo=129, hi=2047, prefix=0, causal=True, plan=2),
        # one long prompt, the heads of one of eight ranks
        dict(name="prefill_long", op="prefill", heads=4, n=1, lo=32768, hi=32768, prefix=0, causal=True, plan=1),
        # a prompt's next 1024 tokens after 7001 that were computed before
        dict(name="prefill_chunk", op="prefill", heads=32, n=1, lo=1024, hi=1024, prefix=7001, causal=True, plan=1),
        # one user, one token: latency over a cache of some thousand tokens
        dict(name="decode_1", op="decode", heads=32, n=1, lo=5003, hi=5003, t=1, tree=False, page=64, plan=1),
        # a serving batch of ragged lengths, one token per sequence
        dict(name="decode_128", op="decode", heads=32, n=128, lo=1024, hi=8192, t=1, tree=False, page=64, plan=2),
        # trees of 8 drafted tokens for 48 sequences, verified in one call
        dict(name="decode_tree8", op="decode", heads=32, n=48, lo=1000, hi=8000, t=8, tree=True, page=16, plan=3),
        # the same step's KDA layers: one sequence, 6 drafted tokens
        dict(name="kda_tree_1", op="tree", heads=32, n=1, t=6, f32=False, plan=1),
        # and the decode workload's batch (256 sequences, 32 heads) with 8 drafted tokens each
        dict(name="kda_tree_256", op="tree", heads=32, n=256, t=8, f32=False, plan=2),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "prefill", "prefill", "decode", "decode", "tree"))
    plan = rng.randrange(1 << 20)
    if op == "append":
        t = rng.choice((0, 0, 1, 2, 4, 7, 16))
        n = _logint(rng, 1, 256) if t else _logint(rng, 1, 16)
        lo = max(1, t) if rng.random() < 0.3 else _logint(rng, max(1, t), 4096)
        return dict(op=op, n=n, lo=lo, hi=max(lo, _logint(rng, 16, 8192)), t=t,
                    page=rng.choice((16, 32, 64, 128)), plan=plan)
    if op == "prefill":
        heads = rng.choice((1, 2, 3, 4, 8, 16, 32))
        room = int(math.sqrt((1 << 32) / heads))       # tokens of a full score matrix within the largest case
        n = _logint(rng, 1, 12)
        hi = _logint(rng, 2, max(2, min(room, 16384) // n))
        lo = hi if n == 1 else rng.randint(1, hi)
        prefix = rng.choice((0, 0, 0, _logint(rng, 1, 4096)))
        if heads * (n * hi) * (n * (hi + prefix)) > 1 << 32:
            prefix = 0
        return dict(op=op, heads=heads, n=n, lo=lo, hi=hi, prefix=prefix,
                    causal=rng.random() < 0.85, plan=plan)
    if op == "decode":
        heads, t = rng.choice((1, 4, 8, 16, 20, 32, 64, 128)), rng.choice((1, 1, 1, 2, 3, 4, 8, 16))
        n = _logint(rng, 1, 128)
        hi = _logint(rng, 16, min(32768, (1 << 20) // n))
        while n * t * heads * hi > 1 << 27 and n > 1:
            n = (n + 1) // 2
        while n * t * heads * hi > 1 << 27 and t > 1:
            t //= 2
        lo = min(hi, t) if rng.random() < 0.3 else rng.randint(min(hi, t), hi)
        return dict(op=op, heads=heads, n=n, lo=lo, hi=hi, t=t, tree=t > 1 and rng.random() < 0.5,
                    page=rng.choice((16, 32, 64, 128)), plan=plan)
    heads = rng.choice((1, 3, 8, 16, 32))
    return dict(op=op, heads=heads, n=_logint(rng, 1, 256), t=rng.choice((1, 2, 3, 4, 5, 8)),
                f32=rng.random() < 0.3, plan=plan)


def _lengths(case):
    """The case's ragged lengths, the same for every seed of the data."""
    g = torch.Generator().manual_seed(case["plan"])
    lens = torch.randint(case["lo"], case["hi"] + 1, (case["n"],), generator=g).tolist()
    if case["n"] > 1:
        lens[0] = case["lo"]
        lens[-1] = case["hi"]
    return lens


def _starts(lens):
    out = [0]
    for x in lens:
        out.append(out[-1] + x)
    return out


# ---------------------------------------------------------------------------- inputs
def _normal(shape, g, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _tables(lens, page, g, spare=3):
    """A page table over a shuffled pool of pages: int32 [N, most], and the pool's size."""
    need = [-(-x // page) for x in lens]
    most, total = max(max(need), 1), sum(need) + spare
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((len(lens), most), dtype=torch.int32, device="cuda")
    at = 0
    for n, k in enumerate(need):
        table[n, :k] = order[at:at + k]
        at += k
    return table, total


def _tree(n, t, g):
    """Ancestor bits of n random trees of t tokens: bit i of [n, j] is set where token i is token j or
    one of its ancestors. Parents come before their children."""
    bits = torch.zeros((n, t), dtype=torch.int64, device="cuda")
    rows = torch.arange(n, device="cuda")
    for j in range(t):
        parent = torch.randint(-1 if j else 0, max(j, 1), (n,), generator=g, device="cuda")
        up = bits[rows, parent.clamp(min=0)] * (parent >= 0) if j else torch.zeros_like(rows)
        bits[:, j] = up | (1 << j)
    return bits.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"op": case["op"]}
    if case["op"] == "append":
        lens = _lengths(case)
        new = [case["t"]] * len(lens) if case["t"] else lens
        table, pool = _tables(lens, case["page"], g)
        starts = _starts(new)
        s.update(x=_normal((starts[-1], WIDTH), g), norm_w=0.5 + torch.rand(LATENT, generator=g, device="cuda"),
                 cache=_normal((pool, case["page"], WIDTH), g), page_table=table,
                 cache_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 cu_seqlens=torch.tensor(starts, dtype=torch.int32, device="cuda"),
                 latent=case["t"] == 0, page=case["page"])
    elif case["op"] == "prefill":
        lens, H = _lengths(case), case["heads"]
        lens_k = [x + case["prefix"] for x in lens]
        cq, ck = _starts(lens), _starts(lens_k)
        # k and v are the two halves of the up-projection's output, as a program has them
        kv = _normal((ck[-1], H, 2 * D), g)
        s.update(q=_normal((cq[-1], H, D + SHARED), g), k=kv[..., :D], v=kv[..., D:],
                 k_shared=_normal((ck[-1], SHARED), g), causal=case["causal"],
                 cu_seqlens=torch.tensor(cq, dtype=torch.int32, device="cuda"),
                 cu_seqlens_k=torch.tensor(ck, dtype=torch.int32, device="cuda") if case["prefix"] else None)
    elif case["op"] == "decode":
        lens = _lengths(case)
        table, pool = _tables(lens, case["page"], g)
        # a query in the latent space: its product with a normalised latent has the spread of a
        # product of two 192-value heads
        q = _normal((case["n"], case["t"], case["heads"], WIDTH), g, scale=math.sqrt((D + SHARED) / WIDTH))
        s.update(q=q, cache=_normal((pool, case["page"], WIDTH), g), page_table=table,
                 cache_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 tree=_tree(case["n"], case["t"], g) if case["tree"] else None)
    else:
        N, t, H = case["n"], case["t"], case["heads"]
        dt = torch.float32 if case["f32"] else torch.bfloat16
        q, k = (torch.nn.functional.normalize(_normal((N, t, H, D), g, torch.float32), dim=-1).to(dt) for _ in "qk")
        s.update(q=q, k=k, v=_normal((N, t, H, D), g, dt),
                 log_alpha=-torch.log1p(torch.exp(-(_normal((N, t, H, D), g, torch.float32) + 3.0))).to(dt),
                 beta=torch.sigmoid(_normal((N, t, H), g, torch.float32)).to(dt),
                 state=_normal((N, H, D, D), g, torch.float32, 0.02), tree=_tree(N, t, g))
    return s


# ---------------------------------------------------------------------------- one pass
def run(s):
    op = s["op"]
    if own:
        import channel_wise_gated_b200 as kda
        if op == "append":
            latent = kda.mla_append(s["x"], s["norm_w"], s["cache"], s["page_table"], s["cache_lens"],
                                    cu_seqlens=s["cu_seqlens"], output_latent=s["latent"], eps=EPS)
            return {"cache": s["cache"], "latent": latent}
        if op == "prefill":
            o, lse = kda.mla_prefill(s["q"], s["k"], s["k_shared"], s["v"], cu_seqlens=s["cu_seqlens"],
                                     cu_seqlens_k=s["cu_seqlens_k"], causal=s["causal"], output_lse=True)
            return {"o": o, "lse": lse}
        if op == "decode":
            o, lse = kda.mla_decode(s["q"], s["cache"], s["page_table"], s["cache_lens"], tree=s["tree"],
                                    scale=SCALE, output_lse=True)
            return {"o": o, "lse": lse}
        return {"o": kda.decode_tree(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], s["state"], tree=s["tree"])}
    return {"append": _append, "prefill": _prefill, "decode": _decode, "tree": _kda_tree}[op](s)


def _append(s):
    """y = x / sqrt(mean(x^2) + eps) * w over the 512 latent values; the row goes to the page that holds its position."""
    x, cu = s["x"].float(), s["cu_seqlens"].long()
    c = x[:, :LATENT]
    y = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * s["norm_w"]
    row = torch.cat([y, x[:, LATENT:]], -1).to(torch.bfloat16)
    token = torch.arange(x.shape[0], device=x.device)
    n = torch.bucketize(token, cu[1:], right=True)
    pos = s["cache_lens"].long()[n] - cu[n + 1] + token
    slot = s["page_table"].long()[n, pos // s["page"]] * s["page"] + pos % s["page"]
    s["cache"].view(-1, WIDTH)[slot] = row
    return {"cache": s["cache"], "latent": row[:, :LATENT].contiguous() if s["latent"] else None}


def _softmax(z):
    """Weights and the logarithm of their sum along the last axis; a row of -inf alone gets zeros and -inf."""
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(z - m)
    l = p.sum(-1, keepdim=True)
    return p / torch.where(l == 0, torch.ones_like(l), l), (torch.log(l) + m).squeeze(-1)


def _prefill(s):
    """softmax of the packed batch's whole score matrix, masked to each row's own sequence and to keys not after it."""
    q, v = s["q"].float(), s["v"].float()
    cq = s["cu_seqlens"].long()
    ck = cq if s["cu_seqlens_k"] is None else s["cu_seqlens_k"].long()
    i, j = torch.arange(q.shape[0], device=q.device), torch.arange(v.shape[0], device=q.device)
    ni, nj = torch.bucketize(i, cq[1:], right=True), torch.bucketize(j, ck[1:], right=True)
    sees = ni[:, None] == nj
    if s["causal"]:      # a sequence's last query sees its last key
        sees = sees & ((ck[1:] - cq[1:])[ni][:, None] + i[:, None] >= j)
    z = torch.einsum("ihd,jhd->hij", q[..., :D], s["k"].float())
    z += torch.einsum("ihd,jd->hij", q[..., D:], s["k_shared"].float())
    p, lse = _softmax(z.mul_(SCALE).masked_fill_(~sees, -math.inf))
    return {"o": torch.einsum("hij,jhd->ihd", p, v).to(torch.bfloat16), "lse": lse.t().contiguous()}


def _decode(s):
    """The cache gathered page by page; token j of t sees the cached prefix and, of the t newest rows, those of its
    ancestor bits (a chain: those not after it)."""
    q, lens = s["q"].float(), s["cache_lens"].long()
    N, t, H, _ = q.shape
    c = s["cache"][s["page_table"].long()].flatten(1, 2).float()
    pos = torch.arange(c.shape[1], device=q.device)
    draft = pos - (lens[:, None, None] - t)                    # [N, 1, L]: the row's number among the t newest
    token = torch.arange(t, device=q.device)[:, None]
    if s["tree"] is None:
        sees = draft <= token
    else:
        sees = (draft < 0) | ((s["tree"].long()[:, :, None] >> draft.clamp(0, t - 1)) & 1 == 1)
    sees = sees & (pos < lens[:, None, None])
    z = torch.einsum("nthd,nld->nthl", q, c).mul_(SCALE)
    p, lse = _softmax(z.masked_fill_(~sees[:, :, None], -math.inf))
    return {"o": torch.einsum("nthl,nld->nthd", p, c[..., :LATENT]).to(torch.bfloat16), "lse": lse}


def _kda_tree(s):
    """The chunk form over each token's path: with G the sum of log alpha along it,
    (I + A) delta = beta (v - (k e^G) S),  A_ri = beta_r sum_c k_r k_i e^(G_r - G_i) over r's proper ancestors i,
    o_r = (q_r e^(G_r)) S + sum_i P_ri delta_i,  P_ri = sum_c q_r k_i e^(G_r - G_i) over r and its ancestors."""
    q, k, v, la, S = (s[n].float().transpose(1, 2) if n != "state" else s[n] for n in ("q", "k", "v", "log_alpha", "state"))
    beta = s["beta"].float().transpose(1, 2)[..., None]                       # [N, H, t, 1]
    t = q.shape[2]
    at = torch.arange(t, device=q.device)
    on = (((s["tree"].long()[..., None] >> at) & 1) == 1)[:, None]            # [N, 1, t, t]
    G = on.float() @ la
    E = torch.exp(torch.where(on[..., None], G[:, :, :, None] - G[:, :, None], -math.inf))
    A = beta * torch.einsum("nhrd,nhid,nhrid->nhri", k, k, E) * (at[:, None] != at)
    P = torch.einsum("nhrd,nhid,nhrid->nhri", q, k, E)
    rhs = beta * (v - (k * G.exp()) @ S)
    eye = torch.eye(t, device=q.device)
    A2 = A @ A                     # A is strictly lower: (I + A)^-1 = (I - A)(I + A^2)(I + A^4)(I + A^8) up to t = 16
    A4 = A2 @ A2
    inv = (eye - A) @ (eye + A2) @ (eye + A4) @ (eye + A4 @ A4)
    o = (q * G.exp()) @ S + P @ (inv @ rhs)
    return {"o": o.transpose(1, 2).to(s["q"].dtype).contiguous()}


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "append":
        rows = case["n"] * case["t"] if case["t"] else sum(_lengths(case))
        return {"bytes": rows * (2 * 2 * WIDTH + (0 if case["t"] else 2 * LATENT)) + 4 * LATENT, "flops": 4 * rows * LATENT}
    if case["op"] == "prefill":
        lens, H = _lengths(case), case["heads"]
        T, Tk = sum(lens), sum(lens) + case["prefix"] * len(lens)
        pairs = sum(x * case["prefix"] + (x * (x + 1) // 2 if case["causal"] else x * x) for x in lens)
        return {"bytes": T * H * (2 * (D + SHARED) + 2 * D + 4) + Tk * (H * 4 * D + 2 * SHARED),
                "flops": 2 * H * pairs * (D + SHARED + D)}
    if case["op"] == "decode":
        rows, keys = case["t"] * case["heads"], sum(_lengths(case))
        return {"bytes": 2 * WIDTH * keys + case["n"] * rows * (2 * WIDTH + 2 * LATENT + 4),
                "flops": 2 * rows * keys * (WIDTH + LATENT)}
    e, chains, t = 4 if case["f32"] else 2, case["n"] * case["heads"], case["t"]
    return {"bytes": chains * (4 * D * D + t * e * (5 * D + 1)), "flops": chains * t * 4 * D * D}


# ---------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        x = s["x"].double()
        w = s["norm_w"].double()
        cache = s["cache"].double()
        scaled = x[:, :LATENT] / (x[:, :LATENT].pow(2).sum(1, keepdim=True) / LATENT + EPS).sqrt()
        rows = torch.cat([scaled * w[None], x[:, LATENT:]], 1)
        lens, starts, table = _lengths(case), s["cu_seqlens"].tolist(), s["page_table"].long()
        for n in range(case["n"]):
            new = rows[starts[n]:starts[n + 1]]
            at = torch.arange(lens[n] - len(new), lens[n], device=x.device)
            cache[table[n, at // case["page"]], at % case["page"]] = new
        return {"cache": cache, "latent": rows[:, :LATENT].clone() if s["latent"] else None}
    if case["op"] == "prefill":
        q, v = s["q"].double(), s["v"].double()
        k = torch.cat([s["k"].double(), s["k_shared"].double()[:, None].expand(-1, case["heads"], -1)], 2)
        cq = s["cu_seqlens"].tolist()
        ck = cq if s["cu_seqlens_k"] is None else s["cu_seqlens_k"].tolist()
        o = torch.zeros(q.shape[:2] + (D,), dtype=torch.float64, device=q.device)
        lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
        for a, b, c, d in zip(cq, cq[1:], ck, ck[1:]):
            for i0 in range(a, b, 1024):
                i1 = min(b, i0 + 1024)
                last = d - b + i1 if case["causal"] else d     # keys behind the block's last row are seen by none of it
                z = q[i0:i1].transpose(0, 1) @ k[c:last].permute(1, 2, 0) / math.sqrt(D + SHARED)
                if case["causal"]:
                    r = torch.arange(i0, i1, device=q.device)[:, None] + (d - b)
                    z.masked_fill_(torch.arange(c, last, device=q.device) > r, -math.inf)
                o[i0:i1] = (torch.softmax(z, -1) @ v[c:last].transpose(0, 1)).transpose(0, 1)
                lse[i0:i1] = torch.logsumexp(z, -1).t()
        return {"o": o, "lse": lse}
    if case["op"] == "decode":
        N, t, H, _ = s["q"].shape
        o = torch.zeros((N, t, H, LATENT), dtype=torch.float64, device="cuda")
        lse = torch.zeros((N, t, H), dtype=torch.float64, device="cuda")
        for n, L in enumerate(_lengths(case)):
            c = s["cache"][s["page_table"][n].long()].reshape(-1, WIDTH)[:L].double()
            z = s["q"][n].double() @ c.t() / math.sqrt(D + SHARED)        # [t, H, L]
            for j in range(t):
                for i in range(t):
                    seen = i <= j if s["tree"] is None else (int(s["tree"][n, j]) >> i) & 1
                    if not seen and L - t + i >= 0:
                        z[j, :, L - t + i] = -math.inf
            o[n] = torch.softmax(z, -1) @ c[:, :LATENT]
            lse[n] = torch.logsumexp(z, -1)
        return {"o": o, "lse": lse}
    # the recurrence itself, from each token's parent's state
    q, k, v = (s[n].double() for n in "qkv")
    alpha, beta = s["log_alpha"].double().exp(), s["beta"].double()
    N, t, H, _ = q.shape
    o = torch.zeros_like(q)
    for b in range(0, N, 32):
        e = slice(b, min(N, b + 32))
        bits, states = s["tree"][e].tolist(), []
        for j in range(t):
            above = [max((i for i in range(j) if row[j] >> i & 1), default=-1) for row in bits]
            S = torch.stack([s["state"][b + n].double() if p < 0 else states[p][n] for n, p in enumerate(above)])
            S = S * alpha[e, j].unsqueeze(-1)
            miss = v[e, j] - torch.einsum("nhcv,nhc->nhv", S, k[e, j])
            S = S + beta[e, j][..., None, None] * k[e, j].unsqueeze(-1) * miss.unsqueeze(-2)
            states.append(S)
            o[e, j] = torch.einsum("nhcv,nhc->nhv", S, q[e, j])
    return {"o": o}
