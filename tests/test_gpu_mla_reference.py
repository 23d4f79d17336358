"""The running reference of kda_mla_prefill's weights where it moves inside unmasked tiles: the first
half's weights, formed with the old reference, are then formed and stored a second time.

Tolerances, before any run. A score is an fp32 sum of 192 exact products, off by at most 192 *
2^-24 of the terms' absolute sum, and twice that (the weight and the sum it is divided by)
enters a weight, relative, beside 2^-8 from its rounding to bf16: o within (2^-8 + 2 e) sum_j w_j
|v_j| + 2^-8 |o|, and lse within e plus its own fp32 rounding, where e is the bound on the
scores, computed from the inputs.
"""

from __future__ import annotations

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


def inputs(T, Tk, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    return r(T, H, D + SH), r(Tk, H, D), r(Tk, SH), r(Tk, H, D)


def check(kda, q, k, ks, v, causal):
    o, lse = kda.mla_prefill(q, k, ks, v, causal=causal, output_lse=True)
    c = [t.cpu() for t in (q, k, ks, v)]
    cq, ck = [0, q.shape[0]], [0, k.shape[0]]
    o_ref, lse_ref = ref.mla_prefill(*c, cq, ck, causal, SCALE)
    spread, _ = ref.mla_prefill(*c[:3], c[3].abs(), cq, ck, causal, SCALE)
    terms = max(float((c[0][:, h, :D].double().abs() @ c[1][:, h].double().abs().t()
                       + c[0][:, h, D:].double().abs() @ c[2].double().abs().t()).max())
                for h in range(q.shape[1]))
    e = 192 * 2.0 ** -24 * terms * SCALE
    h = ref.half_step(torch.bfloat16)
    err = (o.cpu().double() - o_ref).abs()
    assert bool((err <= (h + 2 * e) * spread + h * o_ref.abs()).all())
    big = float(lse_ref.abs().max())
    assert float((lse.cpu().double() - lse_ref).abs().max()) <= e + 4 * 2.0 ** -24 * max(big, 1.0)
    again, lse2 = kda.mla_prefill(q, k, ks, v, causal=causal, output_lse=True)
    assert torch.equal(again, o) and torch.equal(lse2, lse)


@pytest.mark.parametrize("Tq,Tk", [(256, 1024), (300, 1000), (1, 2048)])
def test_every_tile_moves_it_for_some_rows(kda, Tq, Tk):
    """7 nats (10 powers of two) more in every tile for the rows with a positive first value, 7 less
    for the others, whose reference stays that of the first tile: both in one warp."""
    q, k, ks, v = inputs(Tq, Tk, 2, Tq)
    q[..., 0] = torch.where(torch.arange(Tq, device="cuda") % 3 == 0, 10.0, -10.0)[:, None].bfloat16()
    k[..., 0] = (10.0 * (torch.arange(Tk, device="cuda") // 128))[:, None].bfloat16()
    check(kda, q, k, ks, v, causal=False)


@pytest.mark.parametrize("at", [130, 190, 200, 255, 640])
@pytest.mark.parametrize("causal", [False, True])
def test_one_key_moves_it(kda, at, causal):
    """One key far above the rest, in the first or second half of a later tile: the tile's weights
    with the old reference are up to 2^60 and all formed again."""
    q, k, ks, v = inputs(400, 900, 1, at)
    q[..., 1] = 20.0
    k[..., 1] = 0.0
    k[at, :, 1] = 30.0
    check(kda, q, k, ks, v, causal=causal)
