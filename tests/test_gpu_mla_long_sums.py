"""Sums of values over very many keys. Equal scores (q = 0) make every weight 1, exactly, and the
output the mean of the values: what is left is how the accumulators add.

Tolerance, before any run: an accumulator that adds n products of 16 keys in a row, each sum off by
at most 2^-23 of itself (matrix units may cut instead of rounding), is off by n * 2^-23 of the sum of
|v|; n is held at 4,096 and the parts, at most 64 here, are added in fp32: 4,160 * 2^-23 = 5e-4 in
all, and the output is rounded once, 2^-8 of it. 65,536 such sums in a row lose 0.4 to 0.8 %.
"""

from __future__ import annotations

import math

import pytest
import torch

from refs import latent as ref

pytestmark = pytest.mark.gpu

D, SH = ref.D, ref.SHARED
SUM = 4160 * 2.0 ** -23


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


def values(Tk, H, seed):
    """[1, 2) in every third channel, its negative in the next, both signs in the last."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = 1.0 + torch.rand((Tk, H, D), generator=g, device="cuda")
    v[..., 1::3] *= -1
    v[..., 2::3] -= 1.5
    return v.bfloat16()


@pytest.mark.parametrize("Tk", [65536, 65537, 65536 + 100, 131072, 131073, 1048571])
@pytest.mark.parametrize("Tq,causal", [(3, True), (200, False)])
def test_prefill_mean_of_values(kda, Tk, Tq, causal):
    g = torch.Generator(device="cuda").manual_seed(Tk)
    k = torch.randn((Tk, 1, D), generator=g, device="cuda").bfloat16()
    ks = torch.randn((Tk, SH), generator=g, device="cuda").bfloat16()
    v = values(Tk, 1, Tk + 1)
    q = torch.zeros((Tq, 1, D + SH), device="cuda", dtype=torch.bfloat16)
    o, lse = kda.mla_prefill(q, k, ks, v, causal=causal, output_lse=True)
    for i in (0, 1, Tq - 1):
        n = Tk - Tq + 1 + i if causal else Tk
        mean, spread = v[:n, 0].double().mean(0), v[:n, 0].double().abs().mean(0)
        err = (o[i, 0].double() - mean).abs()
        tol = SUM * spread + ref.half_step(torch.bfloat16) * mean.abs()
        assert bool((err <= tol).all()), (i, float((err / spread).max()))
        assert abs(float(lse[i, 0]) - math.log(n)) <= 2.0 ** -22 * math.log(n)


@pytest.mark.parametrize("Tk", [65536 + 1, 70000, 196608 + 128])
@pytest.mark.parametrize("slope", [4.0, -4.0, 0.25])
def test_prefill_scores_move_over_the_parts(kda, Tk, slope):
    """Scores that rise (or fall) by 70 nats over the keys, and by 4: the parts taken out before belong
    to an older reference. Tolerance as for any long prefill, with the sums of one part."""
    from test_gpu_mla_lengths import check_row, heads
    q, k, ks, v = heads(150, Tk, 1, Tk)
    q[..., 0] = slope
    k[..., 0] = (torch.arange(Tk, device="cuda") * 250 // Tk)[:, None].bfloat16()
    o, lse = kda.mla_prefill(q, k, ks, v, output_lse=True)
    for i in (0, 70, 127, 128, 149):
        n = Tk - 149 + i
        check_row(o[i, 0], lse[i, 0], q[i, 0], torch.cat([k[:n, 0], ks[:n]], 1), v[:n, 0], 34 * 512 + 64)


def test_prefill_packed_over_the_parts(kda):
    """Long and short sequences in one batch, rows that see nothing, keys that no row sees."""
    from test_gpu_mla_lengths import check_row, heads, i32
    lq, lk = [200, 1, 130, 40, 3], [65536 + 70, 9, 100, 0, 131072 + 3]
    cq, ck = [0], [0]
    for a, b in zip(lq, lk):
        cq.append(cq[-1] + a)
        ck.append(ck[-1] + b)
    q, k, ks, v = heads(cq[-1], ck[-1], 2, 3)
    o, lse = kda.mla_prefill(q, k, ks, v, cu_seqlens=i32(cq), cu_seqlens_k=i32(ck), output_lse=True)
    for s in range(5):
        for i in {0, lq[s] // 2, lq[s] - 1}:
            n = lk[s] - lq[s] + 1 + i
            for h in range(2):
                r = cq[s] + i
                if n <= 0:
                    assert bool((o[r, h] == 0).all()) and float(lse[r, h]) == -math.inf
                    continue
                e = ck[s] + n
                check_row(o[r, h], lse[r, h], q[r, h], torch.cat([k[ck[s]:e, h], ks[ck[s]:e]], 1), v[ck[s]:e, h],
                          34 * 512 + 64)
    again, l2 = kda.mla_prefill(q, k, ks, v, cu_seqlens=i32(cq), cu_seqlens_k=i32(ck), output_lse=True)
    assert torch.equal(o, again) and torch.equal(lse, l2)
