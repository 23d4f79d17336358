"""kda_mla_append over the whole range of bf16 values and of eps: the squares of a row may leave fp32
at either end, its normalised values do not.

Tolerance, before any run: as the rest of the append's tests, fp32 arithmetic (a sum of 512
squares, one square root, one division, products: 1.6e-5 relative) and one rounding to bf16. The
smallest normalised value of a row here is far above bf16's subnormals.
"""

from __future__ import annotations

import math

import pytest
import torch

from refs import latent as ref

pytestmark = pytest.mark.gpu

W, PAGE, REL = ref.LATENT + ref.SHARED, 16, 1.6e-5


@pytest.fixture(scope="module")
def kda():
    from channel_wise_gated_b200 import build
    build.build()
    import channel_wise_gated_b200 as m
    return m


def append(kda, x, w, eps):
    T = x.shape[0]
    pages = -(-T // PAGE)
    cache = torch.zeros(pages, PAGE, W, device="cuda", dtype=torch.bfloat16)
    table = torch.arange(pages, device="cuda", dtype=torch.int32)[None]
    lat = kda.mla_append(x, w, cache, table, torch.tensor([T], device="cuda", dtype=torch.int32),
                         output_latent=True, eps=eps)
    rows = cache.view(-1, W)[:T]
    assert torch.equal(rows[:, :512], lat) and torch.equal(rows[:, 512:], x[:, 512:])
    assert kda.device_status() == 0
    return lat.cpu().double()


def check(kda, x, w, eps):
    y = append(kda, x, w, eps)
    want = ref.rmsnorm(x[:, :512].cpu(), w.cpu(), float(torch.tensor(eps, dtype=torch.float32)))
    assert bool(((y - want).abs() <= (ref.half_step(torch.bfloat16) + REL) * want.abs()).all())


# powers of two from bf16's smallest normal values to its largest, where the normalised values
# themselves stay in its normal range
POWERS = [-120, -100, -75, -64, -63, -62, -56, -50, -20, 0, 40, 58, 62, 64, 100, 125]
SIZES = [(p, e) for p in POWERS for e in (0.0, 1e-45, 1e-38, 1e-30, 1e-20, 1e-6, 1.0)
         if not e or 2.0 ** p / math.sqrt(e) >= 2.0 ** -100]


@pytest.mark.parametrize("power,eps", SIZES)
def test_every_size_of_row(kda, power, eps):
    g = torch.Generator(device="cuda").manual_seed(power + 200)
    x = torch.randn((33, W), generator=g, device="cuda")
    x = (x.sign() * x.abs().clamp(0.25, 3.0)).double().mul(2.0 ** power).to(torch.bfloat16)
    w = 0.5 + torch.rand(ref.LATENT, generator=g, device="cuda")
    check(kda, x, w, eps)


def test_rows_of_all_sizes_in_one_call(kda):
    """Rows whose squares underflow, overflow and do neither, next to each other, eps 0."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((64, W), generator=g, device="cuda")
    x = x.sign() * x.abs().clamp(0.25, 3.0)
    p = torch.linspace(-120, 125, 64, device="cuda").round()
    x = (x.double() * torch.exp2(p.double())[:, None]).to(torch.bfloat16)
    check(kda, x, 0.5 + torch.rand(ref.LATENT, generator=g, device="cuda"), 0.0)


def test_subnormal_rows(kda):
    """A row of bf16's smallest value alone, and one such value among zeros: 1 and sqrt(512)."""
    x = torch.zeros(2, W, device="cuda")
    x[0, :512] = 2.0 ** -133
    x[1, 7] = 2.0 ** -133
    x = x.to(torch.bfloat16)
    assert float(x[0, 0]) == 2.0 ** -133
    y = append(kda, x, torch.ones(512, device="cuda"), 0.0)
    assert bool((y[0] == 1).all())
    assert float((y[1, 7] - math.sqrt(512)).abs()) <= (ref.half_step(torch.bfloat16) + REL) * math.sqrt(512)
    assert int((y[1] != 0).sum()) == 1


def test_a_row_of_zeros(kda):
    """0 with any eps above 0; with eps = 0 the quotient 0 / 0 that the definition asks for."""
    x = torch.zeros(1, W, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(512, device="cuda")
    for eps in (1e-6, 1e-38, 1e-45):
        assert bool((append(kda, x, w, eps) == 0).all())
    cache = torch.zeros(1, PAGE, W, device="cuda", dtype=torch.bfloat16)
    lat = kda.mla_append(x, w, cache, torch.zeros(1, 1, device="cuda", dtype=torch.int32),
                         torch.ones(1, device="cuda", dtype=torch.int32), output_latent=True, eps=0.0)
    assert bool(torch.isnan(lat).all())
