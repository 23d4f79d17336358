"""Entry points called from host threads that have made no CUDA call before: the first thing such a
thread does may be a call of this library, on tensors that another thread made."""

from __future__ import annotations

import threading

import pytest
import torch

import kda_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kda():
    from channel_wise_gated_b200 import build
    build.build()
    import channel_wise_gated_b200 as m
    return m


def in_new_thread(call):
    """call() in a thread of its own; what it raised."""
    errors = []

    def work():
        try:
            call()
        except Exception as e:   # noqa: BLE001
            errors.append(e)

    torch.cuda.synchronize()
    th = threading.Thread(target=work)
    th.start()
    th.join()
    torch.cuda.synchronize()
    return errors


def calls(kda):
    """Every entry point, with its outputs given (an allocation could be the thread's first CUDA call):
    name -> (call, output)."""
    bf, i32 = torch.bfloat16, torch.int32
    r = lambda *s: torch.randn(s, device="cuda").to(bf)
    d = kda_inputs.make_decode(2, 2, 4, bf, bf, seed=1, device="cuda")
    x = [d[n].transpose(0, 1).contiguous() for n in ("q", "k", "v", "log_alpha", "beta")]
    p = kda_inputs.make_prefill([200, 77], 4, bf, torch.float32, 3.0, True, seed=5, device="cuda")
    c = [p[n] for n in ("q", "k", "v", "log_alpha", "beta")]
    cache, table = r(8, 16, 576), torch.arange(8, device="cuda", dtype=i32).view(2, 4)
    lens = torch.tensor([60, 33], dtype=i32, device="cuda")
    rows, q = r(2, 576), r(2, 1, 4, 576)
    ws = torch.empty(kda.mla_decode_workspace_size(1, 4), dtype=torch.uint8, device="cuda")
    pq, pk, ps, pv = r(50, 2, 192), r(50, 2, 128), r(50, 64), r(50, 2, 128)
    lat, dec, pre, tree = r(2, 512), r(2, 1, 4, 512), r(50, 2, 128), torch.zeros_like(x[0])
    out, final = torch.zeros_like(c[0]), torch.zeros_like(p["h0"])
    return {
        "append": (lambda: kda.mla_append(rows, None, cache, table, lens, latent=lat), lat),
        "prefill": (lambda: kda.mla_prefill(pq, pk, ps, pv, o=pre), pre),
        "decode": (lambda: kda.mla_decode(q, cache, table, lens, o=dec, workspace=ws), dec),
        "tree": (lambda: kda.decode_tree(*x, d["state"], o=tree), tree),
        "chunk": (lambda: kda.chunk_fwd(*c, h0=p["h0"], cu_seqlens=p["cu_seqlens"], o=out, hT=final), out),
    }


@pytest.mark.parametrize("name", ["append", "prefill", "decode", "tree", "chunk"])
def test_first_call_of_a_thread(kda, name):
    torch.manual_seed(0)
    call, out = calls(kda)[name]
    call()
    want = out.clone()
    out.zero_()
    assert in_new_thread(call) == []
    assert torch.equal(out, want)
    assert kda.device_status() == 0
