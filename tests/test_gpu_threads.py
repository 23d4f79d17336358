"""Entry points called from host threads.

* A thread that has made no CUDA call before: the first thing it does may be a call of this library, on
  tensors that another thread made.
* Threads that call one entry point at the same time, each with its own number of tokens and on its own
  stream: their launches share the kernel's attributes, and none may fail or take another's results.
"""

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


def run_at_once(fn, args, n):
    """Four threads call the library's function fn n times each, every thread with its own arguments;
    the statuses that were not 0."""
    bad, go = [], threading.Barrier(len(args))

    def work(a):
        go.wait()
        for _ in range(n):
            st = fn(*a)
            if st:
                bad.append(st)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(a,)) for a in args]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    return bad


@pytest.mark.parametrize("tokens", [(1, 8, 2, 7), (9, 16, 10, 15)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_trees_of_several_sizes_at_once(kda, tokens, dtype):
    """(The entry point itself, so that most of a call's time is spent in the library: with shared
    memory limits set per call, 1,700 to 3,900 of 4 x 10,000 launches were refused.)"""
    from channel_wise_gated_b200 import _native
    lib, args, outs, want, keep = _native.load(), [], [], [], []
    kind = _native.KDA_BF16 if dtype == torch.bfloat16 else _native.KDA_F32
    for t in tokens:
        d = kda_inputs.make_decode(1, 2, t, dtype, dtype, seed=400 + t, device="cuda")
        x = [d[n].transpose(0, 1).contiguous() for n in ("q", "k", "v", "log_alpha", "beta")]
        want.append(kda.decode_tree(*x, d["state"]))
        outs.append(torch.zeros_like(want[-1]))
        stream = torch.cuda.Stream()
        keep.append((x, d, stream))
        args.append([y.data_ptr() for y in x] + [d["state"].data_ptr(), None, outs[-1].data_ptr(), 1, t, 2,
                                                 kind, kind, stream.cuda_stream])
    assert run_at_once(lib.kda_decode_tree, args, 10000) == []
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert kda.device_status() == 0


@pytest.mark.parametrize("tokens", [(1, 2, 1, 2), (3, 8, 4, 7), (12, 16, 13, 15)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_token_runs_of_several_sizes_at_once(kda, tokens, dtype):
    from channel_wise_gated_b200 import _native
    lib, args, outs, want, keep = _native.load(), [], [], [], []
    kind = _native.KDA_BF16 if dtype == torch.bfloat16 else _native.KDA_F32
    for t in tokens:
        d = kda_inputs.make_decode(1, 2, t, dtype, dtype, seed=420 + t, device="cuda")
        x = [d[n].transpose(0, 1).contiguous() for n in ("q", "k", "v", "log_alpha", "beta")]
        x[3].zero_()
        x[4].zero_()     # no decay, beta 0: the state stays as it is over the calls
        want.append(kda.decode_tokens(*x, d["state"].clone()))
        outs.append(torch.zeros_like(want[-1]))
        stream = torch.cuda.Stream()
        keep.append((x, d, stream))
        args.append([y.data_ptr() for y in x] + [d["state"].data_ptr(), outs[-1].data_ptr(), 1, t, 2, kind, kind,
                                                 stream.cuda_stream])
    assert run_at_once(lib.kda_decode_tokens, args, 10000) == []
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert kda.device_status() == 0


def test_all_kinds_on_streams_of_their_own(kda):
    """Every kind of call, each over and over from a thread and a stream of its own: the kernels share the
    SMs' tensor and shared memory, and none its results."""
    torch.manual_seed(1)
    named = calls(kda)
    want = {}
    for name, (call, out) in named.items():
        call()
        want[name] = out.clone()
        out.zero_()
    torch.cuda.synchronize()
    errors, go = [], threading.Barrier(len(named))

    def work(call):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                go.wait()
                for _ in range(500):
                    call()
        except Exception as e:   # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(call,)) for call, _ in named.values()]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert errors == []
    for name, (_, out) in named.items():
        assert torch.equal(out, want[name]), name
    assert kda.device_status() == 0
