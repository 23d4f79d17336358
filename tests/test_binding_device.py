"""The binding calls the library with the tensors' device current and that device's stream, whichever
device is current (no GPU needed: the library and the device state are stand-ins). The library takes
its kernels, its error word and the default stream from the current device."""

from __future__ import annotations

import contextlib

import pytest
import torch

import channel_wise_gated_b200 as kda
from channel_wise_gated_b200 import _native


class Gpu:
    """Two devices, 0 current; a stream's handle is 1000 times its device's number and 7."""

    def __init__(self):
        self.current, self.calls = 0, []

    def __getattr__(self, name):          # any entry point of the library
        if name.endswith("workspace_size"):
            return lambda *a: 0

        def call(*a):
            self.calls.append((name, self.current, a[-1]))
            return 0
        return call

    @contextlib.contextmanager
    def device(self, d):
        before, self.current = self.current, torch.device(d).index if not isinstance(d, int) else d
        try:
            yield
        finally:
            self.current = before


@pytest.fixture
def gpu(monkeypatch):
    g = Gpu()
    monkeypatch.setattr(_native, "load", lambda *a: g)
    monkeypatch.setattr(torch.cuda, "device", g.device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: g.current)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 1000 * i + 7, raising=False)

    class Stream:
        def __init__(self, d):
            d = torch.device(d)
            self.cuda_stream = 1000 * (g.current if d.index is None else d.index) + 7
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: Stream("cuda" if d is None else d))
    return g


class OnDevice1(torch.Tensor):
    """A CPU tensor that says it is on cuda:1."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 1))


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice1)


@pytest.mark.parametrize("device,where", [(None, 0), ("cuda", 0), ("cuda:0", 0), ("cuda:1", 1),
                                          (torch.device("cuda", 1), 1)])
def test_device_status_reads_that_devices_word(gpu, device, where):
    assert kda.device_status(device) == 0
    assert gpu.calls == [("kda_device_status", where, 1000 * where + 7)]
    assert gpu.current == 0


F32, I32 = torch.float32, torch.int32
NEW = {
    "kda_mla_append": lambda: kda.mla_append(t(4, 576), None, t(2, 16, 576), t(2, 1, dtype=I32), t(2, dtype=I32)),
    "kda_mla_prefill": lambda: kda.mla_prefill(t(4, 2, 192), t(4, 2, 128), t(4, 64), t(4, 2, 128), o=t(4, 2, 128)),
    "kda_mla_decode": lambda: kda.mla_decode(t(2, 1, 2, 576), t(2, 16, 576), t(2, 1, dtype=I32), t(2, dtype=I32),
                                             o=t(2, 1, 2, 512), workspace=t(64, dtype=torch.uint8)),
    "kda_decode_tree": lambda: kda.decode_tree(*[t(2, 3, 2, 128)] * 4, t(2, 3, 2), t(2, 2, 128, 128, dtype=F32),
                                               o=t(2, 3, 2, 128)),
}


@pytest.mark.parametrize("name", NEW)
def test_calls_run_on_their_tensors_device(gpu, name):
    NEW[name]()
    assert gpu.calls == [(name, 1, 1007)] and gpu.current == 0


C = (t(70, 2, 128), t(70, 2, 128), t(70, 2, 128), t(70, 2, 128, dtype=F32), t(70, 2, dtype=F32))
OUT = dict(o=t(70, 2, 128), hT=t(1, 2, 128, 128, dtype=F32))
KDA = {
    "kda_chunk_fwd_ws": lambda: kda.chunk_fwd(*C, **OUT),
    "kda_chunk_fwd_simt": lambda: kda.chunk_fwd(*C, **OUT, kernel="simt"),
    "kda_chunk_fwd_static": lambda: kda.chunk_fwd(*C, **OUT, kernel="static"),
    "kda_gdn_chunk_fwd_ws": lambda: kda.gdn_chunk_fwd(*C[:3], t(70, 2, dtype=F32), C[4], **OUT),
    "kda_chunk_fwd_fused": lambda: kda.chunk_fwd_fused(*C[:3], C[0], C[4], C[0], t(128, dtype=F32), **OUT),
    "kda_short_conv_swish": lambda: kda.short_conv_swish(t(5, 2, 128), t(256, 4, dtype=F32), y=t(5, 2, 128)),
    "kda_decode_step": lambda: kda.decode_step(*[t(3, 2, 128)] * 4, t(3, 2), t(3, 2, 128, 128, dtype=F32),
                                               o=t(3, 2, 128)),
    "kda_decode_tokens": lambda: kda.decode_tokens(*[t(2, 3, 2, 128)] * 4, t(2, 3, 2),
                                                   t(2, 2, 128, 128, dtype=F32), o=t(2, 3, 2, 128)),
}


@pytest.mark.parametrize("name", KDA)
def test_kda_calls_run_on_their_tensors_device(gpu, name):
    KDA[name]()
    assert gpu.calls == [(name, 1, 1007)] and gpu.current == 0
