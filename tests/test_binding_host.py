"""The binding's host side on a stand-in for torch.cuda and the library: on which
stream and device a call allocates and launches.  No GPU is touched."""
import contextlib
from types import SimpleNamespace

import pytest
import torch


@pytest.fixture()
def lib(monkeypatch):
    """_lib on a machine with two stand-in GPUs.  lib.log holds what was done, as
    (what, current device, that device's current stream)."""
    from adaln_video_dit_gb300 import build
    build.build()
    from adaln_video_dit_gb300 import _lib
    current = SimpleNamespace(device=0, stream={0: 0, 1: 0})  # default streams: handle 0
    log = []

    def note(what):
        log.append((what, current.device, current.stream[current.device]))

    @contextlib.contextmanager
    def on_device(index):
        before, current.device = current.device, index
        yield
        current.device = before

    @contextlib.contextmanager
    def on_stream(s):
        before = current.stream[s.device_index]
        current.stream[s.device_index] = s.cuda_stream
        with on_device(s.device_index):
            yield
        current.stream[s.device_index] = before

    def empty(*shape, device, dtype):
        shape = shape[0] if isinstance(shape[0], tuple) else shape
        note("empty")
        return Tensor(*shape, dtype=dtype, device=device.index)

    def entry(name):
        def call(*args):
            note(name)
            log.append(("stream", args[-1]))
            return 0
        return call

    cuda = SimpleNamespace(stream=on_stream, device=on_device, current_device=lambda: current.device)
    c = SimpleNamespace(_cuda_getDevice=lambda: current.device,
                        _cuda_getCurrentRawStream=lambda i: current.stream[i])
    names = ("float32", "bfloat16", "int32", "uint8")
    monkeypatch.setattr(_lib, "torch", SimpleNamespace(
        cuda=cuda, _C=c, empty=empty, empty_like=lambda t: empty(t.shape, device=t.device, dtype=t.dtype),
        **{n: getattr(torch, n) for n in names}))
    monkeypatch.setattr(_lib, "raw", SimpleNamespace(**{n: entry(n) for n in _lib.EXPORTS}))
    monkeypatch.setattr(_lib, "_binding", SimpleNamespace(
        **{n: entry(n) for n in ("qk_rope_fwd", "qk_rope_bwd", "ffn_fwd", "ffn_bwd")}))
    monkeypatch.setattr(_lib, "log", log, raising=False)
    return _lib


class Tensor:
    """What the binding asks of a CUDA tensor."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.float32, device=0):
        self.shape, self.dtype, self.device = shape, dtype, torch.device("cuda", device)

    def get_device(self):
        return self.device.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def numel(self):
        return 1 << 30

    def element_size(self):
        return 1


def adaln_calls(L, device=0, **kw):
    """Every AdaLN call, its outputs and workspace to be allocated."""
    x, m, v = (Tensor(*s, device=device) for s in ((6, 8), (2, 8), (6,)))
    seg = Tensor(6, dtype=torch.int32, device=device)
    return {"adaln_fwd": lambda: L.adaln_fwd(x, m, m, seg, 1e-6, **kw),
            "adaln_bwd": lambda: L.adaln_bwd(x, x, v, v, m, seg, **kw),
            "adaln_bwd_noalloc": lambda: L.adaln_bwd_noalloc(x, x, v, v, m, seg, **kw)}


def other_calls(L, device=0, **kw):
    x = Tensor(4, 2, 8, device=device)
    return {"qk_rope_fwd": lambda: L.adaln_qk_rope_fwd(x, x, x, x, (4,), **kw),
            "qk_rope_bwd": lambda: L.adaln_qk_rope_bwd(x, x, x, x, (4,), **kw),
            "ffn_fwd": lambda: L.adaln_ffn_fwd(x, x, x, x, **kw),
            "ffn_bwd": lambda: L.adaln_ffn_bwd(x, x, x, x, x, x, **kw)}


def test_a_call_on_a_given_stream_allocates_there(lib):
    s = SimpleNamespace(cuda_stream=77, device_index=0, device=torch.device("cuda", 0))
    for name, call in {**adaln_calls(lib, stream=s), **other_calls(lib, stream=s)}.items():
        lib.log.clear()
        call()
        whats = [e for e in lib.log if e[0] != "stream"]
        assert (name, 0, 77) in whats and all(e[1:] == (0, 77) for e in whats), (name, lib.log)
        if name.startswith("adaln"):
            assert ("empty", 0, 77) in whats and ("stream", 77) in lib.log
