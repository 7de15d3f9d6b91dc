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
    def on_device(device):
        index = device if isinstance(device, int) else device.index
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


class Host(Tensor):
    is_cuda = False

    def __init__(self, *shape, dtype=None):
        super().__init__(*shape, dtype=dtype or torch.float32)


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


def test_a_call_runs_on_its_tensors_device(lib):
    """With cuda:0 current, calls on cuda:1 (on its current stream, whose handle is
    the same 0, or on a given one) allocate, size and launch on cuda:1."""
    s = SimpleNamespace(cuda_stream=77, device_index=1, device=torch.device("cuda", 1))
    for kw, stream in (({}, 0), ({"stream": s}, 77)):
        for name, call in {**adaln_calls(lib, 1, **kw), **other_calls(lib, 1, **kw)}.items():
            lib.log.clear()
            call()
            whats = [e for e in lib.log if e[0] != "stream"]
            assert (name, 1, stream) in whats and all(e[1:] == (1, stream) for e in whats), (name, lib.log)
            assert lib.torch.cuda.current_device() == 0
    host = {n: Host(*s, dtype=d) for n, s, d in (
        ("x", (6, 8), None), ("y", (6, 8), None), ("dx", (6, 8), None), ("mean", (6,), None),
        ("rstd", (6,), None), ("dshift", (2, 8), None), ("dscale", (2, 8), None),
        ("seg", (6,), torch.int32))}
    lib.log.clear()
    lib.adaln_fwd_bwd_host(host["x"], host["x"], host["dshift"], host["dshift"], host["seg"], 1e-6, host,
                           Tensor(1, dtype=torch.uint8, device=1))
    assert lib.log[0] == ("adaln_fwd_bwd_host", 1, 0)
    for kw in (dict(device=1), dict(device=torch.device("cuda", 1)), dict(stream=s)):
        lib.log.clear()
        lib.adaln_get_status(**kw)
        assert lib.log[0] == ("adaln_get_status", 1, 0) and lib.torch.cuda.current_device() == 0


def test_tensors_and_streams_of_two_devices_are_refused(lib):
    s = SimpleNamespace(cuda_stream=77, device_index=1, device=torch.device("cuda", 1))
    for name, call in {**adaln_calls(lib, 0, stream=s), **other_calls(lib, 0, stream=s)}.items():
        with pytest.raises(ValueError, match="cuda:1"):
            call()
    x, m = Tensor(6, 8), Tensor(2, 8)
    seg, far = Tensor(6, dtype=torch.int32), Tensor(2, 8, device=1)
    v, w = Tensor(6), Tensor(6, device=1)
    for call in (lambda: lib.adaln_fwd(x, m, far, seg, 1e-6), lambda: lib.adaln_fwd(x, m, m, seg, 1e-6, mean=w),
                 lambda: lib.adaln_bwd(x, x, w, v, m, seg), lambda: lib.adaln_bwd(x, x, v, v, far, seg),
                 lambda: lib.adaln_bwd(x, x, v, v, m, seg, workspace=far),
                 lambda: lib.adaln_bwd_noalloc(x, x, v, v, m, seg, dshift=far),
                 lambda: lib.adaln_get_status(stream=s, device=0)):
        with pytest.raises(ValueError, match="cuda:1"):
            call()
    assert not [e for e in lib.log if e[0] in lib.EXPORTS and "size" not in e[0]]
