"""The binding's host side of the branch's calls (dropout, experts) on a stand-in for
two GPUs: on which stream and device a call allocates and launches.  No GPU is touched."""
from types import SimpleNamespace

import pytest
import torch

from test_binding_host import Tensor, lib  # noqa: F401 (a fixture)


@pytest.fixture()
def branch(lib, monkeypatch):  # noqa: F811
    """The stand-in, with the branch's marshalling in it: each call notes where it is."""
    def entry(name, result):
        def call(*args):
            lib.torch.empty(1, device=torch.device("cuda", args[0].get_device()), dtype=torch.uint8)
            lib.log.append((name, "on", args[-1]))
            return result
        return call

    monkeypatch.setattr(lib, "_binding", SimpleNamespace(
        route=entry("route", (None, None, None, 64)),
        **{n: entry(n, None) for n in ("dropout_fwd", "dropout_bwd", "expert_sort_fwd", "expert_sort_bwd",
                                       "expert_combine_fwd", "expert_combine_bwd", "experts_ffn_fwd",
                                       "experts_ffn_bwd")}))
    return lib


def calls(L, device=0, **kw):
    x, w, e = Tensor(6, 8, device=device), Tensor(2, 8, 8, device=device), Tensor(6, 2, dtype=torch.int32, device=device)
    r = L.Route(e, e, e, 64, 64)
    return [lambda: L.adaln_dropout_fwd(x, 0.1, (1, 2), **kw), lambda: L.adaln_dropout_bwd(x, 0.1, (1, 2), **kw),
            lambda: L.adaln_route(e, 2, **kw), lambda: L.adaln_expert_sort_fwd(x, r, **kw),
            lambda: L.adaln_expert_sort_bwd(x, r, **kw), lambda: L.adaln_expert_combine_fwd(x, x, r, **kw),
            lambda: L.adaln_expert_combine_bwd(x, x, x, r, **kw),
            lambda: L.adaln_experts_ffn_fwd(x, w, w, w, e, **kw),
            lambda: L.adaln_experts_ffn_bwd(x, x, w, w, w, e, x, **kw)]


@pytest.mark.parametrize("device", [0, 1])
def test_a_call_runs_on_its_tensors_device_and_stream(branch, device):
    s = SimpleNamespace(cuda_stream=77, device_index=device, device=torch.device("cuda", device))
    for kw, stream in (({}, 0), ({"stream": s}, 77)):
        for call in calls(branch, device, **kw):
            branch.log.clear()
            call()
            assert branch.log[0] == ("empty", device, stream), branch.log
            assert len(branch.log) == 2 and branch.log[1][1:] == ("on", kw.get("stream"))
    far = SimpleNamespace(cuda_stream=77, device_index=1 - device, device=torch.device("cuda", 1 - device))
    for call in calls(branch, device, stream=far):
        branch.log.clear()
        with pytest.raises(ValueError, match="cuda:"):
            call()
        assert not branch.log
