"""Host-side checks of the residual branch's entry points (dropout with gate and
residual): refused before any CUDA call, no address is dereferenced; what the nodes
save; and the generator of the tests' own reference against published values."""
import ctypes

import numpy as np
import pytest

from philox import kept, philox

A, B = 0x10000, 0x20000


@pytest.fixture(scope="module")
def lib():
    from adaln_video_dit_gb300 import build
    build.build()
    from adaln_video_dit_gb300 import _lib
    return _lib


def test_the_reference_generator_gives_the_published_values():
    """The known answers published with the generator."""
    for c, k, want in (
            ((0,) * 4, (0,) * 2, (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        assert tuple(int(x) for x in philox(c, k)) == want
    # (Of 2^20 draws the share kept is within five standard deviations of its mean.)
    for p in (0.1, 0.5):
        share = kept(np.arange(1024), 1024, p, 5, 9)[0].mean()
        assert abs(share - (1 - p)) <= 5 * (p * (1 - p)) ** 0.5 / 1024


def drop_fwd(lib, rng=True, **kw):
    r = lib.Rng(1, 2, None) if rng is True else rng
    a = dict(h=A, x=A, gate=A, seg=A, T=10, D=64, nseg=2, dt=lib.ADALN_BF16, p=0.1,
             rng=ctypes.byref(r) if r is not None else None, y=B)
    a.update(kw)
    return lib.raw.adaln_dropout_fwd(*a.values(), None)


def drop_bwd(lib, rng=True, **kw):
    r = lib.Rng(1, 2, None) if rng is True else rng
    a = dict(dy=A, h=A, gate=A, seg=A, T=10, D=64, nseg=2, dt=lib.ADALN_BF16, p=0.1,
             rng=ctypes.byref(r) if r is not None else None, dh=B, dgate=B, ws=B, wsb=1 << 30)
    a.update(kw)
    return lib.raw.adaln_dropout_bwd(*a.values(), None)


@pytest.mark.parametrize("call", [drop_fwd, drop_bwd])
def test_dropout_refusals(lib, call):
    assert call(lib, dt=2) == lib.ADALN_ERR_DTYPE
    for bad in (dict(T=-1), dict(T=2 ** 31), dict(D=0), dict(D=12), dict(D=2 ** 18 + 8), dict(nseg=0),
                dict(nseg=2 ** 24 + 1), dict(D=6, dt=lib.ADALN_F32), dict(T=2 ** 31 - 1, D=2 ** 8)):
        assert call(lib, **bad) == lib.ADALN_ERR_DIM, bad
    for p in (-0.1, 1.5, float("nan"), float("inf")):
        assert call(lib, p=p) == lib.ADALN_ERR_ARG
    assert call(lib, rng=None) == lib.ADALN_ERR_NULL
    assert call(lib, rng=lib.Rng(0, 0, A + 4)) == lib.ADALN_ERR_ALIGN
    assert call(lib, seg=None) == lib.ADALN_ERR_NULL
    assert call(lib, gate=A + 8) == lib.ADALN_ERR_ALIGN
    assert call(lib, seg=A + 2) == lib.ADALN_ERR_ALIGN


def test_dropout_only_what_is_missing_is_refused(lib):
    assert drop_fwd(lib, h=None) == lib.ADALN_ERR_NULL
    assert drop_fwd(lib, y=None) == lib.ADALN_ERR_NULL
    for k in ("h", "x", "y"):
        assert drop_fwd(lib, **{k: A + 8}) == lib.ADALN_ERR_ALIGN, k
    for k in ("dy", "h", "gate", "dh", "ws"):
        assert drop_bwd(lib, **{k: None}) == lib.ADALN_ERR_NULL, k
    for k in ("dy", "h", "dh", "dgate", "ws"):
        assert drop_bwd(lib, **{k: A + 8}) == lib.ADALN_ERR_ALIGN, k
    assert drop_fwd(lib, T=0, h=None, y=None) == lib.ADALN_OK
    assert drop_bwd(lib, T=0, dy=None, dh=None, dgate=None) == lib.ADALN_OK
    assert lib.raw.adaln_dropout_bwd_workspace_size(4, 64, 1, 1, None) == lib.ADALN_ERR_NULL
    n = ctypes.c_size_t(0)
    assert lib.raw.adaln_dropout_bwd_workspace_size(4, 60, 1, 1, ctypes.byref(n)) == lib.ADALN_ERR_DIM


def test_kernel_ids(lib):
    n, ms = ctypes.c_int64(-1), ctypes.c_double(-1)
    got = [lib.raw.adaln_trace_get(i, ctypes.byref(n), ctypes.byref(ms)) for i in range(-1, 9)]
    assert got[lib.ADALN_KERNEL_DROPOUT + 1] == lib.ADALN_OK
    assert got[0] == got[6] == got[9] == lib.ADALN_ERR_ARG


def test_dropout_saves_h_for_a_gates_gradient_only(lib, monkeypatch):
    import torch
    from adaln_video_dit_gb300 import autograd
    seen = []

    def fwd(h, p, rng, x=None, gate=None, seg_id=None):
        seen.append((tuple(h.shape), None if x is None else tuple(x.shape), p))
        return h * 1

    def bwd(dy, p, rng, h=None, gate=None, seg_id=None):
        seen.append(("back", h is not None, rng))
        return dy * 2, None if h is None else torch.full(gate.shape, 3.0)

    monkeypatch.setattr(autograd._lib, "adaln_dropout_fwd", fwd)
    monkeypatch.setattr(autograd._lib, "adaln_dropout_bwd", bwd)
    h, x = (torch.ones(2, 3, 8, requires_grad=True) for _ in range(2))
    gate, seg = torch.zeros(2, 8, requires_grad=True), torch.zeros(6, dtype=torch.int32)
    autograd.gated_residual(x, h, gate, seg, 0.5, (1, 2)).sum().backward()
    assert seen == [((6, 8), (6, 8), 0.5), ("back", True, (1, 2))]
    assert torch.equal(h.grad, torch.full((2, 3, 8), 2.0)) and torch.equal(x.grad, torch.ones(2, 3, 8))
    assert torch.equal(gate.grad, torch.full((2, 8), 3.0))
    seen.clear()
    autograd.gated_residual(x, h, gate.detach(), seg, 0.5, (1, 2)).sum().backward()
    assert seen[1] == ("back", False, (1, 2))
    seen.clear()  # a branch without a gradient costs no backward call
    autograd.gated_residual(x, h.detach(), gate.detach(), seg, 0.5, (1, 2)).sum().backward()
    assert len(seen) == 1
    # A generator's state changed between forward and backward would give another mask.
    rng = torch.tensor([1, 2])
    y = autograd.dropout(h, 0.5, rng)
    rng += 1
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        y.sum().backward()
    out = autograd.dropout(h, 0.5, (1, 2))
    first, = torch.autograd.grad((out * out).sum(), h, create_graph=True)
    with pytest.raises(RuntimeError, match="twice"):
        first.sum().backward()
    with pytest.raises(ValueError):
        autograd.GatedResidual(1.5)
    seen.clear()
    m = autograd.GatedResidual(0.5).eval()
    m(x, h, gate, seg)
    assert seen[0][2] == 0.0


def route(lib, **kw):
    a = dict(expert=A, T=10, k=2, E=4, align=64, row=B, starts=B, counts=B, ws=B, wsb=1 << 30)
    a.update(kw)
    return lib.raw.adaln_route(*a.values(), None)


def sort_fwd(lib, **kw):
    a = dict(x=A, row=A, starts=A, counts=A, T=10, k=2, E=4, align=64, D=64, dt=lib.ADALN_BF16, rows=256,
             xs=B)
    a.update(kw)
    return lib.raw.adaln_expert_sort_fwd(*a.values(), None)


def sort_bwd(lib, **kw):
    a = dict(dxs=A, row=A, T=10, k=2, D=64, dt=lib.ADALN_BF16, rows=256, dx=B)
    a.update(kw)
    return lib.raw.adaln_expert_sort_bwd(*a.values(), None)


def combine_fwd(lib, **kw):
    a = dict(ys=A, weight=A, row=A, T=10, k=2, D=64, dt=lib.ADALN_BF16, rows=256, y=B)
    a.update(kw)
    return lib.raw.adaln_expert_combine_fwd(*a.values(), None)


def combine_bwd(lib, **kw):
    a = dict(dy=A, ys=A, weight=A, row=A, starts=A, counts=A, T=10, k=2, E=4, align=64, D=64,
             dt=lib.ADALN_BF16, rows=256, dys=B, dw=B)
    a.update(kw)
    return lib.raw.adaln_expert_combine_bwd(*a.values(), None)


def test_route_refusals(lib):
    for bad in (dict(T=-1), dict(T=2 ** 31), dict(k=0), dict(k=33), dict(E=0), dict(E=257), dict(align=0),
                dict(align=4097), dict(T=2 ** 31 - 1), dict(T=2 ** 30 - 1, E=256, align=4096)):
        assert route(lib, **bad) == lib.ADALN_ERR_DIM, bad
    for k in ("expert", "row", "starts", "counts"):
        assert route(lib, **{k: None}) == lib.ADALN_ERR_NULL, k
        assert route(lib, **{k: A + 2}) == lib.ADALN_ERR_ALIGN, k
    big = dict(T=70000)
    assert route(lib, ws=None, **big) == lib.ADALN_ERR_NULL
    assert route(lib, ws=A + 8, **big) == lib.ADALN_ERR_ALIGN
    assert route(lib, wsb=16, **big) == lib.ADALN_ERR_WORKSPACE
    assert route(lib, T=0, starts=None) == lib.ADALN_ERR_NULL
    n = ctypes.c_int64(0)
    for (T, k, E, align), rows in (((10, 2, 4, 64), 256), ((0, 2, 4, 64), 0), ((1, 2, 8, 64), 128),
                                   ((5, 3, 8, 1), 15), ((100, 1, 2, 64), 192)):
        assert lib.raw.adaln_route_rows(T, k, E, align, ctypes.byref(n)) == lib.ADALN_OK
        assert n.value == rows, (T, k, E, align)
    assert lib.raw.adaln_route_rows(1, 1, 1, 1, None) == lib.ADALN_ERR_NULL
    assert lib.adaln_route_workspace_size(65536, 2, 256) == 0 < lib.adaln_route_workspace_size(65537, 2, 1)


@pytest.mark.parametrize("call", [sort_fwd, sort_bwd, combine_fwd, combine_bwd])
def test_expert_copy_refusals(lib, call):
    names = call(lib, T=0) == lib.ADALN_OK and {
        sort_fwd: ("x", "row", "starts", "counts", "xs"), sort_bwd: ("dxs", "row", "dx"),
        combine_fwd: ("ys", "weight", "row", "y"),
        combine_bwd: ("dy", "ys", "weight", "row", "starts", "counts", "dys", "dw")}[call]
    assert call(lib, dt=2) == lib.ADALN_ERR_DTYPE
    for bad in (dict(T=-1), dict(T=2 ** 31), dict(k=0), dict(k=33), dict(D=0), dict(D=12), dict(D=2 ** 18 + 8),
                dict(rows=-1), dict(rows=2 ** 31)):
        assert call(lib, **bad) == lib.ADALN_ERR_DIM, bad
    if "starts" in names:
        for bad in (dict(E=0), dict(E=257), dict(align=0), dict(align=4097)):
            assert call(lib, **bad) == lib.ADALN_ERR_DIM, bad
    for k in names:
        assert call(lib, **{k: None}) == lib.ADALN_ERR_NULL, k
        assert call(lib, **{k: A + 2}) == lib.ADALN_ERR_ALIGN, k
        assert call(lib, **{k: None}, T=0) == lib.ADALN_OK, k


def test_expert_statuses(lib):
    assert lib.strerror(lib.ADALN_ERR_EXPERT) != lib.strerror(12345)
    n, ms = ctypes.c_int64(-1), ctypes.c_double(-1)
    assert lib.raw.adaln_trace_get(lib.ADALN_KERNEL_EXPERTS, ctypes.byref(n), ctypes.byref(ms)) == lib.ADALN_OK


def test_expert_nodes_keep_shapes_and_types(lib, monkeypatch):
    import torch
    from adaln_video_dit_gb300 import autograd
    L = autograd._lib
    monkeypatch.setattr(L, "adaln_route", lambda e, E, align: L.Route(
        e, torch.zeros(E + 1, dtype=torch.int32), torch.zeros(E, dtype=torch.int32), 7, align))
    monkeypatch.setattr(L, "adaln_expert_sort_fwd", lambda x, r: torch.ones(r.rows, x.shape[1]))
    monkeypatch.setattr(L, "adaln_expert_sort_bwd", lambda d, r: torch.full((len(r.row), d.shape[1]), 2.0))
    monkeypatch.setattr(L, "adaln_expert_combine_fwd", lambda ys, w, r: torch.ones(len(r.row), ys.shape[1]))
    monkeypatch.setattr(L, "adaln_expert_combine_bwd", lambda d, ys, w, r: (ys * 0 + 3, w * 0 + 4))
    x = torch.zeros(2, 5, 8, requires_grad=True)
    weight = torch.zeros(2, 5, 3, dtype=torch.bfloat16, requires_grad=True)
    r = autograd.route(torch.zeros(2, 5, 3, dtype=torch.int64), 4)
    assert r.row.shape == (10, 3) and r.row.dtype == torch.int32
    xs = autograd.expert_sort(x, r)
    xs.retain_grad()
    y = autograd.expert_combine(xs, weight, r)
    assert xs.shape == (7, 8) and y.shape == (2, 5, 8)
    y.sum().backward()
    assert torch.equal(xs.grad, torch.full((7, 8), 3.0)) and torch.equal(x.grad, torch.full((2, 5, 8), 2.0))
    assert weight.grad.dtype == torch.bfloat16 and weight.grad.shape == (2, 5, 3)
    for out, leaf in ((autograd.expert_sort(x, r), x), (autograd.expert_combine(xs.detach(), weight, r), weight)):
        first, = torch.autograd.grad((out * out).sum(), leaf, create_graph=True)
        with pytest.raises(RuntimeError, match="twice"):
            first.sum().backward()


def experts_fwd(lib, **kw):
    a = dict(xs=A, wg=A, wu=A, wd=A, starts=A, rows=256, E=4, D=64, F=128, dt=lib.ADALN_BF16, act=0, ys=B,
             saved=B, ws=B, wsb=1 << 30)
    a.update(kw)
    return lib.raw.adaln_experts_ffn_fwd(*a.values(), None)


def experts_bwd(lib, **kw):
    a = dict(dys=A, xs=A, wg=A, wu=A, wd=A, starts=A, saved=A, rows=256, E=4, D=64, F=128,
             dt=lib.ADALN_BF16, act=0, dxs=B, dwg=B, dwu=B, dwd=B, ws=B, wsb=1 << 30)
    a.update(kw)
    return lib.raw.adaln_experts_ffn_bwd(*a.values(), None)


@pytest.mark.parametrize("call", [experts_fwd, experts_bwd])
def test_experts_ffn_refusals(lib, call):
    assert call(lib, dt=lib.ADALN_F32) == lib.ADALN_ERR_DTYPE
    for bad in (dict(rows=-1), dict(rows=2 ** 24 + 1), dict(E=0), dict(E=257), dict(D=0), dict(D=12),
                dict(F=4), dict(F=100), dict(D=2 ** 18 + 8), dict(F=-8)):
        assert call(lib, **bad) == lib.ADALN_ERR_DIM, bad
    assert call(lib, act=3) == lib.ADALN_ERR_ARG
    for k in ("xs", "wg", "wu", "wd", "ws"):
        assert call(lib, **{k: None}) == lib.ADALN_ERR_NULL, k
        assert call(lib, **{k: A + 8}) == lib.ADALN_ERR_ALIGN, k
    assert call(lib, starts=None) == lib.ADALN_ERR_NULL
    assert call(lib, starts=A + 2) == lib.ADALN_ERR_ALIGN


def test_experts_ffn_only_what_is_missing_is_refused(lib):
    assert experts_fwd(lib, ys=None) == lib.ADALN_ERR_NULL
    assert experts_fwd(lib, saved=B + 8) == lib.ADALN_ERR_ALIGN
    for k in ("dys", "saved", "dxs", "dwg", "dwu", "dwd"):
        assert experts_bwd(lib, **{k: None}) == lib.ADALN_ERR_NULL, k
        assert experts_bwd(lib, **{k: A + 8}) == lib.ADALN_ERR_ALIGN, k
    assert experts_bwd(lib, rows=0, dwd=None) == lib.ADALN_ERR_NULL
    for rows in (0, 63):  # no expert can have a row
        assert experts_fwd(lib, rows=rows, xs=None, ys=None, ws=None, saved=None) == lib.ADALN_OK
    n = ctypes.c_size_t(0)
    f = lib.raw.adaln_experts_ffn_saved_size
    assert f(64, 2, 64, 40, lib.ADALN_BF16, ctypes.byref(n)) == lib.ADALN_OK
    assert n.value == 2 * 2 * 6144
    assert f(64, 2, 64, 40, lib.ADALN_BF16, None) == lib.ADALN_ERR_NULL
    g = lib.raw.adaln_experts_ffn_workspace_size
    assert g(64, 2, 64, 40, lib.ADALN_BF16, None, None) == lib.ADALN_ERR_NULL
    assert g(64, 2, 64, 41, lib.ADALN_BF16, None, None) == lib.ADALN_ERR_DIM


def test_experts_ffn_saves_only_for_a_gradient(lib, monkeypatch):
    import torch
    from adaln_video_dit_gb300 import autograd
    asked = []

    def fwd(xs, wg, wu, wd, starts, act, save):
        asked.append(save)
        return xs * 1, torch.zeros(1, dtype=torch.uint8) if save else None

    monkeypatch.setattr(autograd._lib, "adaln_experts_ffn_fwd", fwd)
    monkeypatch.setattr(autograd._lib, "adaln_experts_ffn_bwd", lambda dys, xs, wg, wu, wd, *a, **kw: (
        dys * xs, wg * 1, wu * 1, wd * 1))
    m = autograd.MixtureFFN(8, 16, 4)
    r = lib.Route(None, torch.zeros(5, dtype=torch.int32), None, 64, 64)
    with pytest.raises(ValueError, match="64"):
        autograd.experts_ffn(torch.ones(64, 8, dtype=torch.bfloat16), m.wg, m.wu, m.wd, r._replace(align=32))
    x = torch.ones(64, 8, dtype=torch.bfloat16)
    call = lambda t: autograd.experts_ffn(t, m.wg, m.wu, m.wd, r)  # noqa: E731
    assert call(x).requires_grad
    with torch.no_grad():
        assert not call(x).requires_grad
    m.requires_grad_(False)
    call(x)
    leaf = x.clone().requires_grad_()
    out = call(leaf)
    assert asked == [True, False, False, True]
    first, = torch.autograd.grad((out * out).sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError, match="twice"):
        first.sum().backward()
    for bad in (dict(top_k=0), dict(top_k=5), dict(act="relu")):
        with pytest.raises(ValueError):
            autograd.MixtureFFN(8, 16, 4, **bad)


def test_experts_are_of_a_signed_integer_type(lib, monkeypatch):
    """Anything else is refused before the call: uint32 and uint64 values that fit no
    int32 would wrap to an expert, or to -1."""
    import torch
    from adaln_video_dit_gb300 import autograd
    monkeypatch.setattr(autograd._lib, "adaln_route", lambda e, E, align: e)
    for dt in (torch.int8, torch.int16, torch.int32, torch.int64):
        got = autograd.route(torch.tensor([[1, -1]], dtype=dt), 5)
        assert got.dtype == torch.int32 and got.tolist() == [[1, -1]]
    for dt, v in ((torch.uint8, 1), (torch.uint16, 1), (torch.uint32, 2 ** 32 - 1), (torch.uint64, 2 ** 32 + 3),
                  (torch.bool, 1), (torch.float32, 1), (torch.bfloat16, 1), (torch.complex64, 1)):
        with pytest.raises(TypeError, match="signed integer"):
            autograd.route(torch.tensor([[1, v]], dtype=dt), 5)


def test_anomaly_detection_finds_nothing_in_rows_that_hold_nothing(lib, monkeypatch):
    """The calls leave the rows behind the last expert as they were.  A gradient with NaN
    there is no anomaly: where that is looked for, the nodes hand in zeros; elsewhere
    nothing, which costs nothing."""
    import torch
    from adaln_video_dit_gb300 import autograd
    L, given = autograd._lib, []
    used, rows = 3, 7

    def rows_of(like, out):
        given.append(out is not None)
        out = torch.full_like(like, float("nan")) if out is None else out
        out[:used] = 1
        return out

    monkeypatch.setattr(L, "adaln_expert_sort_fwd", lambda x, r: torch.ones(rows, x.shape[1], dtype=x.dtype))
    monkeypatch.setattr(L, "adaln_expert_sort_bwd", lambda d, r: d[:used] * 1)
    monkeypatch.setattr(L, "adaln_experts_ffn_fwd", lambda xs, *a, **kw: (xs * 1, xs))
    monkeypatch.setattr(L, "adaln_experts_ffn_bwd", lambda dys, xs, wg, wu, wd, starts, saved, act, dxs=None: (
        rows_of(xs, dxs), wg * 0, wu * 0, wd * 0))
    monkeypatch.setattr(L, "adaln_expert_combine_fwd", lambda ys, w, r: ys[:used] * 1)
    monkeypatch.setattr(L, "adaln_expert_combine_bwd", lambda d, ys, w, r, dys=None: (rows_of(ys, dys), w * 0))
    r = L.Route(torch.zeros(used, 1, dtype=torch.int32), torch.zeros(3, dtype=torch.int32),
                torch.zeros(2, dtype=torch.int32), rows, 64)

    def step():
        given.clear()
        x, w = torch.ones(used, 8, requires_grad=True), torch.ones(used, 1, requires_grad=True)
        m = [torch.ones(2, 8, 8, requires_grad=True) for _ in range(3)]
        autograd.expert_combine(autograd.experts_ffn(autograd.expert_sort(x, r), *m, r), w, r).sum().backward()
        return x.grad

    want = step()
    assert given == [False, False]
    with torch.autograd.detect_anomaly():
        assert torch.equal(step(), want)
    assert given == [True, True]
