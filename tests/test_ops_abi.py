"""Host-side argument checks of the rotary and feed-forward entry points: refused before any
CUDA call (no GPU is touched; addresses are never dereferenced)."""
import ctypes

import pytest

A, B, ODD = 0x10000, 0x20000, 0x10001


@pytest.fixture(scope="module")
def lib():
    from adaln_video_dit_gb300 import build
    build.build()
    from adaln_video_dit_gb300 import _lib
    return _lib


def rope_of(lib, **kw):
    a = dict(table=A, pos=B, rows=9, axes=3, pairs=(22, 21, 21, 0), interleaved=1)
    a.update(kw)
    a["pairs"] = (ctypes.c_int32 * 4)(*a["pairs"])
    return lib.Rope(*a.values())


def rope_fwd(lib, rope=None, **kw):
    h = lib.Heads(A, 1024, 128)
    a = dict(q=h, k=h, T=10, hq=8, hk=2, dh=128, dt=lib.ADALN_BF16, rope=rope or rope_of(lib),
             norm=1, wq=A, wk=A, eps=1e-6, qo=h, ko=h)
    a.update(kw)
    return lib.raw.adaln_qk_rope_fwd(*a.values(), None)


def rope_bwd(lib, rope=None, **kw):
    h = lib.Heads(A, 1024, 128)
    a = dict(dqo=h, dko=h, q=h, k=h, T=10, hq=8, hk=2, dh=128, dt=lib.ADALN_BF16,
             rope=rope or rope_of(lib), norm=1, wq=A, wk=A, eps=1e-6, dq=h, dk=h, dwq=A, dwk=A,
             ws=B, wsb=1 << 30)
    a.update(kw)
    return lib.raw.adaln_qk_rope_bwd(*a.values(), None)


@pytest.mark.parametrize("call", [rope_fwd, rope_bwd])
def test_rope_refusals(lib, call):
    H = lib.Heads
    assert call(lib, dt=2) == lib.ADALN_ERR_DTYPE
    for bad in (dict(T=-1), dict(T=2 ** 31), dict(dh=0), dict(dh=513), dict(hq=-1),
                dict(hq=4097), dict(hq=0, hk=0), dict(dh=126), dict(q=H(A, -8, 128))):
        assert call(lib, **bad) == lib.ADALN_ERR_DIM, bad
    for bad in (dict(axes=0), dict(axes=5), dict(rows=0), dict(pairs=(65, -1, 0, 0)),
                dict(pairs=(0, 0, 0, 0)), dict(pairs=(2 ** 31 - 1,) * 3 + (0,))):
        assert call(lib, rope=rope_of(lib, **bad)) == lib.ADALN_ERR_DIM, bad
    for bad in (dict(q=None), dict(k=None), dict(q=H(None, 1024, 128))):
        assert call(lib, **bad) == lib.ADALN_ERR_NULL, bad
    for bad in (dict(table=None), dict(pos=None)):
        assert call(lib, rope=rope_of(lib, **bad)) == lib.ADALN_ERR_NULL
    for bad in (dict(q=H(ODD, 1024, 128)), dict(wk=ODD), dict(k=H(A + 2, 1024, 128),
                                                                dt=lib.ADALN_F32)):
        assert call(lib, **bad) == lib.ADALN_ERR_ALIGN, bad
    assert call(lib, rope=rope_of(lib, table=A + 4)) == lib.ADALN_ERR_ALIGN
    assert call(lib, rope=rope_of(lib, pos=A + 2)) == lib.ADALN_ERR_ALIGN
    for eps in (-1e-6, float("nan"), float("inf")):
        assert call(lib, eps=eps) == lib.ADALN_ERR_ARG


def test_rope_only_what_is_missing_is_refused(lib):
    none = lib.Heads(None, 0, 0)
    rope = rope_of(lib, table=None, pos=None)
    assert rope_fwd(lib, rope=rope, T=0, q=none, k=none, qo=none, ko=none) == lib.ADALN_OK
    assert rope_fwd(lib, T=0, hk=0, k=None, ko=None) == lib.ADALN_OK
    assert rope_bwd(lib, norm=0, q=None, k=None) == lib.ADALN_ERR_ARG  # no weights, no gradients
    assert rope_bwd(lib, norm=0, T=0, q=None, k=None, dwq=None, dwk=None, ws=None) == lib.ADALN_OK
    assert rope_bwd(lib, ws=None) == lib.ADALN_ERR_NULL
    assert rope_bwd(lib, ws=A + 8) == lib.ADALN_ERR_ALIGN
    assert rope_bwd(lib, dwk=A + 2) == lib.ADALN_ERR_ALIGN
    n = lib.raw.adaln_qk_rope_bwd_workspace_size
    assert n(1, 1, 1, 0, 0, None) == lib.ADALN_ERR_DIM
    assert n(1, 1, 1, 8, 0, None) == lib.ADALN_ERR_NULL


def test_rope_binding_rejects_host_tensors(lib):
    import torch
    x = torch.zeros(4, 2, 8)
    with pytest.raises(ValueError):
        lib.adaln_qk_rope_fwd(x, None, torch.zeros(3, 4, 2), torch.zeros(4, 1, dtype=torch.int32),
                              (4,))
    assert lib.strerror(lib.ADALN_ERR_POS) != lib.strerror(12345)


def ffn_fwd(lib, **kw):
    a = dict(x=A, wg=A, wu=A, wd=A, T=10, D=64, F=128, dt=lib.ADALN_BF16, act=0, y=B, saved=B, ws=B,
             wsb=1 << 30)
    a.update(kw)
    return lib.raw.adaln_ffn_fwd(*a.values(), None)


def ffn_bwd(lib, **kw):
    a = dict(dy=A, x=A, wg=A, wu=A, wd=A, saved=A, T=10, D=64, F=128, dt=lib.ADALN_BF16, act=0,
             dx=B, dwg=B, dwu=B, dwd=B, ws=B, wsb=1 << 30)
    a.update(kw)
    return lib.raw.adaln_ffn_bwd(*a.values(), None)


@pytest.mark.parametrize("call", [ffn_fwd, ffn_bwd])
def test_ffn_refusals(lib, call):
    assert call(lib, dt=lib.ADALN_F32) == lib.ADALN_ERR_DTYPE
    for bad in (dict(T=-1), dict(T=2 ** 24 + 1), dict(D=0), dict(D=12), dict(F=4), dict(F=100),
                dict(D=2 ** 18 + 8), dict(F=-8)):
        assert call(lib, **bad) == lib.ADALN_ERR_DIM, bad
    assert call(lib, act=3) == lib.ADALN_ERR_ARG
    for k in ("x", "wg", "wu", "wd", "ws"):
        assert call(lib, **{k: None}) == lib.ADALN_ERR_NULL, k
        assert call(lib, **{k: A + 8}) == lib.ADALN_ERR_ALIGN, k


def test_ffn_only_what_is_missing_is_refused(lib):
    assert ffn_fwd(lib, y=None) == lib.ADALN_ERR_NULL
    assert ffn_fwd(lib, saved=B + 8) == lib.ADALN_ERR_ALIGN
    assert ffn_bwd(lib, saved=None) == lib.ADALN_ERR_NULL
    assert ffn_bwd(lib, T=0, dwd=None) == lib.ADALN_ERR_NULL
    assert ffn_fwd(lib, T=0, x=None, y=None, ws=None, saved=None) == lib.ADALN_OK
    n = ctypes.c_size_t(0)
    assert lib.raw.adaln_ffn_saved_size(40, 64, 40, lib.ADALN_BF16, ctypes.byref(n)) == lib.ADALN_OK
    assert n.value == 2 * 2 * 6144  # blocks of 32 x 32 values, two of 24 bits each
    assert lib.raw.adaln_ffn_saved_size(40, 64, 40, lib.ADALN_BF16, None) == lib.ADALN_ERR_NULL
    assert lib.raw.adaln_ffn_workspace_size(40, 64, 40, lib.ADALN_BF16, None, None) == lib.ADALN_ERR_NULL
    assert lib.raw.adaln_ffn_workspace_size(40, 64, 41, lib.ADALN_BF16, None, None) == lib.ADALN_ERR_DIM


def test_gated_ffn_saves_only_for_a_gradient(lib, monkeypatch):
    """Nothing is saved under no_grad() or inference_mode(), where the weights
    still require a gradient, nor for frozen weights."""
    import torch
    from adaln_video_dit_gb300 import autograd
    asked = []

    def fake(x, wg, wu, wd, act, save):
        asked.append(save)
        return torch.zeros_like(x), torch.zeros(1, dtype=torch.uint8) if save else None

    monkeypatch.setattr(autograd._lib, "adaln_ffn_fwd", fake)
    m, x = autograd.GatedFFN(8, 16), torch.zeros(3, 8, dtype=torch.bfloat16)
    assert m(x).requires_grad
    with torch.no_grad():
        assert not m(x).requires_grad
    with torch.inference_mode():
        m(x)
    m.requires_grad_(False)
    m(x)
    m(x.clone().requires_grad_())
    assert asked == [True, False, False, False, True]


def test_gradients_of_gradients_are_refused(lib, monkeypatch):
    """The backward passes have no derivative: asking for one is an error, not a zero."""
    import torch
    from adaln_video_dit_gb300 import autograd
    monkeypatch.setattr(autograd._lib, "adaln_ffn_fwd", lambda x, *a, **kw: (x * 1, x * 1))
    monkeypatch.setattr(autograd._lib, "adaln_ffn_bwd",
                        lambda dy, x, wg, wu, wd, *a, **kw: (dy * x, wg * 1, wu * 1, wd * 1))
    monkeypatch.setattr(autograd._lib, "adaln_qk_rope_fwd", lambda q, k, *a, **kw: (q * 1, None))
    monkeypatch.setattr(autograd._lib, "adaln_qk_rope_bwd",
                        lambda dq, dk, *a, **kw: (dq * 1, None, None, None))
    x = torch.ones(2, 8, dtype=torch.bfloat16, requires_grad=True)
    q = torch.ones(2, 1, 8, requires_grad=True)
    table, pos = torch.ones(1, 4, 2), torch.zeros(2, 1, dtype=torch.int32)
    for out, leaf in ((autograd.GatedFFN(8, 16)(x), x),
                      (autograd.qk_norm_rope(q, None, None, None, table, pos, (4,))[0], q)):
        first, = torch.autograd.grad((out * out).sum(), leaf, create_graph=True)
        with pytest.raises(RuntimeError, match="twice"):
            first.sum().backward()


def test_rope_outputs_that_overlap_themselves_are_refused(lib):
    H = lib.Heads
    for out in (H(A, 0, 128), H(A, 1024, 0), H(A, 127, 128), H(A, 1024, 127)):
        for bad in (dict(qo=out), dict(ko=out)):
            assert rope_fwd(lib, **bad) == lib.ADALN_ERR_DIM
        for bad in (dict(dq=out), dict(dk=out)):
            assert rope_bwd(lib, **bad) == lib.ADALN_ERR_DIM
            assert rope_bwd(lib, norm=0, dwq=None, dwk=None, **bad) == lib.ADALN_ERR_DIM
    # One token or one head has no next one, and an input may repeat (the calls
    # below get as far as the next refusal).
    far = dict(eps=-1.0)
    assert rope_fwd(lib, T=1, qo=H(A, 0, 128), **far) == lib.ADALN_ERR_ARG
    assert rope_fwd(lib, hq=1, qo=H(A, 1024, 0), **far) == lib.ADALN_ERR_ARG
    assert rope_fwd(lib, q=H(A, 0, 128), k=H(A, 1024, 0), **far) == lib.ADALN_ERR_ARG


def test_rope_outputs_that_overlap_across_both_axes_are_refused(lib):
    """Strides that are each at least dh may still bring two heads of different
    tokens together: every small layout, against the list of its elements."""
    H = lib.Heads
    for out, heads in ((H(A, 128, 128), 8), (H(A, 256, 128), 8), (H(A, 128, 256), 8),
                       (H(A, 300, 200), 4), (H(A, 1023, 128), 8)):
        assert rope_fwd(lib, qo=out, hq=heads) == lib.ADALN_ERR_DIM
        assert rope_fwd(lib, ko=out, hk=heads) == lib.ADALN_ERR_DIM
        assert rope_bwd(lib, dq=out, hq=heads) == lib.ADALN_ERR_DIM
        assert rope_bwd(lib, norm=0, dwq=None, dwk=None, dk=out, hk=heads) == lib.ADALN_ERR_DIM
    rope = rope_of(lib, axes=1, pairs=(1, 0, 0, 0))
    refused = 0
    for T in (1, 2, 3, 5):
        for heads in (1, 2, 4):
            for ts in range(0, 14):
                for hs in range(0, 14):
                    at = [t * ts + h * hs + d for t in range(T) for h in range(heads)
                          for d in range(2)]
                    rc = rope_fwd(lib, rope=rope, T=T, dh=2, hk=0, k=None, ko=None, hq=heads,
                                  qo=H(A, ts, hs), eps=-1.0)  # the next refusal, if not this one
                    meet = len(set(at)) < len(at)
                    assert rc == (lib.ADALN_ERR_DIM if meet else lib.ADALN_ERR_ARG), (T, heads, ts, hs)
                    refused += meet
    assert refused > 500
    # Strides whose products pass 64 bits.
    big = 1 << 62
    assert rope_fwd(lib, qo=H(A, big, big), eps=-1.0) == lib.ADALN_ERR_DIM
    assert rope_fwd(lib, qo=H(A, 128, big), eps=-1.0) == lib.ADALN_ERR_ARG


def test_norm_of_queries_alone_has_a_backward(lib, monkeypatch):
    """Without keys (a cross attention's queries) the keys' weight, which QKNormRope
    holds all the same, is not used: it has no gradient, and the backward runs."""
    import torch
    from adaln_video_dit_gb300 import autograd
    monkeypatch.setattr(autograd._lib, "adaln_qk_rope_fwd", lambda q, k, *a, **kw: (q * 1, None))
    monkeypatch.setattr(autograd._lib, "adaln_qk_rope_bwd",
                        lambda dq, dk, *a, **kw: (dq * 1, None, torch.full((8,), 3.0), None))
    m = autograd.QKNormRope(8, (4,))
    q = torch.ones(2, 1, 8, requires_grad=True)
    out, none = m(q, None, torch.ones(1, 4, 2), torch.zeros(2, 1, dtype=torch.int32))
    assert none is None
    out.sum().backward()
    assert torch.equal(q.grad, torch.ones_like(q))
    assert torch.equal(m.wq.grad, torch.full((8,), 3.0)) and m.wk.grad is None


def test_gradients_of_the_modulations_gradients_are_refused(lib, monkeypatch):
    """The AdaLN's backward has no derivative either."""
    import torch
    from adaln_video_dit_gb300 import autograd
    monkeypatch.setattr(autograd._lib, "adaln_fwd", lambda x, *a: (x * 1, x[:, 0] * 1, x[:, 0] * 1))
    monkeypatch.setattr(autograd._lib, "adaln_bwd",
                        lambda dy, x, mean, rstd, scale, seg: (dy * x, scale * 1, scale * 1))
    x = torch.ones(2, 8, requires_grad=True)
    m, seg = torch.zeros(1, 8, requires_grad=True), torch.zeros(2, dtype=torch.int32)
    out = autograd.adaln_modulate(x, m, m, seg)
    first, = torch.autograd.grad((out * out).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="twice"):
        first.sum().backward()


def test_rotary_nodes_take_leading_dimensions(lib, monkeypatch):
    """[..., heads, dh] with pos [..., axes], as the other nodes take [..., D]: the
    call gets tokens, a packed projection's views without a copy."""
    import torch
    from adaln_video_dit_gb300 import autograd
    seen = []

    def fwd(q, k, table, pos, *how, **kw):
        seen.append((q.shape, q.stride(), q.data_ptr(), k if k is None else k.shape, pos.shape))
        return q * 2, None if k is None else k * 3

    monkeypatch.setattr(autograd._lib, "adaln_qk_rope_fwd", fwd)
    monkeypatch.setattr(autograd._lib, "adaln_qk_rope_bwd", lambda dq, dk, *a, **kw: (
        dq * 2, None if dk is None else dk * 3, None, None))
    qkv = torch.randn(2, 5, 3, 4, 8, requires_grad=True)
    q, k, _ = qkv.unbind(2)
    table, pos = torch.ones(1, 4, 2), torch.zeros(2, 5, 1, dtype=torch.int32)
    qo, ko = autograd.qk_norm_rope(q, k, None, None, table, pos, (4,))
    assert seen == [((10, 4, 8), (96, 8, 1), qkv.data_ptr(), (10, 4, 8), (10, 1))]
    assert torch.equal(qo, 2 * q) and torch.equal(ko, 3 * k)
    (qo.sum() + ko.sum()).backward()
    assert torch.equal(qkv.grad[:, :, 0], torch.full((2, 5, 4, 8), 2.0))
    assert torch.equal(qkv.grad[:, :, 1], torch.full((2, 5, 4, 8), 3.0))
    out, none = autograd.qk_rope(q[0, 0], None, table, pos[0, 0], (4,))  # one token's heads
    assert none is None and out.shape == (4, 8) and seen[-1][0] == (1, 4, 8)
