"""Rotary positions and per-head norm of queries and keys (adaln_qk_rope_*)
against the definition in 64 bits.

Tolerances, from the arithmetic (u = 2^-24, the fp32 rounding unit):
  a rotated element is two products and one sum of values with at most 5
  roundings each of their own norm, and the head's mean of squares is a sum of
  dh <= 512 squares in chains of at most 32 a lane and a tree of 5 levels, so
  its square root and quotient carry at most 32 u: 64 u of the head's largest
  |n| bounds the forward;
  dx adds two terms of sizes r |h| and r |x r| mean|h x r|, each with the
  forward's error and one more sum of that length: 128 u of their sum;
  dw sums its terms in chains of at most 64 here (128 in the cases of 12000
  tokens: tokens of a lane, lanes, warps and partial sums): 80 u (144 u) of the
  sum of |terms|;
  a bf16 output adds its one rounding, 2^-8 of the element.
"""
import pytest
import torch

from gpu_helpers import PAD, CANARY, status_ok

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def table_of(rows, P, seed=0):
    g = torch.Generator().manual_seed(seed)
    a = torch.rand(rows, P, generator=g, dtype=torch.float64) * 40 - 20
    a[0] = 0  # position 0 turns nothing
    return torch.stack([a.cos(), a.sin()], -1).float()


def rotation(table, pos, pairs):
    """cos, sin [T, 1, P] in 64 bits."""
    axis = torch.tensor([a for a, n in enumerate(pairs) for _ in range(n)])
    p = pos.long()[:, axis]
    cs = table.double()[p.clamp(min=0), torch.arange(axis.numel())]
    on = p >= 0
    return torch.where(on, cs[..., 0], 1.0)[:, None], torch.where(on, cs[..., 1], 0.0)[:, None]


def rotate(n, cos, sin, interleaved):
    P = cos.shape[-1]
    i, j = (torch.arange(0, 2 * P, 2), torch.arange(1, 2 * P, 2)) if interleaved else \
        (torch.arange(P), torch.arange(P, 2 * P))
    out = n.clone()
    out[..., i] = n[..., i] * cos - n[..., j] * sin
    out[..., j] = n[..., j] * cos + n[..., i] * sin
    return out


def reference(x, w, dy, cos, sin, interleaved, norm, eps):
    """Forward and gradients of one side in 64 bits, with the error scales."""
    x, dy = x.double(), dy.double()
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double()
    g = rotate(dy, cos, -sin, interleaved)
    if not norm:
        y = rotate(x, cos, sin, interleaved)
        return dict(y=y, dx=g, ys=x.abs().amax(-1, keepdim=True),
                    dxs=dy.abs().amax(-1, keepdim=True))
    r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    n = x * r * w
    h, xr = g * w, x * r
    dx = r * (h - xr * (h * xr).mean(-1, keepdim=True))
    return dict(y=rotate(n, cos, sin, interleaved), dx=dx, dw=(g * xr).sum((0, 1)),
                ys=n.abs().amax(-1, keepdim=True),
                dxs=r * (h.abs().amax(-1, keepdim=True)
                         + xr.abs() * (h * xr).abs().mean(-1, keepdim=True)),
                dws=(g * xr).abs().sum((0, 1)))


def close(got, ref, scale, c, name):
    got = got.double().cpu()
    bound = c * U * scale + 1e-37
    if name != "dw" and close.bf16:
        bound = bound + 2.0 ** -8 * ref.abs()
    bad = (got - ref).abs() > bound
    assert not bool(bad.any()), \
        f"{name}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst x" \
        f"{float(((got - ref).abs() / bound).max()):.3g}"


close.bf16 = False


def guarded(shape, stride, dtype):
    """A strided view inside a canary-filled buffer, and a check of what lies
    outside the view."""
    n = 1 + sum((s - 1) * t for s, t in zip(shape, stride))
    es = torch.empty((), dtype=dtype).element_size()
    raw = torch.full((n * es + 2 * PAD,), CANARY, dtype=torch.uint8, device="cuda")
    view = raw[PAD:PAD + n * es].view(dtype).as_strided(shape, stride)

    def check():
        torch.cuda.synchronize()
        keep = torch.ones(n, dtype=torch.bool, device="cuda")
        keep.as_strided(shape, stride).fill_(False)
        inside = raw[PAD:PAD + n * es].view(n, es)[keep]
        assert bool((raw[:PAD] == CANARY).all()) and bool((raw[-PAD:] == CANARY).all())
        assert bool((inside == CANARY).all())
    return view, check


def positions(T, axes, rows, text, seed=0):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, rows, (T, axes), generator=g, dtype=torch.int32)
    p[:text] = -1
    if T > 3:
        p[3, 0] = -1  # one axis alone unrotated
        p[-1] = 0
    return p


def split(P, axes):
    n = [P // axes] * axes
    n[0] += P - sum(n)
    return tuple(n)


CASES = [
    # T, hq, hk, dh, rot, axes, interleaved, dtype, layout
    (256, 4, 4, 32, 32, 3, True, "f32", "dense"),
    (300, 12, 12, 128, 128, 3, True, "bf16", "packed"),
    (300, 12, 4, 128, 128, 3, False, "bf16", "packed"),
    (1, 12, 12, 128, 128, 3, True, "bf16", "dense"),
    (1, 1, 1, 128, 128, 1, False, "f32", "dense"),
    (67, 5, 1, 80, 80, 3, False, "f32", "dense"),
    (67, 5, 2, 80, 80, 3, True, "bf16", "packed"),
    (67, 3, 3, 72, 36, 3, True, "bf16", "dense"),
    (67, 3, 3, 72, 36, 3, False, "bf16", "dense"),
    (67, 3, 3, 72, 72, 2, False, "f32", "packed"),
    (33, 2, 1, 256, 128, 3, False, "bf16", "packed"),
    (33, 2, 1, 256, 256, 3, True, "f32", "packed"),
    (33, 2, 1, 512, 512, 3, True, "bf16", "dense"),
    (33, 2, 1, 512, 200, 3, False, "f32", "dense"),
    (33, 2, 1, 8, 8, 1, True, "bf16", "dense"),
    (33, 2, 1, 2, 2, 1, True, "f32", "dense"),
    (33, 3, 2, 7, 6, 2, True, "bf16", "dense"),
    (33, 3, 2, 37, 20, 4, False, "f32", "odd"),
    (33, 3, 2, 64, 64, 4, True, "bf16", "odd"),
    (33, 3, 2, 64, 64, 3, False, "bf16", "head_major"),
    (257, 17, 0, 64, 64, 3, True, "bf16", "dense"),
    (2000, 3, 1, 64, 48, 3, False, "bf16", "dense"),
    # halves that only 8- or 4-byte vectors fit
    (67, 5, 2, 80, 40, 3, False, "bf16", "packed"),
    (67, 3, 1, 200, 100, 3, False, "bf16", "dense"),
    (67, 3, 1, 40, 36, 3, False, "f32", "dense"),
    (67, 3, 1, 68, 36, 3, False, "bf16", "dense"),
    # many tokens of few heads: several tokens side by side in a warp
    (12001, 3, 1, 64, 64, 3, True, "bf16", "packed"),
    (12001, 8, 1, 32, 32, 3, False, "f32", "dense"),
    (12001, 2, 5, 80, 80, 3, False, "f32", "packed"),
    (12001, 4, 1, 72, 36, 3, False, "bf16", "dense"),
    (12001, 1, 2, 256, 128, 3, True, "bf16", "dense"),
]


def strides(layout, T, h, total, dh):
    if layout == "packed":
        return (total * dh, dh, 1)
    if layout == "odd":  # no vector fits: an odd token stride
        return (h * (dh + 1) + 3, dh + 1, 1)
    if layout == "head_major":
        return (dh, T * dh, 1)
    return (h * dh, dh, 1)


@pytest.mark.parametrize("norm,weights", [(False, False), (True, True), (True, False)])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_against_64_bits(adaln, case, norm, weights):
    T, hq, hk, dh, rot, axes, inter, dt, layout = case
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    close.bf16 = dt == "bf16"
    P, rows, eps = rot // 2, 19, 1e-6
    pairs = split(P, axes)
    table, pos = table_of(rows, P), positions(T, axes, rows, min(2, T // 2))
    cos, sin = rotation(table, pos, pairs)
    g = torch.Generator().manual_seed(5)
    total = hq + 2 * hk + 1
    host, dev, checks = {}, {}, []
    for n, h in (("q", hq), ("k", hk)):
        if h == 0:
            continue
        x = (torch.randn(T, h, dh, generator=g) * 1.5).to(dtype)
        dy = torch.randn(T, h, dh, generator=g).to(dtype)
        x[0, 0] = 0  # a head of zeros
        if T > 5:
            x[5, 0] *= 1e-3  # a head whose mean square is near eps
        w = (1 + 0.3 * torch.randn(dh, generator=g)).to(dtype) if weights else None
        host[n] = (x, dy, w)
        st = strides(layout, T, h, total, dh)
        views = {}
        for k, src in (("x", x), ("dy", dy), ("out", None), ("dx", None)):
            views[k], chk = guarded((T, h, dh), st, dtype)
            checks.append(chk)
            if src is not None:
                views[k].copy_(src)
        views["w"] = None if w is None else w.cuda()
        dev[n] = views
    tb, ps = table.cuda(), pos.cuda()
    both = lambda k: tuple(dev[n][k] if n in dev else None for n in ("q", "k"))  # noqa: E731
    q, k = both("x")
    qo, ko = both("out")
    dyq, dyk = both("dy")
    dq, dk = both("dx")
    wq, wk = both("w")
    how = dict(axis_pairs=pairs, interleaved=inter, norm=norm, wq=wq, wk=wk, eps=eps)
    adaln.adaln_qk_rope_fwd(q, k, tb, ps, q_out=qo, k_out=ko, **how)
    back = dict(how, q=q, k=k) if norm else how
    _, _, dwq, dwk = adaln.adaln_qk_rope_bwd(dyq, dyk, tb, ps, dq=dq, dk=dk, **back)
    for c in checks:
        c()
    status_ok()
    for n, dw in (("q", dwq), ("k", dwk)):
        if n not in host:
            continue
        x, dy, w = host[n]
        ref = reference(x, w, dy, cos, sin, inter, norm, eps)
        close(dev[n]["out"], ref["y"], ref["ys"], 64, n + " out")
        close(dev[n]["dx"], ref["dx"], ref["dxs"], 128, "d" + n)
        if norm:
            close(dw, ref["dw"], ref["dws"], 80 if T < 10000 else 144, "dw")


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dh", [64, 36])
def test_in_place_gives_the_same_bits(adaln, dt, dh):
    T, h, rows, pairs = 300, 5, 11, (dh // 2,)
    q = torch.randn(T, h, dh, device="cuda").to(dt)
    w = torch.randn(dh, device="cuda").to(dt)
    tb, ps = table_of(rows, dh // 2).cuda(), positions(T, 1, rows, 2).cuda()
    how = dict(axis_pairs=pairs, interleaved=False, norm=True, wq=w)
    out, _ = adaln.adaln_qk_rope_fwd(q, None, tb, ps, **how)
    dy = torch.randn_like(q)
    dq, _, dw, _ = adaln.adaln_qk_rope_bwd(dy, None, tb, ps, q=q, **how)
    a = q.clone()
    adaln.adaln_qk_rope_fwd(a, None, tb, ps, q_out=a, **how)
    assert torch.equal(a, out)
    b = dy.clone()
    _, _, dw2, _ = adaln.adaln_qk_rope_bwd(b, None, tb, ps, q=q, dq=b, **how)
    assert torch.equal(b, dq) and torch.equal(dw, dw2)


def test_unrotated_elements_pass_exactly(adaln):
    """Infinities and NaN stay in their own element where nothing turns them:
    a text token, position 0 and the elements past the rotated ones."""
    for dt, dh, rot in ((torch.bfloat16, 64, 32), (torch.float32, 37, 20)):
        for inter in (True, False):
            q = torch.randn(4, 2, dh, device="cuda").to(dt)
            q[0, 0, 1] = float("inf")
            q[1, 1, 0] = float("nan")
            q[2, 0, rot:] = torch.finfo(dt).min
            q[2, 0, rot + 1] = float("inf")
            ps = torch.tensor([[-1], [0], [3], [4]], dtype=torch.int32, device="cuda")
            out, _ = adaln.adaln_qk_rope_fwd(q, None, table_of(9, rot // 2).cuda(), ps,
                                             axis_pairs=(rot // 2,), interleaved=inter)
            assert torch.equal(out[:2].isnan(), q[:2].isnan())
            assert torch.equal(out[:2].nan_to_num(7.0), q[:2].nan_to_num(7.0))
            assert torch.equal(out[2:, :, rot:], q[2:, :, rot:])
            assert bool(out[2:, :, :rot].isfinite().all())
    status_ok()


def test_positions_outside_the_table_are_recorded(adaln):
    q = torch.randn(40, 2, 64, device="cuda")
    tb = table_of(6, 32).cuda()
    ps = torch.zeros(40, 1, dtype=torch.int32, device="cuda") + 2
    want, _ = adaln.adaln_qk_rope_fwd(q, None, tb, ps, axis_pairs=(32,))
    status_ok()
    many = torch.zeros(12000, 1, dtype=torch.int32, device="cuda")  # several tokens to a warp
    many[7001] = 6
    adaln.adaln_qk_rope_fwd(torch.randn(12000, 1, 64, device="cuda"), None, tb, many, axis_pairs=(32,))
    assert adaln.adaln_get_status() == (adaln.ADALN_ERR_POS, adaln.ADALN_DEV_POS_RANGE)
    for bad in (6, -2, 2 ** 31 - 1, -2 ** 31):
        ps[17] = bad
        out, _ = adaln.adaln_qk_rope_fwd(q, None, tb, ps, axis_pairs=(32,))
        rc, bits = adaln.adaln_get_status()
        assert rc == adaln.ADALN_ERR_POS and bits == adaln.ADALN_DEV_POS_RANGE
        assert torch.equal(out[17], q[17])
        assert torch.equal(out[:17], want[:17]) and torch.equal(out[18:], want[18:])
    status_ok()


def test_no_tokens(adaln):
    q = torch.empty(0, 4, 64, device="cuda", dtype=torch.bfloat16)
    tb, ps = table_of(3, 32).cuda(), torch.empty(0, 1, dtype=torch.int32, device="cuda")
    out, kout = adaln.adaln_qk_rope_fwd(q, q, tb, ps, axis_pairs=(32,), norm=True)
    assert out.shape == q.shape and kout.shape == q.shape
    dq, dk, dwq, dwk = adaln.adaln_qk_rope_bwd(q, q, tb, ps, axis_pairs=(32,), norm=True, q=q, k=q,
                                               dwq=torch.ones(64, device="cuda"))
    assert not dwq.any() and not dwk.any()
    status_ok()


def test_gradients_against_differences(adaln):
    """Directional differences of the kernel's own forward.  The loss is summed
    in 64 bits; the step of 2^-6 leaves a truncation error of about 2^-12 of
    the third derivative and a rounding error of about U 2^6 of the loss's
    terms: 1e-3 of the sum of |terms| holds both."""
    T, hq, hk, dh = 19, 3, 2, 40
    pairs = (8, 6, 6)
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x = {"q": r(T, hq, dh), "k": r(T, hk, dh), "wq": 1 + 0.2 * r(dh), "wk": 1 + 0.2 * r(dh)}
    dy = (r(T, hq, dh), r(T, hk, dh))
    tb, ps = table_of(9, 20).cuda(), positions(T, 3, 9, 1).cuda()
    for inter in (True, False):
        def loss(v):
            o = adaln.adaln_qk_rope_fwd(v["q"], v["k"], tb, ps, pairs, inter, True, v["wq"], v["wk"])
            return sum((a.double() * b.double()).sum() for a, b in zip(o, dy))

        grads = dict(zip(("q", "k", "wq", "wk"), adaln.adaln_qk_rope_bwd(
            *dy, tb, ps, pairs, inter, True, q=x["q"], k=x["k"], wq=x["wq"], wk=x["wk"])))
        for n in x:
            d = torch.randn(x[n].shape, device="cuda", generator=g)
            h = 2.0 ** -6
            up, down = (loss(dict(x, **{n: x[n] + s * d})) for s in (h, -h))
            terms = (grads[n].double() * d.double())
            assert abs(float((up - down) / (2 * h) - terms.sum())) <= 1e-3 * float(terms.abs().sum())


def test_weight_gradients_are_reproducible_over_streams(adaln):
    T, h, dh = 5000, 12, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(T, h, dh, device="cuda", generator=g).bfloat16()
    dy = torch.randn(T, h, dh, device="cuda", generator=g).bfloat16()
    tb, ps = table_of(50, 64).cuda(), positions(T, 3, 50, 7).cuda()
    how = dict(axis_pairs=(22, 21, 21), norm=True)
    first = adaln.adaln_qk_rope_bwd(dy, dy, tb, ps, q=q, k=q, **how)
    assert torch.equal(first[2], first[3])  # both sides sum in the same order
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.full((adaln.adaln_qk_rope_bwd_workspace_size(T, h, h, dh, torch.bfloat16),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    for _ in range(3):
        with torch.cuda.stream(s):
            again = adaln.adaln_qk_rope_bwd(dy, dy, tb, ps, q=q, k=q, workspace=ws, **how)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_offsets_past_32_bits(adaln):
    """Two tokens more than 2^32 bytes apart."""
    dh, far = 64, (1 << 31) + 64
    if torch.cuda.mem_get_info()[0] < 6 << 30:
        pytest.fail("needs 6 GB of device memory")
    buf = torch.empty(far + dh, dtype=torch.bfloat16, device="cuda")
    q = buf.as_strided((2, 1, dh), (far, dh, 1))
    q.copy_(torch.randn(2, 1, dh))
    tb = table_of(6, 32).cuda()
    ps = torch.tensor([[4], [5]], dtype=torch.int32, device="cuda")
    dense, _ = adaln.adaln_qk_rope_fwd(q.contiguous(), None, tb, ps, axis_pairs=(32,))
    adaln.adaln_qk_rope_fwd(q, None, tb, ps, axis_pairs=(32,), q_out=q)
    assert torch.equal(q, dense)


def test_trace_counts_the_launches(adaln):
    q = torch.randn(8, 2, 64, device="cuda")
    tb, ps = table_of(6, 32).cuda(), positions(8, 1, 6, 0).cuda()
    adaln.adaln_trace_begin(8)
    adaln.adaln_qk_rope_fwd(q, None, tb, ps, axis_pairs=(32,))
    adaln.adaln_qk_rope_bwd(q, None, tb, ps, axis_pairs=(32,), norm=True, q=q)
    adaln.adaln_trace_end()
    assert adaln.adaln_trace_get(adaln.ADALN_KERNEL_QK_ROPE)[0] == 3
    assert adaln.adaln_trace_get(adaln.ADALN_KERNEL_FWD)[0] == 0


def test_binding_refuses(adaln):
    q = torch.randn(8, 2, 64, device="cuda")
    tb, ps = table_of(6, 32).cuda(), positions(8, 1, 6, 0).cuda()
    f = adaln.adaln_qk_rope_fwd
    with pytest.raises(ValueError):
        f(q[:, :, ::2], None, tb, ps, axis_pairs=(32,))
    with pytest.raises(ValueError):
        f(q, None, tb, ps, axis_pairs=(31,))
    with pytest.raises(ValueError):
        f(q, None, tb, ps[:7], axis_pairs=(32,))
    with pytest.raises(ValueError):
        f(q, q[:7], tb, ps, axis_pairs=(32,))
    with pytest.raises(TypeError):
        f(q, None, tb, ps, axis_pairs=(32,), norm=True, wq=torch.ones(64, device="cuda").bfloat16())
    with pytest.raises(TypeError):
        f(q.half(), None, tb, ps, axis_pairs=(32,))
    with pytest.raises(ValueError):
        f(q, None, tb.cpu(), ps, axis_pairs=(32,))
    with pytest.raises(adaln.AdalnError):
        f(q, None, tb, ps, axis_pairs=(32,), norm=True, eps=-1.0)
    with pytest.raises(ValueError):
        adaln.adaln_qk_rope_bwd(q, None, tb, ps, axis_pairs=(32,), norm=True)
    with pytest.raises(adaln.AdalnError) as e:
        adaln.adaln_qk_rope_bwd(q, None, tb, ps, axis_pairs=(32,), norm=True, q=q,
                                workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == adaln.ADALN_ERR_WORKSPACE


@pytest.mark.parametrize("dh,rot", [(64, 64), (80, 40), (37, 20), (200, 100)])
def test_heads_of_tiny_values_without_eps(adaln, dh, rot):
    """eps = 0 and heads of rms 1e-17 to 1e-9: r^3 passes the largest fp32 where the
    gradients, of order r, do not.  The squares of the smallest are still normal."""
    T, h, axes, inter = 40, 4, 2, dh % 3 == 1
    close.bf16 = False
    pairs, rows = split(rot // 2, axes), 9
    table, pos = table_of(rows, rot // 2), positions(T, axes, rows, 2)
    cos, sin = rotation(table, pos, pairs)
    g = torch.Generator().manual_seed(dh)
    rms = torch.tensor([1e-17, 1e-13, 1e-11, 1e-9])[:, None]
    x, dy = torch.randn(T, h, dh, generator=g) * rms, torch.randn(T, h, dh, generator=g)
    w = 1 + 0.3 * torch.randn(dh, generator=g)
    how = dict(axis_pairs=pairs, interleaved=inter, norm=True, wq=w.cuda(), eps=0.0)
    tb, ps = table.cuda(), pos.cuda()
    out, _ = adaln.adaln_qk_rope_fwd(x.cuda(), None, tb, ps, **how)
    dq, _, dw, _ = adaln.adaln_qk_rope_bwd(dy.cuda(), None, tb, ps, q=x.cuda(), **how)
    ref = reference(x, w, dy, cos, sin, inter, True, 0.0)
    close(out, ref["y"], ref["ys"], 64, "out")
    close(dq, ref["dx"], ref["dxs"], 128, "dq")
    close(dw, ref["dw"], ref["dws"], 80, "dw")
    status_ok()


@pytest.mark.parametrize("dt,dh,hk", [(torch.bfloat16, 128, 2), (torch.bfloat16, 72, 2),
                                      (torch.float32, 64, 1), (torch.float32, 80, 3)])
@pytest.mark.parametrize("T", [40, 6000])
def test_weights_at_element_alignment_take_the_same_path(adaln, dt, dh, hk, T):
    """Weights in the middle of a flat parameter buffer: the same bits as aligned
    ones (the scalar path would round in another order)."""
    g = torch.Generator(device="cuda").manual_seed(T + dh)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g).to(dt)  # noqa: E731
    q, k, dq, dk = r(T, 3, dh), r(T, hk, dh), r(T, 3, dh), r(T, hk, dh)
    flat = r(2 * dh + 1)
    wq, wk = flat[1:dh + 1], flat[dh + 1:]
    assert wq.data_ptr() % 16 and wk.data_ptr() % flat.element_size() == 0
    tb, ps = table_of(9, dh // 2).cuda(), positions(T, 3, 9, 2).cuda()
    for inter in (True, False):
        got, want = ([*adaln.adaln_qk_rope_fwd(q, k, tb, ps, split(dh // 2, 3), inter, True, *w),
                      *adaln.adaln_qk_rope_bwd(dq, dk, tb, ps, split(dh // 2, 3), inter, True, q, k, *w)]
                     for w in ((wq, wk), (wq.clone(), wk.clone())))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    status_ok()
