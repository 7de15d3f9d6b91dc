"""Dropout with the gate and the residual of a branch (adaln_dropout_*) against the
definition in 64 bits, its mask made by a plain generator of the tests' own.

Tolerances, with u = 2^-24 (fp32) and r = 2^-8 (bf16 outputs) or u (fp32 ones): y is
x + g (f h) in three fp32 roundings and the output's, f itself rounded once, so

  |error| <= r |y| + 4 u (|x| + |g f h|)

and dh = g (f dy) likewise with 3 u; dgate is an fp32 sum of n products f dy h, each
rounded twice and then added, in some order: (n + 3) u sum |terms|.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import check_guards, guarded_empty, status_ok
from philox import kept

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def segments(T, nseg, seed=0):
    """Non-decreasing segment ids, some segments empty."""
    g = np.random.default_rng(seed)
    return torch.from_numpy(np.sort(g.integers(0, nseg, T)).astype(np.int32)).cuda()


def inputs(T, D, nseg, dt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g).to(dt)  # noqa: E731
    return r(T, D), r(T, D), r(nseg, D), segments(T, nseg, seed), r(T, D)


def mask(T, D, p, rng):
    keep, factor = kept(np.arange(T), D, p, *rng)
    return torch.from_numpy(keep).cuda(), factor


def close(got, ref, terms, dt, steps, name):
    bound = (2.0 ** -8 if dt == BF16 else U) * ref.abs() + steps * U * terms + 1e-40
    err = (got.double() - ref).abs()
    assert not bool((err > bound).any()), f"{name}: worst x{float((err / bound).max()):.3g}"


def call(L, h, x, gate, seg, dy, p, rng):
    """Forward and backward, every buffer inside guard bands, poisoned."""
    guards, out = {}, {}
    for k in ("y", "dh"):
        guards[k], out[k] = guarded_empty(h.shape, h.dtype)
    if gate is not None:
        guards["dgate"], out["dgate"] = guarded_empty(gate.shape, F32)
        guards["ws"], out["ws"] = guarded_empty(
            (L.adaln_dropout_bwd_workspace_size(*h.shape, len(gate), h.dtype),), torch.uint8)
        out["ws"].fill_(0xFF)
    L.adaln_dropout_fwd(h, p, rng, x=x, gate=gate, seg_id=seg, y=out["y"])
    L.adaln_dropout_bwd(dy, p, rng, h=h if gate is not None else None, gate=gate, seg_id=seg, dh=out["dh"],
                        dgate=out.get("dgate"), workspace=out.get("ws"))
    check_guards(guards)
    status_ok()
    return out


def against(out, h, x, gate, seg, dy, p, rng):
    dt = h.dtype
    keep, f = mask(*h.shape, p, rng)
    m = keep.double() * f
    b = seg.long() if seg is not None else None
    g = gate.double()[b] if gate is not None else 1.0
    k = g * m * h.double()
    ref, terms = (k, k.abs()) if x is None else (k + x.double(), k.abs() + x.double().abs())
    close(out["y"], ref, terms, dt, 4, "y")
    dh = g * m * dy.double()
    close(out["dh"], dh, dh.abs(), dt, 3, "dh")
    if gate is not None:
        each = m * dy.double() * h.double()
        ref = torch.zeros(gate.shape, dtype=torch.float64, device="cuda")
        n = torch.bincount(b, minlength=len(gate))[:, None]
        close(out["dgate"], ref.index_add(0, b, each),
              (n + 3) * torch.zeros_like(ref).index_add(0, b, each.abs()), F32, 1, "dgate")
        assert not bool(out["dgate"][n[:, 0] == 0].any())
    return keep


SHAPES = [(1, 8, 1), (1, 128, 3), (2, 24, 1), (3, 1000, 2), (4, 64, 9), (5, 512, 1), (17, 2056, 4),
          (63, 5120, 2), (64, 72, 64), (301, 1000, 37), (1023, 1536, 5), (4099, 264, 700),
          (9001, 64, 1), (20011, 8, 3), (700, 13824, 2)]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_against_64_bits(adaln, shape, dt):
    T, D, nseg = shape
    p, rng = (0.1, 0.5, 0.9)[(T + D) % 3], (T * 977 + (D << 40), (1 << 62) - D)
    h, x, gate, seg, dy = inputs(T, D, nseg, dt, seed=T)
    against(call(adaln, h, x, gate, seg, dy, p, rng), h, x, gate, seg, dy, p, rng)
    against(call(adaln, h, None, None, None, dy, p, rng), h, None, None, None, dy, p, rng)
    against(call(adaln, h, x, None, None, dy, p, rng), h, x, None, None, dy, p, rng)
    against(call(adaln, h, None, gate, seg, dy, p, rng), h, None, gate, seg, dy, p, rng)


@pytest.mark.parametrize("D", [4, 12, 1004])
def test_fp32_rows_that_end_inside_a_group(adaln, D):
    h, x, gate, seg, dy = inputs(57, D, 4, F32, seed=D)
    against(call(adaln, h, x, gate, seg, dy, 0.25, (3, 4)), h, x, gate, seg, dy, 0.25, (3, 4))


@pytest.mark.parametrize("p", [0.0, 2.0 ** -18, 2.0 ** -17, 1 - 2.0 ** -17, 1 - 2.0 ** -16, 1.0])
def test_the_ends_of_p(adaln, p):
    """Nothing, one in 65536, all but one and all of the elements dropped (p is taken to
    the next multiple of 2^-16, halves upwards)."""
    h, x, gate, seg, dy = inputs(400, 1024, 3, F32, seed=1)
    keep = against(call(adaln, h, x, gate, seg, dy, p, (1, 0)), h, x, gate, seg, dy, p, (1, 0))
    if p in (0.0, 2.0 ** -18, 1 - 2.0 ** -17, 1.0):
        assert bool((keep == (p < 0.5)).all())
        for rng in (None, (7, 8)):
            assert torch.equal(adaln.adaln_dropout_fwd(h, p, rng, x=x, gate=gate, seg_id=seg),
                               adaln.adaln_dropout_fwd(h, p, (1, 0), x=x, gate=gate, seg_id=seg))
    else:
        assert bool(keep.any()) and not bool(keep.all())


def test_the_mask_depends_on_seed_offset_and_place_alone(adaln):
    """Across element types, row counts, the forward and the backward; and any of the
    128 bits of (seed, offset) changes it."""
    one = torch.ones(300, 512, device="cuda")
    base = adaln.adaln_dropout_fwd(one, 0.5, (5, 6))
    assert torch.equal(base, adaln.adaln_dropout_fwd(one.bfloat16(), 0.5, (5, 6)).float())
    assert torch.equal(base[:7], adaln.adaln_dropout_fwd(one[:7], 0.5, (5, 6)))
    assert torch.equal(base, adaln.adaln_dropout_bwd(one, 0.5, (5, 6))[0])
    state = torch.tensor([5, 6], device="cuda")
    assert torch.equal(base, adaln.adaln_dropout_fwd(one, 0.5, state))
    for bit in range(64):
        for rng in ((5 ^ 1 << bit, 6), (5, 6 ^ 1 << bit)):
            other = adaln.adaln_dropout_fwd(one, 0.5, rng)
            # (153,600 places, each equal with probability 1/2: ten deviations)
            assert abs(float((other == base).float().mean()) - 0.5) < 0.013
    signed = torch.tensor([-1, -2], device="cuda")
    assert torch.equal(adaln.adaln_dropout_fwd(one, 0.5, signed),
                       adaln.adaln_dropout_fwd(one, 0.5, (2 ** 64 - 1, -2)))


@pytest.mark.parametrize("dt", [F32, BF16])
def test_a_dropped_element_takes_nothing(adaln, dt):
    """Infinities and NaN in h, dy and the gate where the mask drops; what is kept
    takes them by the formula."""
    T, D = 40, 256
    h, x, gate, seg, dy = inputs(T, D, 2, dt, seed=3)
    keep, f = mask(T, D, 0.5, (9, 9))
    clean = call(adaln, h, x, gate, seg, dy, 0.5, (9, 9))
    for bad in (float("inf"), float("nan"), torch.finfo(dt).min):
        h2, dy2 = (torch.where(keep, t, torch.full_like(t, bad)) for t in (h, dy))
        out = call(adaln, h2, x, gate, seg, dy2, 0.5, (9, 9))
        for k in ("y", "dh", "dgate"):
            assert torch.equal(out[k], clean[k]), (bad, k)
        gate2 = gate.clone()
        gate2[:, 7] = bad
        y = adaln.adaln_dropout_fwd(h, 0.5, (9, 9), x=x, gate=gate2, seg_id=seg)
        assert torch.equal(y[:, 7][~keep[:, 7]], x[:, 7][~keep[:, 7]])
        if bad != bad or bad == float("inf"):
            assert not bool(y[:, 7][keep[:, 7]].isfinite().any())
    zero = torch.zeros_like(h)  # a kept zero times an infinite gate is no number
    gate[:] = float("inf")
    y = adaln.adaln_dropout_fwd(zero, 0.5, (9, 9), gate=gate, seg_id=seg)
    assert torch.equal(y.isnan(), keep) and not bool(y[~keep].any())


@pytest.mark.parametrize("dt", [F32, BF16])
def test_in_place_gives_the_same_bits(adaln, dt):
    h, x, gate, seg, dy = inputs(777, 520, 6, dt, seed=5)
    how = dict(gate=gate, seg_id=seg)
    want = call(adaln, h, x, gate, seg, dy, 0.3, (1, 1))
    for which in range(2):
        a = [h.clone(), x.clone()]
        adaln.adaln_dropout_fwd(a[0], 0.3, (1, 1), x=a[1], y=a[which], **how)
        assert torch.equal(a[which], want["y"])
        a = [dy.clone(), h.clone()]
        _, dgate = adaln.adaln_dropout_bwd(a[0], 0.3, (1, 1), h=a[1], dh=a[which], **how)
        assert torch.equal(a[which], want["dh"]) and torch.equal(dgate, want["dgate"])


def test_no_tokens(adaln):
    h = torch.empty(0, 64, device="cuda")
    gate, seg = torch.ones(3, 64, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    assert adaln.adaln_dropout_fwd(h, 0.1, (1, 2), x=h, gate=gate, seg_id=seg).shape == (0, 64)
    dh, dgate = adaln.adaln_dropout_bwd(h, 0.1, (1, 2), h=h, gate=gate, seg_id=seg,
                                        dgate=torch.ones(3, 64, device="cuda"))
    assert dh.shape == (0, 64) and not bool(dgate.any())
    status_ok()


def test_bad_segments_are_recorded(adaln):
    h, x, gate, seg, dy = inputs(500, 64, 5, F32)
    for at, bad, bit in ((17, 5, adaln.ADALN_DEV_SEG_RANGE), (499, 2 ** 31 - 1, adaln.ADALN_DEV_SEG_RANGE),
                         (0, -1, adaln.ADALN_DEV_SEG_RANGE), (300, 0, adaln.ADALN_DEV_SEG_ORDER)):
        s = seg.clone()
        s[at] = bad
        for back in (False, True):
            if back:
                adaln.adaln_dropout_bwd(dy, 0.1, (1, 2), h=h, gate=gate, seg_id=s)
            else:
                adaln.adaln_dropout_fwd(h, 0.1, (1, 2), x=x, gate=gate, seg_id=s)
            rc, bits = adaln.adaln_get_status()
            assert rc == adaln.ADALN_ERR_SEG and bits & bit, (at, bad, back)
    status_ok()


def test_reproducible_over_streams_and_workspaces(adaln):
    h, x, gate, seg, dy = inputs(5003, 1000, 37, BF16, seed=2)
    first = call(adaln, h, x, gate, seg, dy, 0.2, (3, 1))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(s):
            y = adaln.adaln_dropout_fwd(h, 0.2, (3, 1), x=x, gate=gate, seg_id=seg)
            dh, dgate = adaln.adaln_dropout_bwd(dy, 0.2, (3, 1), h=h, gate=gate, seg_id=seg)
        torch.cuda.synchronize()
        assert all(torch.equal(a, first[k]) for a, k in ((y, "y"), (dh, "dh"), (dgate, "dgate")))


def test_in_a_cuda_graph_with_a_new_mask_each_replay(adaln):
    h, x, gate, seg, dy = inputs(300, 256, 4, BF16, seed=6)
    state = torch.tensor([11, 0], device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = adaln.adaln_dropout_fwd(h, 0.4, state, x=x, gate=gate, seg_id=seg)
        dh, dgate = adaln.adaln_dropout_bwd(dy, 0.4, state, h=h, gate=gate, seg_id=seg)
    for step in range(3):
        state[1] = step
        graph.replay()
        torch.cuda.synchronize()
        want = call(adaln, h, x, gate, seg, dy, 0.4, (11, step))
        assert all(torch.equal(a, want[k]) for a, k in ((y, "y"), (dh, "dh"), (dgate, "dgate")))


def test_offsets_past_32_bits(adaln):
    """More than 2^32 bytes and 2^31 elements: rows around the 2^31st element and at
    both ends, and the whole gradient of a gate."""
    T, D = 70000, 32768
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.fail("needs 40 GB of device memory")
    g = torch.Generator(device="cuda").manual_seed(0)
    h = torch.randn(T, D, device="cuda", generator=g, dtype=BF16)
    gate, seg = torch.randn(2, D, device="cuda", generator=g).bfloat16(), segments(T, 2)
    y = adaln.adaln_dropout_fwd(h, 0.2, (1, 2), x=h, gate=gate, seg_id=seg)
    dh, dgate = adaln.adaln_dropout_bwd(h, 0.2, (1, 2), h=h, gate=gate, seg_id=seg)
    at = (1 << 31) // D
    rows = np.array([0, 1, at - 1, at, at + 1, T - 2, T - 1])
    keep, f = kept(rows, D, 0.2, 1, 2)
    m, rows = torch.from_numpy(keep).cuda().double() * f, torch.from_numpy(rows).cuda()
    k = gate.double()[seg[rows].long()] * m * h[rows].double()
    close(dh[rows], k, k.abs(), BF16, 3, "dh")
    close(y[rows], h[rows].double() + k, h[rows].double().abs() + k.abs(), BF16, 4, "y")
    # f h^2 summed over some 35000 rows, of which 0.8 are kept: its mean is n, its
    # deviation sqrt(n (3 / 0.8 - 1)), and 65536 columns stay within six of them.
    n = torch.bincount(seg.long(), minlength=2).double()[:, None]
    assert bool(((dgate.double() - n).abs() < 6 * (n * 2.75).sqrt() + 1e-3 * n).all())
    status_ok()


def test_gradients_against_differences(adaln):
    """Directional differences of the kernel's own forward (linear in each argument,
    so only rounding is left: 1e-3 of the sum of |terms|)."""
    h, x, gate, seg, dy = inputs(50, 40, 3, F32, seed=8)
    v = dict(h=h, x=x, gate=gate)
    dh, dgate = adaln.adaln_dropout_bwd(dy, 0.3, (2, 2), h=h, gate=gate, seg_id=seg)

    def loss(a):
        y = adaln.adaln_dropout_fwd(a["h"], 0.3, (2, 2), x=a["x"], gate=a["gate"], seg_id=seg)
        return (y.double() * dy.double()).sum()

    for name, grad in (("h", dh), ("x", dy), ("gate", dgate)):
        d = torch.randn_like(v[name])
        slope = (loss(dict(v, **{name: v[name] + d})) - loss(dict(v, **{name: v[name] - d}))) / 2
        terms = grad.double() * d.double()
        assert abs(float(slope - terms.sum())) <= 1e-3 * float(terms.abs().sum()), name


def test_nodes(adaln):
    """The nodes equal the calls; masks drawn from torch's generator follow its seed,
    and a recomputation by torch's checkpointing draws the same ones."""
    from torch.utils.checkpoint import checkpoint

    from adaln_video_dit_gb300.autograd import GatedResidual, dropout, gated_residual
    h, x, gate, seg, dy = inputs(6, 64, 2, F32, seed=4)
    leaves = [t.view(2, 3, 64).clone().requires_grad_() for t in (x, h)] + [gate.clone().requires_grad_()]
    y = gated_residual(*leaves, seg, 0.3, (5, 5))
    y.backward(dy.view(2, 3, 64))
    want = call(adaln, h, x, gate, seg, dy, 0.3, (5, 5))
    assert torch.equal(y.detach().view(6, 64), want["y"])
    for t, k in zip(leaves, (dy, want["dh"], want["dgate"])):
        assert torch.equal(t.grad.view(k.shape), k)
    m, x, h = GatedResidual(0.5), leaves[0], leaves[1]
    torch.manual_seed(3)
    a = m(x, h, leaves[2], seg)
    b = m(x, h, leaves[2], seg)
    torch.manual_seed(3)
    assert torch.equal(a, m(x, h, leaves[2], seg)) and not torch.equal(a, b)
    grads = []
    for again in (False, True):
        torch.manual_seed(7)
        f = lambda v: m(x, v * 2, leaves[2], seg)  # noqa: E731
        out = checkpoint(f, h, use_reentrant=False) if again else f(h)
        grads.append(torch.autograd.grad(out.square().sum(), h)[0])
    assert torch.equal(*grads)
    assert torch.equal(m.eval()(x, h, leaves[2], seg), gated_residual(x, h, leaves[2], seg))
    assert torch.equal(dropout(h, 0.0), h)


def test_each_gradient_has_its_inputs_shape(adaln):
    from adaln_video_dit_gb300.autograd import gated_residual
    h, x, gate, seg, dy = inputs(6, 64, 2, F32, seed=5)
    shapes = ((6, 64), (1, 6, 64), (2, 3, 64))
    for hs in shapes:
        for xs in shapes:
            leaves = [x.view(xs).clone().requires_grad_(), h.view(hs).clone().requires_grad_()]
            gated_residual(*leaves, gate, seg, 0.3, (5, 5)).backward(dy.view(hs))
            assert leaves[0].grad.shape == xs and leaves[1].grad.shape == hs
            assert torch.equal(leaves[0].grad.view(6, 64), dy)


def test_trace_counts_the_launches(adaln):
    h, x, gate, seg, dy = inputs(9, 64, 2, F32)
    adaln.adaln_trace_begin(8)
    adaln.adaln_dropout_fwd(h, 0.1, (1, 2))
    adaln.adaln_dropout_bwd(dy, 0.1, (1, 2), h=h, gate=gate, seg_id=seg)
    adaln.adaln_trace_end()
    assert adaln.adaln_trace_get(adaln.ADALN_KERNEL_DROPOUT)[0] == 3
    assert adaln.adaln_trace_get(adaln.ADALN_KERNEL_FWD)[0] == 0


def test_binding_refuses(adaln):
    h, x, gate, seg, dy = inputs(8, 64, 2, F32)
    f, b = adaln.adaln_dropout_fwd, adaln.adaln_dropout_bwd
    for bad in (dict(x=x[:7]), dict(gate=gate), dict(seg_id=seg), dict(gate=gate[:, :32], seg_id=seg),
                dict(gate=gate, seg_id=seg[:7]), dict(x=x.cpu()), dict(rng=(1, 2, 3)),
                dict(rng=torch.zeros(3, dtype=torch.int64, device="cuda")), dict(rng=torch.zeros(2).long())):
        with pytest.raises(ValueError):
            f(h, 0.1, **{"rng": (1, 2), **bad})
    for bad in (dict(x=x.bfloat16()), dict(gate=gate.bfloat16(), seg_id=seg), dict(gate=gate, seg_id=seg.long()),
                dict(rng=torch.zeros(2, device="cuda")), dict(rng=(1.5, 2))):
        with pytest.raises(TypeError):
            f(h, 0.1, **{"rng": (1, 2), **bad})
    with pytest.raises(ValueError):
        f(h.t(), 0.1, (1, 2))
    with pytest.raises(TypeError):
        f(h.half(), 0.1, (1, 2))
    for bad in (dict(p=1.1), dict(p=-1.0), dict(p=0.1, rng=None)):
        with pytest.raises(adaln.AdalnError):
            f(h, **{"rng": (1, 2), **bad})
    with pytest.raises(ValueError):
        b(dy, 0.1, (1, 2), h=h)
    with pytest.raises(adaln.AdalnError) as e:
        b(dy, 0.1, (1, 2), h=h, gate=gate, seg_id=seg,
          workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == adaln.ADALN_ERR_WORKSPACE


@pytest.mark.parametrize("where", ["first", "last", "amid"])
def test_one_long_segment_among_many_short_ones(adaln, where):
    """Nearly all tokens in one of 300 segments, the others with one, two or none."""
    T, D, nseg = 30011, 264, 300
    h, x, gate, _, dy = inputs(T, D, nseg, BF16, seed=11)
    at = {"first": 0, "last": nseg - 1, "amid": 140}[where]
    n = np.arange(nseg) % 3
    n[at] = 0
    n[at] = T - n.sum()
    seg = torch.from_numpy(np.repeat(np.arange(nseg), n).astype(np.int32)).cuda()
    against(call(adaln, h, x, gate, seg, dy, 0.1, (5, 6)), h, x, gate, seg, dy, 0.1, (5, 6))
