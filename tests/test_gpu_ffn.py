"""The gated feed-forward block (adaln_ffn_*) against the definition in 64 bits.

Tolerances, from the arithmetic: an output is rounded to bf16 once (2^-8 of the
element at most), and it sums products of which one factor (h, or dg and du)
was rounded to bf16 once, so

  |error| <= 2^-8 |ref| + (2^-8 + K 2^-23 + c) sum |rounded factor| |other|

with K 2^-23 for an fp32 sum of K terms and, in c, what the rounded factor
carries from its own fp32 sums (K 2^-23 of their absolute terms) and from the
activation (at most 2^-15 from 24-bit g and u, and as much from the fast
exponential).  Roundings are independent, so over a tensor of many elements the
2-norm of the error is at most sqrt(2) 2^-8 / sqrt(3) of the result's: 4e-3
holds that with a margin of a fifth.
"""
import math

import pytest
import torch

from gpu_helpers import check_guards, guarded_empty, status_ok

pytestmark = pytest.mark.gpu
ACTS = ("silu", "gelu_tanh", "gelu")


def act_of(act, g):
    """act(g) and act'(g) in 64 bits."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        p = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    s = torch.sigmoid(2 * k * (g + 0.044715 * g ** 3))
    return g * s, s + g * s * (1 - s) * 2 * k * (1 + 3 * 0.044715 * g * g)


def inputs(T, D, F, seed=0, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return ((gain * r(T, D)).bfloat16(), (r(F, D) / math.sqrt(D)).bfloat16(),
            (r(F, D) / math.sqrt(D)).bfloat16(), (r(D, F) / math.sqrt(F)).bfloat16(),
            (0.1 * r(T, D)).bfloat16())


def reference(x, wg, wu, wd, dy, act):
    """{name: (value, bound)} in 64 bits."""
    x, wg, wu, wd, dy = (t.double() for t in (x, wg, wu, wd, dy))
    (T, D), F = x.shape, wg.shape[0]
    u23, c = 2.0 ** -23, 2.0 ** -14
    g, u = x @ wg.t(), x @ wu.t()
    eg, eu = D * u23 * (x.abs() @ wg.abs().t()), D * u23 * (x.abs() @ wu.abs().t())
    a, da = act_of(act, g)
    h = a * u
    # |act'| and |act''| are below 1.2, so the error of g enters by at most that
    eh = 1.2 * eg * u.abs() + (a.abs() + 1.2 * eg) * eu + (2.0 ** -8 + c) * h.abs()
    dh = dy @ wd
    edh = D * u23 * (dy.abs() @ wd.abs())
    dg, du = dh * u * da, dh * a
    edg = (edh * (u * da).abs() + dh.abs() * (1.2 * eu + 1.2 * eg * u.abs())
           + (2.0 ** -8 + c) * dg.abs() + c * (dh * u).abs())
    edu = edh * a.abs() + 1.2 * dh.abs() * eg + (2.0 ** -8 + c) * du.abs()

    def of(ref, err):
        return ref, 2.0 ** -8 * ref.abs() + 1.01 * err + 1e-30

    return {
        "y": of(h @ wd.t(), (eh + F * u23 * h.abs()) @ wd.abs().t()),
        "dx": of(dg @ wg + du @ wu, (edg + 2 * F * u23 * dg.abs()) @ wg.abs()
                 + (edu + 2 * F * u23 * du.abs()) @ wu.abs()),
        "dwg": of(dg.t() @ x, (edg + T * u23 * dg.abs()).t() @ x.abs()),
        "dwu": of(du.t() @ x, (edu + T * u23 * du.abs()).t() @ x.abs()),
        "dwd": of(dy.t() @ h, dy.abs().t() @ (eh + T * u23 * h.abs())),
    }


def check(name, got, ref, bound):
    err = (got.double() - ref).abs()
    bad = err > bound
    assert not bool(bad.any()), \
        f"{name}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst x{float((err / bound).max()):.3g}"
    if ref.numel() >= 4096:
        rel = float(err.norm() / ref.norm())
        assert rel <= 4e-3, f"{name}: normwise {rel:.3g}"


def call(L, x, wg, wu, wd, dy, act):
    """Forward and backward with every buffer inside guard bands, poisoned."""
    (T, D), F = x.shape, wg.shape[0]
    guards, out = {}, {}
    for k, shape in (("y", (T, D)), ("dx", (T, D)), ("dwg", (F, D)), ("dwu", (F, D)),
                     ("dwd", (D, F))):
        guards[k], out[k] = guarded_empty(shape, torch.bfloat16)
    wf, wb = L.adaln_ffn_workspace_size(T, D, F)
    for k, n in (("saved", L.adaln_ffn_saved_size(T, D, F)), ("wf", wf), ("wb", wb)):
        guards[k], out[k] = guarded_empty((n,), torch.uint8)
        out[k].fill_(0xFF)
    y0, none = L.adaln_ffn_fwd(x, wg, wu, wd, act=act, y=out["y"], workspace=out["wf"])
    assert none is None
    y0 = y0.clone()
    out["wf"].fill_(0xFF)
    L.adaln_ffn_fwd(x, wg, wu, wd, act=act, y=out["y"], saved=out["saved"], workspace=out["wf"])
    assert torch.equal(y0, out["y"])  # saving changes nothing
    L.adaln_ffn_bwd(dy, x, wg, wu, wd, out["saved"], act=act, dx=out["dx"], dwg=out["dwg"],
                    dwu=out["dwu"], dwd=out["dwd"], workspace=out["wb"])
    check_guards(guards)
    status_ok()
    return out


SHAPES = [
    (1, 8, 8), (1, 64, 128), (1, 1536, 4096), (2, 512, 1376), (3, 72, 40), (16, 1536, 512),
    (17, 256, 8192), (32, 392, 904), (33, 392, 904), (40, 264, 6000), (64, 520, 2000), (65, 128, 128), (127, 1000, 344),
    (128, 128, 128), (129, 136, 264), (200, 5120, 648), (255, 256, 512), (256, 256, 256),
    (257, 520, 312), (300, 64, 1000), (513, 264, 2056), (1111, 1000, 2728), (2500, 512, 768),
    (4100, 8, 16),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_against_64_bits(adaln, shape):
    T, D, F = shape
    act = ACTS[(T + D + F) // 8 % 3]
    data = inputs(T, D, F, seed=T + F)
    out = call(adaln, *data, act)
    for name, (ref, bound) in reference(*data, act).items():
        check(name, out[name], ref, bound)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T", [5, 300])
def test_activations_over_their_range(adaln, act, T):
    """Pre-activations up to several hundred, both signs."""
    data = inputs(T, 256, 384, seed=9, gain=80.0)
    out = call(adaln, *data, act)
    for name, (ref, bound) in reference(*data, act).items():
        check(name, out[name], ref, bound)


@pytest.mark.parametrize("T", [3, 400])
def test_what_is_not_finite_stays_in_its_row(adaln, T):
    x, wg, wu, wd, dy = inputs(T, 200, 328, seed=4)
    y, saved = adaln.adaln_ffn_fwd(x, wg, wu, wd, save=True)
    dx = adaln.adaln_ffn_bwd(dy, x, wg, wu, wd, saved)[0]
    x2, dy2 = x.clone(), dy.clone()
    x2[1, 7] = float("nan")
    dy2[T - 1, 3] = float("inf")
    y2, saved2 = adaln.adaln_ffn_fwd(x2, wg, wu, wd, save=True)
    dx2 = adaln.adaln_ffn_bwd(dy2, x2, wg, wu, wd, saved2)[0]
    keep = torch.ones(T, dtype=torch.bool)
    keep[1] = False
    assert bool(y2[1].isnan().all()) and torch.equal(y2[keep], y[keep])
    keep[T - 1] = False
    assert bool(dx2[1].isnan().all()) and not bool(dx2[T - 1].isfinite().any())
    assert torch.equal(dx2[keep], dx[keep])
    status_ok()


def test_no_tokens(adaln):
    x, wg, wu, wd, dy = inputs(0, 64, 96)
    y, saved = adaln.adaln_ffn_fwd(x, wg, wu, wd, save=True)
    assert y.shape == (0, 64)
    grads = [torch.ones_like(wg), torch.ones_like(wu), torch.ones_like(wd)]
    dx, *_ = adaln.adaln_ffn_bwd(dy, x, wg, wu, wd, saved, dwg=grads[0], dwu=grads[1], dwd=grads[2])
    assert dx.shape == (0, 64) and not any(bool(g.any()) for g in grads)
    status_ok()


@pytest.mark.parametrize("shape", [(1, 1536, 4096), (50, 512, 1376), (700, 512, 1376)])
def test_reproducible_over_streams_and_workspaces(adaln, shape):
    x, wg, wu, wd, dy = inputs(*shape, seed=2)
    y, saved = adaln.adaln_ffn_fwd(x, wg, wu, wd, save=True)
    first = (y, *adaln.adaln_ffn_bwd(dy, x, wg, wu, wd, saved))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s):
            y2, saved2 = adaln.adaln_ffn_fwd(x, wg, wu, wd, save=True)
            again = (y2, *adaln.adaln_ffn_bwd(dy, x, wg, wu, wd, saved2))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_inputs_written_by_the_previous_kernel_are_seen(adaln):
    """Weights and tokens written on the stream just before the call."""
    x, wg, wu, wd, _ = inputs(20, 512, 1376, seed=1)
    want, _ = adaln.adaln_ffn_fwd(x, wg, wu, wd)
    bufs = [torch.empty_like(t) for t in (x, wg, wu, wd)]
    for i in range(20):
        for b in bufs:
            b.zero_()
        adaln.adaln_ffn_fwd(*bufs)
        for b, t in zip(bufs, (x, wg, wu, wd)):
            b.copy_(t)
        y, _ = adaln.adaln_ffn_fwd(*bufs)
        assert torch.equal(y, want), i


def test_offsets_past_32_bits(adaln):
    """T x F beyond 2^32 bytes in every hidden array (and 2^31 elements): rows at
    both ends and around the 2^31st element of the hidden arrays are right, and
    the weight gradients sum over all of them."""
    T, D, F = 300000, 64, 8192
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.fail("needs 60 GB of device memory")
    x, wg, wu, wd, dy = inputs(T, D, F, seed=12)
    y, saved = adaln.adaln_ffn_fwd(x, wg, wu, wd, save=True)
    dx, dwg, dwu, dwd = adaln.adaln_ffn_bwd(dy, x, wg, wu, wd, saved)
    del saved
    at = (1 << 31) // F
    rows = torch.tensor([0, 1, 255, 256, at - 1, at, at + 1, T - 2, T - 1], device="cuda")
    ref = reference(x[rows], wg, wu, wd, dy[rows], "silu")
    for name, got in (("y", y), ("dx", dx)):
        check(name, got[rows], *ref[name])
    sums = {"dwg": 0, "dwu": 0, "dwd": 0}
    for i in range(0, T, 30000):
        part = reference(x[i:i + 30000], wg, wu, wd, dy[i:i + 30000], "silu")
        sums = {k: v + part[k][0] for k, v in sums.items()}
    for name, got in (("dwg", dwg), ("dwu", dwu), ("dwd", dwd)):
        rel = float((got.double() - sums[name]).norm() / sums[name].norm())
        assert rel <= 4e-3, f"{name}: normwise {rel:.3g}"
    status_ok()


@pytest.mark.parametrize("T", [1, 300])
def test_in_a_cuda_graph(adaln, T):
    x, wg, wu, wd, dy = inputs(T, 256, 512, seed=6)
    y, saved = adaln.adaln_ffn_fwd(x, wg, wu, wd, save=True)
    want = (y.clone(), *[t.clone() for t in adaln.adaln_ffn_bwd(dy, x, wg, wu, wd, saved)])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, saved = adaln.adaln_ffn_fwd(x, wg, wu, wd, save=True)
        got = (y, *adaln.adaln_ffn_bwd(dy, x, wg, wu, wd, saved))
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradients_against_differences(adaln):
    """Directional differences of the 64-bit definition, at the inputs' bf16
    values: the kernel's gradients agree with the slope to the roundings of
    their elements (1e-2 of the sum of |terms| in a random direction)."""
    T, D, F = 70, 96, 160
    data = dict(zip(("x", "wg", "wu", "wd", "dy"), inputs(T, D, F, seed=8)))
    v = {k: t.double() for k, t in data.items()}

    def loss(p):
        return (((act_of("gelu", p["x"] @ p["wg"].t())[0] * (p["x"] @ p["wu"].t())) @ p["wd"].t())
                * v["dy"]).sum()

    y, saved = adaln.adaln_ffn_fwd(*(data[k] for k in ("x", "wg", "wu", "wd")), act="gelu", save=True)
    grads = dict(zip(("x", "wg", "wu", "wd"), adaln.adaln_ffn_bwd(
        data["dy"], *(data[k] for k in ("x", "wg", "wu", "wd")), saved, act="gelu")))
    g = torch.Generator(device="cuda").manual_seed(1)
    for n, grad in grads.items():
        d = torch.randn(grad.shape, device="cuda", generator=g, dtype=torch.float64)
        h = 1e-5
        slope = (loss(dict(v, **{n: v[n] + h * d})) - loss(dict(v, **{n: v[n] - h * d}))) / (2 * h)
        terms = grad.double() * d
        assert abs(float(slope - terms.sum())) <= 1e-2 * float(terms.abs().sum()), n


def test_binding_refuses(adaln):
    x, wg, wu, wd, dy = inputs(4, 64, 96)
    with pytest.raises(adaln.AdalnError) as e:
        adaln.adaln_ffn_fwd(*(t.float() for t in (x, wg, wu, wd)))
    assert e.value.code == adaln.ADALN_ERR_DTYPE
    for bad in ((x[:, ::2], wg, wu, wd), (x, wg[:90], wu, wd), (x, wg, wu, wd.t()),
                (x, wg.cpu(), wu, wd)):
        with pytest.raises(ValueError):
            adaln.adaln_ffn_fwd(*bad)
    with pytest.raises(TypeError):
        adaln.adaln_ffn_fwd(x, wg.float(), wu, wd)
    with pytest.raises(ValueError):
        adaln.adaln_ffn_fwd(x, wg, wu, wd, act="relu")
    with pytest.raises(adaln.AdalnError) as e:
        adaln.adaln_ffn_fwd(x, wg, wu, wd, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == adaln.ADALN_ERR_WORKSPACE
    with pytest.raises(ValueError):
        adaln.adaln_ffn_fwd(x, wg, wu, wd, saved=torch.empty(16, dtype=torch.uint8, device="cuda"))
    _, saved = adaln.adaln_ffn_fwd(x, wg, wu, wd, save=True)
    with pytest.raises(ValueError):
        adaln.adaln_ffn_bwd(dy[:3], x, wg, wu, wd, saved)
    with pytest.raises(ValueError):
        adaln.adaln_ffn_bwd(dy, x, wg, wu, wd, saved[:-300])
