"""The experts' feed-forward on sorted rows (adaln_experts_ffn_*), and a mixture of
experts with all that belongs to it, against the definition in 64 bits.

Each expert's rows go through the gated feed-forward block, so the bounds are that
block's (test_gpu_ffn.reference derives them), expert by expert; the rows between the
experts' tokens are zeros and stay so.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import check_guards, guarded_empty, status_ok
from test_gpu_ffn import ACTS, act_of, check, reference

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def sizes(E, total, seed, how="mixed"):
    """Tokens of every expert: uneven, some without any; all of one; or even."""
    g = np.random.default_rng(seed)
    if how == "one":
        return [total if e == E // 2 else 0 for e in range(E)]
    if how == "even":
        return [total // E] * E
    share = g.random(E) ** 2 * (g.random(E) > 0.2)
    share[seed % E] += 0.1
    return [int(n) for n in np.floor(total * share / share.sum())]


def inputs(tokens, D, F, seed=0, spare=1, gain=1.0):
    """(xs, wg, wu, wd, starts, dys): sorted arrays with `spare` blocks of 64 rows of NaN
    behind the last expert."""
    E = len(tokens)
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, device="cuda", generator=g) * std).bfloat16()  # noqa: E731
    starts = np.concatenate([[0], np.cumsum([-(-n // 64) * 64 for n in tokens])])
    rows = int(starts[-1]) + 64 * spare
    xs, dys = torch.zeros(rows, D, device="cuda", dtype=BF16), torch.zeros(rows, D, device="cuda", dtype=BF16)
    for e, n in enumerate(tokens):
        at = int(starts[e])
        xs[at:at + n] = r(n, D, std=gain)
        dys[at:at + n] = r(n, D, std=0.1)
    xs[int(starts[-1]):] = float("nan")
    dys[int(starts[-1]):] = float("nan")
    return (xs, r(E, F, D, std=D ** -0.5), r(E, F, D, std=D ** -0.5), r(E, D, F, std=F ** -0.5),
            torch.from_numpy(starts.astype(np.int32)).cuda(), dys)


def call(L, xs, wg, wu, wd, starts, dys, act):
    """Forward and backward, every buffer inside guard bands, poisoned."""
    (rows, D), (E, F, _) = xs.shape, wg.shape
    guards, out = {}, {}
    for k, shape in (("ys", (rows, D)), ("dxs", (rows, D)), ("dwg", (E, F, D)), ("dwu", (E, F, D)),
                     ("dwd", (E, D, F))):
        guards[k], out[k] = guarded_empty(shape, BF16)
        out[k].fill_(7.0)
    wf, wb = L.adaln_experts_ffn_workspace_size(rows, E, D, F)
    for k, n in (("saved", L.adaln_experts_ffn_saved_size(rows, E, D, F)), ("wf", wf), ("wb", wb)):
        guards[k], out[k] = guarded_empty((n,), torch.uint8)
        out[k].fill_(0xFF)
    y0, none = L.adaln_experts_ffn_fwd(xs, wg, wu, wd, starts, act=act, ys=out["ys"], workspace=out["wf"])
    assert none is None
    y0 = y0.clone()
    out["wf"].fill_(0xFF)
    L.adaln_experts_ffn_fwd(xs, wg, wu, wd, starts, act=act, ys=out["ys"], saved=out["saved"],
                            workspace=out["wf"])
    assert torch.equal(y0.view(torch.int16), out["ys"].view(torch.int16))  # saving changes nothing
    L.adaln_experts_ffn_bwd(dys, xs, wg, wu, wd, starts, out["saved"], act=act, dxs=out["dxs"],
                            dwg=out["dwg"], dwu=out["dwu"], dwd=out["dwd"], workspace=out["wb"])
    check_guards(guards)
    status_ok()
    return out


def against(out, tokens, xs, wg, wu, wd, starts, dys, act):
    at = starts.tolist()
    for e, n in enumerate(tokens):
        rows = slice(at[e], at[e] + n)
        pads = slice(at[e] + n, at[e + 1])
        for k in ("ys", "dxs"):
            assert not bool(out[k][pads].any()), (k, e)
        if n == 0:
            assert not any(bool(out[k][e].any()) for k in ("dwg", "dwu", "dwd"))
            continue
        ref = reference(xs[rows], wg[e], wu[e], wd[e], dys[rows], act)
        for k, name in (("y", "ys"), ("dx", "dxs")):
            check(f"{name} of expert {e}", out[name][rows], *ref[k])
        for k in ("dwg", "dwu", "dwd"):
            check(f"{k} of expert {e}", out[k][e], *ref[k])
    for k in ("ys", "dxs"):  # what lies behind the last expert is left as it was
        assert bool((out[k][at[-1]:] == 7.0).all())


SHAPES = [
    # E, tokens, D, F, how
    (1, 1, 8, 8, "mixed"), (2, 3, 64, 128, "mixed"), (8, 8, 1536, 512, "even"), (8, 16, 512, 1376, "mixed"),
    (4, 300, 264, 904, "mixed"), (3, 777, 72, 40, "mixed"), (5, 1280, 256, 256, "even"),
    (8, 1111, 1000, 2728, "mixed"), (64, 700, 128, 136, "mixed"), (256, 900, 64, 72, "mixed"),
    (33, 33, 392, 328, "even"), (7, 2100, 520, 312, "one"), (2, 4100, 512, 768, "mixed"),
    (4, 256, 5120, 648, "even"), (16, 64, 200, 8200, "mixed"), (256, 1, 8, 16, "one"),
    (3, 700, 256, 8200, "mixed"), (2, 600, 1000, 4096, "even"),  # few tiles: split sums
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_against_64_bits(adaln, shape):
    E, total, D, F, how = shape
    act = ACTS[(total + D + F) // 8 % 3]
    tokens = sizes(E, total, total, how)
    data = inputs(tokens, D, F, seed=total + F)
    against(call(adaln, *data, act), tokens, *data, act)


@pytest.mark.parametrize("act", ACTS)
def test_activations_over_their_range(adaln, act):
    tokens = [5, 0, 300, 70]
    data = inputs(tokens, 256, 384, seed=9, gain=80.0)
    against(call(adaln, *data, act), tokens, *data, act)


def test_rows_about_a_tile(adaln):
    """Every number of rows about the edges of blocks, tiles and pairs of tiles."""
    tokens = [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257, 511, 512, 513, 0, 1]
    data = inputs(tokens, 136, 264, seed=1)
    against(call(adaln, *data, "silu"), tokens, *data, "silu")


@pytest.mark.parametrize("spare", [0, 40])
@pytest.mark.parametrize("tokens,D,F", [([3, 0, 64, 1, 40, 63, 2, 0], 264, 520), ([5], 1536, 4096), ([1] * 20, 72, 200),
                                        ([0, 0, 130, 0, 0, 0, 0, 7], 200, 72), ([64] * 9, 8, 8)])
def test_few_rows(adaln, tokens, D, F, spare):
    """The form for few rows (no spare ones) and, on the same rows with many spare ones
    behind them, the other."""
    data = inputs(tokens, D, F, seed=len(tokens), spare=spare)
    for act in ACTS:
        against(call(adaln, *data, act), tokens, *data, act)


def test_one_expert_equals_the_block(adaln):
    """The same products in the same order: the same bits as the feed-forward block."""
    tokens = [1024]
    xs, wg, wu, wd, starts, dys = inputs(tokens, 512, 1376, seed=3, spare=0)
    ys, saved = adaln.adaln_experts_ffn_fwd(xs, wg, wu, wd, starts, save=True)
    y, saved1 = adaln.adaln_ffn_fwd(xs, wg[0], wu[0], wd[0], save=True)
    assert torch.equal(ys, y)
    got = adaln.adaln_experts_ffn_bwd(dys, xs, wg, wu, wd, starts, saved)
    want = adaln.adaln_ffn_bwd(dys, xs, wg[0], wu[0], wd[0], saved1)
    for a, b in zip(got[1:], want[1:]):
        assert torch.equal(a[0], b)


def test_an_experts_rows_do_not_depend_on_the_others(adaln):
    """NaN and infinities in one expert's tokens and weights stay with it, also where
    its tile reaches into the next expert's rows."""
    tokens = [70, 3, 260, 0, 40]
    xs, wg, wu, wd, starts, dys = inputs(tokens, 200, 328, seed=4)
    clean = call(adaln, xs, wg, wu, wd, starts, dys, "silu")
    at = starts.tolist()
    x2, g2, d2 = xs.clone(), wg.clone(), wd.clone()
    x2[at[1]] = float("nan")
    g2[1] = float("inf")
    d2[1] = float("nan")
    g2[3] = float("nan")  # an expert without rows
    out = call(adaln, x2, g2, wu, d2, starts, dys, "silu")
    for e in (0, 2, 4):
        rows = slice(at[e], at[e + 1])
        assert torch.equal(out["ys"][rows], clean["ys"][rows])
        assert torch.equal(out["dxs"][rows], clean["dxs"][rows])
    for k in ("dwg", "dwu", "dwd"):
        for e in (0, 2, 3, 4):
            assert torch.equal(out[k][e], clean[k][e]), (k, e)
    assert not bool(out["ys"][at[1]:at[1] + 3].isfinite().any())


@pytest.mark.parametrize("spare", [0, 40])
def test_bad_starts_are_recorded(adaln, spare):
    """In both forms: no multiple of 64, not from 0 on, decreasing, past the rows."""
    xs, wg, wu, wd, starts, dys = inputs([70, 3, 0, 0, 60], 64, 96, seed=2, spare=spare)
    rows = len(xs)
    for at, bad in ((1, 100), (0, -64), (0, 64), (2, 64), (5, rows + 64), (1, 2 ** 31 - 64), (5, 0),
                    (slice(0, 6), rows), (slice(0, 2), 128)):
        s = starts.clone()
        s[at] = bad
        _, saved = adaln.adaln_experts_ffn_fwd(xs, wg, wu, wd, s, save=True)
        assert adaln.adaln_get_status() == (adaln.ADALN_ERR_EXPERT, adaln.ADALN_DEV_EXPERT_RANGE), (at, bad)
        adaln.adaln_experts_ffn_bwd(dys, xs, wg, wu, wd, s, saved)
        assert adaln.adaln_get_status() == (adaln.ADALN_ERR_EXPERT, adaln.ADALN_DEV_EXPERT_RANGE), (at, bad)
    status_ok()


def test_no_rows(adaln):
    """No rows at all, and rows of which no expert has any."""
    for rows in (0, 128):
        _, wg, wu, wd, _, _ = inputs([1, 1], 64, 96)
        x = torch.full((rows, 64), 7.0, device="cuda", dtype=BF16)
        starts = torch.zeros(3, dtype=torch.int32, device="cuda")
        ys, saved = adaln.adaln_experts_ffn_fwd(x, wg, wu, wd, starts, save=True, ys=x.clone())
        assert torch.equal(ys, x)
        grads = [torch.ones_like(t) for t in (wg, wu, wd)]
        dxs, *_ = adaln.adaln_experts_ffn_bwd(x, x, wg, wu, wd, starts, saved, dxs=x.clone(), dwg=grads[0],
                                              dwu=grads[1], dwd=grads[2])
        assert torch.equal(dxs, x) and not any(bool(t.any()) for t in grads)
    status_ok()


@pytest.mark.parametrize("total", [6, 900])
def test_on_streams_and_in_a_graph(adaln, total):
    """The same bits on another stream, and at a graph's replay on other starts."""
    tokens, others = sizes(6, total, 1), sizes(6, total, 2)
    xs, wg, wu, wd, starts, dys = inputs(tokens, 256, 512, seed=6, spare=6)
    more = inputs(others, 256, 512, seed=7, spare=12)
    kept = [torch.zeros_like(xs) for _ in range(2)]

    def all_of_it(ys, dxs):
        _, saved = adaln.adaln_experts_ffn_fwd(xs, wg, wu, wd, starts, save=True, ys=ys)
        return (ys, *adaln.adaln_experts_ffn_bwd(dys, xs, wg, wu, wd, starts, saved, dxs=dxs))

    new = lambda: all_of_it(torch.zeros_like(xs), torch.zeros_like(xs))  # noqa: E731
    first = new()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(s):
            again = new()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = all_of_it(*kept)
    n = min(len(xs), len(more[0]))
    assert int(more[4][-1]) <= n
    for t, v in ((xs, more[0]), (dys, more[5])):
        t.fill_(float("nan"))
        t[:n].copy_(v[:n])
    starts.copy_(more[4])
    for t in kept:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(new(), again))
    status_ok()


def test_offsets_past_32_bits(adaln):
    """Hidden arrays past 2^31 elements and 2^32 bytes, weights past 2^31 elements."""
    D, F, tokens = 64, 8192, [140000, 0, 129999]
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.fail("needs 60 GB of device memory")
    xs, wg, wu, wd, starts, dys = inputs(tokens, D, F, seed=12)
    ys, saved = adaln.adaln_experts_ffn_fwd(xs, wg, wu, wd, starts, save=True)
    dxs, dwg, dwu, dwd = adaln.adaln_experts_ffn_bwd(dys, xs, wg, wu, wd, starts, saved)
    del saved
    at, mid = starts.tolist(), (1 << 31) // F
    for e, rows in ((0, [0, 1, 139999]), (2, [at[2], mid - 1, mid, mid + 1, at[2] + 129998])):
        rows = torch.tensor(rows, device="cuda")
        ref = reference(xs[rows], wg[e], wu[e], wd[e], dys[rows], "silu")
        check("ys", ys[rows], *ref["y"])
        check("dxs", dxs[rows], *ref["dx"])
    sums = {"dwg": 0, "dwu": 0, "dwd": 0}
    for i in range(at[2], at[2] + 129999, 30000):
        j = min(i + 30000, at[2] + 129999)
        part = reference(xs[i:j], wg[2], wu[2], wd[2], dys[i:j], "silu")
        sums = {k: v + part[k][0] for k, v in sums.items()}
    for name, got in (("dwg", dwg), ("dwu", dwu), ("dwd", dwd)):
        rel = float((got[2].double() - sums[name]).norm() / sums[name].norm())
        assert rel <= 4e-3, f"{name}: normwise {rel:.3g}"
        assert not bool(got[1].any())
    del xs, wg, wu, wd, dys, ys, dxs, dwg, dwu, dwd
    xs, wg, wu, wd, starts, dys = inputs([0] * 200 + [5], 2048, 5400, seed=1)  # 2.2e9 elements each
    ys, saved = adaln.adaln_experts_ffn_fwd(xs, wg, wu, wd, starts, save=True)
    ref = reference(xs[:5], wg[200], wu[200], wd[200], dys[:5], "silu")
    check("ys", ys[:5], *ref["y"])
    dxs, dwg, dwu, dwd = adaln.adaln_experts_ffn_bwd(dys, xs, wg, wu, wd, starts, saved)
    for name, got in (("dwg", dwg), ("dwu", dwu), ("dwd", dwd)):
        check(name, got[200], *ref[name])
        assert not bool(got[:200].any())
    check("dxs", dxs[:5], *ref["dx"])
    status_ok()


def plain_mixture(x, w, expert, wg, wu, wd, act):
    """A mixture of experts, token by token's choices, in the type of its arguments."""
    y = torch.zeros_like(x)
    for j in range(expert.shape[1]):
        for e in range(len(wg)):
            t = (expert[:, j] == e).nonzero()[:, 0]
            h = act_of(act, x[t] @ wg[e].t())[0] * (x[t] @ wu[e].t())
            y = y.index_add(0, t, w[t, j:j + 1] * (h @ wd[e].t()))
    return y


@pytest.mark.parametrize("T,E,k,D,F", [(1, 4, 2, 64, 96), (37, 8, 3, 128, 200), (700, 6, 2, 264, 520)])
def test_a_mixture_of_experts_as_a_whole(adaln, T, E, k, D, F):
    """Route, sort, experts, combine and back, in one graph of nodes.  Sorted arrays are
    bf16 between the operators (2^-8 each, three or four of them on the longest way) and
    the block's own roundings are two: over many elements the 2-norm of the error is at
    most sqrt(6) 2^-8 / sqrt(3) = 5.6e-3 of the result's; 8e-3 holds that."""
    from adaln_video_dit_gb300.autograd import expert_combine, expert_sort, experts_ffn, route
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s, std=1.0: (torch.randn(*s, device="cuda", generator=g) * std).bfloat16()  # noqa: E731
    leaves = [r(T, D), torch.rand(T, k, device="cuda", generator=g), r(E, F, D, std=D ** -0.5),
              r(E, F, D, std=D ** -0.5), r(E, D, F, std=F ** -0.5)]
    expert = torch.rand(T, E, device="cuda", generator=g).topk(k)[1]
    expert[T // 3] = -1  # a padded token
    dy = r(T, D)
    x, w, wg, wu, wd = (t.requires_grad_() for t in leaves)
    way = route(expert, E)
    y = expert_combine(experts_ffn(expert_sort(x, way), wg, wu, wd, way, "gelu"), w, way)
    y.backward(dy)
    wide = [t.detach().double().requires_grad_() for t in leaves]
    ref = plain_mixture(wide[0], wide[1], expert, *wide[2:], "gelu")
    grads = torch.autograd.grad(ref, wide, dy.double())
    for name, got, want in zip(("y", "dx", "dw", "dwg", "dwu", "dwd"),
                               (y, *(t.grad for t in leaves)), (ref, *grads)):
        assert bool(got.isfinite().all()), name
        want = want.detach()
        off, size = float((got.detach().double() - want).norm()), float(want.norm())
        assert off <= 8e-3 * size if size > 0 else off == 0, (name, off, size)
    assert not bool(y[T // 3].any()) and not bool(x.grad[T // 3].any())
    status_ok()


def test_the_mixture_module(adaln):
    from adaln_video_dit_gb300.autograd import MixtureFFN
    torch.manual_seed(5)
    m = MixtureFFN(128, 256, 8, top_k=2, device="cuda")
    x = torch.randn(3, 40, 128, device="cuda").bfloat16().requires_grad_()
    mask = torch.ones(3, 40, dtype=torch.bool, device="cuda")
    mask[1, 30:] = False
    y = m(x, mask)
    assert y.shape == x.shape and not bool(y[1, 30:].any()) and bool(y[0].any())
    y.float().square().sum().backward()
    assert all(bool(t.grad.isfinite().all()) and bool(t.grad.any()) for t in m.parameters())
    assert not bool(x.grad[1, 30:].any())
    with torch.no_grad():
        assert torch.equal(m(x, mask), y)
    status_ok()


def test_trace_counts_the_launches(adaln):
    xs, wg, wu, wd, starts, dys = inputs([300, 500], 64, 96)
    adaln.adaln_trace_begin(16)
    _, saved = adaln.adaln_experts_ffn_fwd(xs, wg, wu, wd, starts, save=True)
    adaln.adaln_experts_ffn_bwd(dys, xs, wg, wu, wd, starts, saved)
    adaln.adaln_trace_end()
    assert adaln.adaln_trace_get(adaln.ADALN_KERNEL_EXPERTS)[0] >= 4
    assert adaln.adaln_trace_get(adaln.ADALN_KERNEL_FFN)[0] == 0


def test_binding_refuses(adaln):
    xs, wg, wu, wd, starts, dys = inputs([30, 50], 64, 96)
    f = adaln.adaln_experts_ffn_fwd
    with pytest.raises(adaln.AdalnError) as e:
        f(*(t.float() for t in (xs, wg, wu, wd)), starts)
    assert e.value.code == adaln.ADALN_ERR_DTYPE
    for bad in ((xs[:, ::2], wg, wu, wd, starts), (xs, wg[:, :90], wu, wd, starts), (xs, wg[:1], wu, wd, starts),
                (xs, wg, wu, wd.transpose(1, 2), starts), (xs, wg.cpu(), wu, wd, starts),
                (xs, wg, wu, wd, starts[:2]), (xs, wg, wu, wd, starts.cpu()), (xs, wg[0], wu[0], wd[0], starts)):
        with pytest.raises(ValueError):
            f(*bad)
    for bad in ((xs, wg.float(), wu, wd, starts), (xs, wg, wu, wd, starts.long())):
        with pytest.raises(TypeError):
            f(*bad)
    with pytest.raises(ValueError):
        f(xs, wg, wu, wd, starts, act="relu")
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(adaln.AdalnError) as e:
        f(xs, wg, wu, wd, starts, workspace=small)
    assert e.value.code == adaln.ADALN_ERR_WORKSPACE
    with pytest.raises(ValueError):
        f(xs, wg, wu, wd, starts, saved=small)
    _, saved = f(xs, wg, wu, wd, starts, save=True)
    with pytest.raises(ValueError):
        adaln.adaln_experts_ffn_bwd(dys[:3], xs, wg, wu, wd, starts, saved)
    with pytest.raises(ValueError):
        adaln.adaln_experts_ffn_bwd(dys, xs, wg, wu, wd, starts, saved[:-300])
    with pytest.raises(ValueError):
        adaln.adaln_experts_ffn_bwd(dys, xs, wg, wu, wd, starts, None)


@pytest.mark.parametrize("tokens,D,F,forward,backward", [
    ([300, 500], 64, 96, 2, 2),           # tiles; sums over k as they are
    ([250, 250, 200], 256, 8200, 3, 3),   # few tiles: both sums over F split and joined
    ([3, 0, 64, 1], 264, 520, 2, 3),      # few rows: dh, dx, and the weight gradients
], ids=["tiles", "split", "few"])
def test_launches_of_each_form(adaln, tokens, D, F, forward, backward):
    """As many as a call needs, none beside them."""
    xs, wg, wu, wd, starts, dys = inputs(tokens, D, F, spare=0)
    counts = []
    for call in (lambda: adaln.adaln_experts_ffn_fwd(xs, wg, wu, wd, starts, save=True)[1],
                 lambda: adaln.adaln_experts_ffn_bwd(dys, xs, wg, wu, wd, starts, saved)):
        adaln.adaln_trace_begin(16)
        saved = call()
        adaln.adaln_trace_end()
        counts.append(adaln.adaln_trace_get(adaln.ADALN_KERNEL_EXPERTS)[0])
    assert counts == [forward, backward]
    status_ok()
