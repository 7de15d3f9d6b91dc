"""Tokens sorted by expert and back (adaln_route, adaln_expert_*) against the
definition: places and copies exactly, sums in 64 bits.

Tolerances, with u = 2^-24 and r = 2^-8 (bf16 outputs) or u (fp32 ones): a sum of k
products in fp32 is within (k + 1) u sum |terms|, then rounded to its type (r of it);
dys is one product, r of it and u; dweight is an fp32 sum of D products: (D + 2) u
sum |terms|.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import check_guards, guarded_empty, status_ok

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def layout(expert, E, align):
    """(row, starts, counts), pair by pair."""
    counts = np.bincount(expert[expert >= 0].reshape(-1), minlength=E)
    starts = np.concatenate([[0], np.cumsum(-(-counts // align) * align)])
    nxt, row = starts[:-1].copy(), np.full(expert.size, -1)
    for i, e in enumerate(expert.reshape(-1)):
        if e >= 0:
            row[i] = nxt[e]
            nxt[e] += 1
    return row.reshape(expert.shape), starts, counts


def choices(T, k, E, seed, how="mixed"):
    """Experts of every token: uneven, some twice, some -1; or all of one expert."""
    g = np.random.default_rng(seed)
    if how == "one":
        return np.full((T, k), E - 1, np.int32)
    e = np.minimum((E * g.random((T, k)) ** 2).astype(np.int32), E - 1)
    return np.where(g.random((T, k)) < 0.1, -1, e).astype(np.int32)


def check_route(L, expert, E, align):
    row, starts, counts = layout(expert, E, align)
    T, k = expert.shape
    guards, out = {}, {}
    for n, shape in (("row", (T, k)), ("starts", (E + 1,)), ("counts", (E,))):
        guards[n], out[n] = guarded_empty(shape, torch.int32)
    guards["ws"], out["ws"] = guarded_empty((L.adaln_route_workspace_size(T, k, E),), torch.uint8)
    out["ws"].fill_(0xFF)
    r = L.adaln_route(torch.from_numpy(expert).cuda(), E, align, row=out["row"], starts=out["starts"],
                      counts=out["counts"], workspace=out["ws"])
    check_guards(guards)
    for got, want in ((r.row, row), (r.starts, starts), (r.counts, counts)):
        assert np.array_equal(got.cpu().numpy(), want)
    assert r.rows == L.adaln_route_rows(T, k, E, align) >= starts[-1] and r.rows % align == 0
    return r, row, starts


@pytest.mark.parametrize("how", ["mixed", "one"])
@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (1, 2, 8), (1, 32, 256), (3, 5, 4), (31, 1, 7),
                                   (33, 1, 64), (100, 8, 256), (1111, 6, 64), (2048, 8, 16), (4096, 1, 9), (4097, 1, 9), (16384, 1, 256),
                                   (16385, 1, 3), (8200, 2, 256), (32768, 4, 96), (131073, 1, 7), (200001, 3, 8),
                                   (300000, 8, 64)])
def test_places(adaln, T, k, E, how):
    for align in (64, 1) if T < 2048 else (64,):
        check_route(adaln, choices(T, k, E, T + k, how), E, align)
    status_ok()


@pytest.mark.parametrize("align", [2, 3, 128, 1000, 4096])
def test_places_with_other_alignments(adaln, align):
    check_route(adaln, choices(700, 3, 9, align), 9, align)


def test_experts_out_of_range_are_recorded(adaln):
    for T in (400, 9000, 70000):
        expert = choices(T, 2, 5, 1)
        want = expert.copy()
        for at, bad in ((3, 5), (T - 1, -2), (77, 2 ** 31 - 1), (78, -2 ** 31)):
            expert[at, 1] = bad
            want[at, 1] = -1
            r = adaln.adaln_route(torch.from_numpy(expert).cuda(), 5)
            assert adaln.adaln_get_status() == (adaln.ADALN_ERR_EXPERT, adaln.ADALN_DEV_EXPERT_RANGE)
            assert np.array_equal(r.row.cpu().numpy(), layout(want, 5, 64)[0])
            expert[at, 1] = want[at, 1]
    status_ok()


def close(got, ref, bound, name):
    err = (got.double() - ref).abs()
    assert not bool((err > bound + 1e-40).any()), f"{name}: worst x{float((err / bound).max()):.3g}"


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("T,k,E,D,align", [
    (1, 1, 1, 8, 64), (1, 2, 8, 1536, 64), (1, 32, 256, 64, 64), (5, 3, 4, 24, 1), (64, 2, 8, 5120, 64),
    (333, 6, 64, 1000, 64), (1111, 5, 16, 264, 128), (2000, 8, 96, 72, 3), (4097, 1, 3, 2056, 64),
    (9000, 2, 8, 512, 64), (50, 4, 200, 8200, 64), (33001, 2, 8, 256, 64), (8003, 1, 5, 1536, 64),
    (30005, 2, 4, 200, 64), (20001, 3, 4, 72, 64)])
def test_copies_and_sums(adaln, T, k, E, D, align, dt):
    expert = choices(T, k, E, T + D)
    r, row, starts = check_route(adaln, expert, E, align)
    g = torch.Generator(device="cuda").manual_seed(T)
    n = lambda *s: torch.randn(*s, device="cuda", generator=g).to(dt)  # noqa: E731
    x, dy, ys, dxs = n(T, D), n(T, D), n(r.rows, D), n(r.rows, D)
    weight = torch.rand(T, k, device="cuda", generator=g)
    guards, out = {}, {}
    for name, shape, t in (("xs", (r.rows, D), dt), ("dx", (T, D), dt), ("y", (T, D), dt),
                           ("dys", (r.rows, D), dt), ("dw", (T, k), F32)):
        guards[name], out[name] = guarded_empty(shape, t)
        out[name].fill_(7.0)
    adaln.adaln_expert_sort_fwd(x, r, xs=out["xs"])
    adaln.adaln_expert_sort_bwd(dxs, r, dx=out["dx"])
    adaln.adaln_expert_combine_fwd(ys, weight, r, y=out["y"])
    adaln.adaln_expert_combine_bwd(dy, ys, weight, r, dys=out["dys"], dweight=out["dw"])
    check_guards(guards)
    status_ok()
    at, there = torch.from_numpy(row).cuda(), torch.from_numpy(row >= 0).cuda()
    half = 2.0 ** -8 if dt == BF16 else U
    end = int(starts[-1])
    tokens = torch.arange(T, device="cuda")[:, None].expand(T, k)[there]
    want = torch.zeros(end, D, device="cuda", dtype=dt)
    want[at[there]] = x[tokens]
    assert torch.equal(out["xs"][:end], want)
    for name in ("xs", "dys"):  # what lies behind the last expert is left as it was
        assert bool((out[name][end:] == 7.0).all())
    picked = [t.double()[at.clamp(min=0)] * there[..., None] for t in (ys, dxs)]
    w = weight.double()[..., None]
    for name, terms in (("y", w * picked[0]), ("dx", picked[1])):
        ref = terms.sum(1)
        close(out[name], ref, half * ref.abs() + (k + 1) * U * terms.abs().sum(1), name)
    want = torch.zeros(end, D, device="cuda", dtype=torch.float64)
    want[at[there]] = (w * dy.double()[:, None])[there]
    close(out["dys"][:end], want, (half + U) * want.abs(), "dys")
    assert torch.equal(out["dys"][:end] == 0, want == 0)
    terms = dy.double()[:, None] * picked[0]
    close(out["dw"], terms.sum(2), (D + 2) * U * terms.abs().sum(2), "dw")
    assert not bool(out["dw"][~there].any())


def test_rows_out_of_range_are_recorded(adaln):
    """A route read with fewer rows than it was made for: what lies outside is skipped."""
    T, k, E, D = 200, 2, 4, 64
    r, row, _ = check_route(adaln, choices(T, k, E, 3), E, 64)
    x, weight = torch.randn(T, D, device="cuda"), torch.rand(T, k, device="cuda")
    few = r._replace(rows=128)
    xs = adaln.adaln_expert_sort_fwd(x, few)
    assert adaln.adaln_get_status() == (adaln.ADALN_ERR_EXPERT, adaln.ADALN_DEV_EXPERT_RANGE)
    whole = adaln.adaln_expert_sort_fwd(x, r)
    status_ok()
    assert torch.equal(xs, whole[:128])
    for call in (lambda: adaln.adaln_expert_sort_bwd(xs, few),
                 lambda: adaln.adaln_expert_combine_fwd(xs, weight, few),
                 lambda: adaln.adaln_expert_combine_bwd(x, xs, weight, few)):
        call()
        assert adaln.adaln_get_status() == (adaln.ADALN_ERR_EXPERT, adaln.ADALN_DEV_EXPERT_RANGE)


def test_what_is_not_finite_stays_with_its_token(adaln):
    T, k, E, D = 100, 2, 4, 128
    r, row, _ = check_route(adaln, choices(T, k, E, 5), E, 64)
    x, weight = torch.randn(T, D, device="cuda"), torch.rand(T, k, device="cuda")
    ys = torch.full((r.rows, D), float("nan"), device="cuda")  # also where no token's row is
    at = torch.from_numpy(row).cuda()
    ys[at[at >= 0]] = 1.0
    ys[at[7][at[7] >= 0]] = float("inf")
    y = adaln.adaln_expert_combine_fwd(ys, weight, r)
    assert bool(y[7].isinf().all()) and bool(torch.cat([y[:7], y[8:]]).isfinite().all())
    x[3, 5] = float("nan")
    dys, dw = adaln.adaln_expert_combine_bwd(x, ys, weight, r)
    rows = at[3][at[3] >= 0]
    assert bool(dys[rows, 5].isnan().all())
    dys[rows] = 0
    assert bool(dys[: int(r.starts[-1])].isfinite().all())
    keep = torch.ones(T, dtype=torch.bool)
    keep[[3, 7]] = False
    assert bool(dw[keep].isfinite().all()) and bool(dw[3][at[3] >= 0].isnan().all())


def test_no_tokens(adaln):
    x = torch.empty(0, 64, device="cuda")
    r = adaln.adaln_route(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 4)
    assert r.rows == 0 and not bool(r.starts.any()) and not bool(r.counts.any())
    w = torch.empty(0, 2, device="cuda")
    assert adaln.adaln_expert_sort_fwd(x, r).shape == (0, 64)
    assert adaln.adaln_expert_sort_bwd(x, r).shape == (0, 64)
    assert adaln.adaln_expert_combine_fwd(x, w, r).shape == (0, 64)
    dys, dw = adaln.adaln_expert_combine_bwd(x, x, w, r)
    assert dys.shape == (0, 64) and dw.shape == (0, 2)
    status_ok()


def test_offsets_past_32_bits(adaln):
    """Sorted rows past 2^31 elements and 2^32 bytes."""
    T, k, E, D = 40000, 4, 8, 16384
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.fail("needs 30 GB of device memory")
    expert = choices(T, k, E, 1)
    r, row, starts = check_route(adaln, expert, E, 64)
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(T, D, device="cuda", generator=g, dtype=BF16)
    xs = adaln.adaln_expert_sort_fwd(x, r)
    assert int(starts[-1]) * D > 1 << 31
    pairs = np.argwhere(row >= 0)
    pairs = pairs[np.argsort(row[tuple(pairs.T)])]
    beside = int(np.searchsorted(row[tuple(pairs.T)], (1 << 31) // D))
    for i in (0, beside - 1, beside, beside + 1, len(pairs) - 1):
        t, j = pairs[i]
        assert torch.equal(xs[row[t, j]], x[t])
    weight = torch.full((T, k), 0.25, device="cuda")
    n = torch.from_numpy((expert >= 0).sum(1)).cuda()
    y = adaln.adaln_expert_combine_fwd(xs, weight, r)  # n / 4 of x, exact in fp32 but for n = 3
    assert torch.equal(y, (x.float() * (0.25 * n)[:, None]).bfloat16())
    dys, dw = adaln.adaln_expert_combine_bwd(x, xs, weight, r)
    t, j = pairs[-1]
    assert torch.equal(dys[row[t, j]], x[t] * 0.25)
    assert abs(float(dw[t, j]) - float(x[t].double().square().sum())) <= D * U * 2 * D
    status_ok()


def test_as_many_pairs_as_32_bits_hold(adaln):
    """Pairs whose number, rounded up to the alignment, only just fits: 2^31 - 2, by threes."""
    T = 2 ** 31 - 2
    r = adaln.adaln_route(torch.zeros(T, 1, dtype=torch.int32, device="cuda"), 1, align=3)
    assert r.rows == T and r.starts.tolist() == [0, T] and r.counts.tolist() == [T]
    for at in range(0, T, 1 << 28):
        n = min(1 << 28, T - at)
        assert torch.equal(r.row[at:at + n, 0], torch.arange(at, at + n, dtype=torch.int32, device="cuda"))
    status_ok()
    del r
    torch.cuda.empty_cache()


def test_on_streams_and_in_a_graph(adaln):
    T, k, E, D = 9000, 2, 8, 256
    expert = torch.from_numpy(choices(T, k, E, 2)).cuda()
    x, weight = torch.randn(T, D, device="cuda").bfloat16(), torch.rand(T, k, device="cuda")

    def all_of_it():
        r = adaln.adaln_route(expert, E)
        xs = adaln.adaln_expert_sort_fwd(x, r, xs=torch.zeros(r.rows, D, device="cuda", dtype=BF16))
        dys, dw = adaln.adaln_expert_combine_bwd(
            x, xs, weight, r, dys=torch.zeros(r.rows, D, device="cuda", dtype=BF16))
        return [r.row, r.starts, r.counts, xs, adaln.adaln_expert_combine_fwd(xs, weight, r), dys, dw,
                adaln.adaln_expert_sort_bwd(xs, r)]

    first = all_of_it()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(s):
            again = all_of_it()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = all_of_it()
    expert.copy_(torch.from_numpy(choices(T, k, E, 9)).cuda())  # another route at the replay
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(all_of_it(), again))


def test_nodes(adaln):
    from adaln_video_dit_gb300.autograd import expert_combine, expert_sort, route
    x = torch.randn(2, 30, 64, device="cuda", requires_grad=True)
    weight = torch.rand(2, 30, 3, device="cuda", requires_grad=True)
    expert = torch.from_numpy(choices(60, 3, 5, 4)).cuda().view(2, 30, 3)
    r = route(expert.long(), 5)
    xs = expert_sort(x, r)
    y = expert_combine(xs * 2, weight, r)
    y.backward(torch.ones_like(y))
    there = (expert >= 0).double()
    factor = 2 * (there * weight.detach().double()).sum(-1, keepdim=True)
    assert y.shape == x.shape
    close(y, factor * x.detach().double(), 8 * U * 2 * x.detach().double().abs() * 3, "y")
    close(x.grad, factor.expand(x.shape), 8 * U * 6 * torch.ones_like(factor), "dx")
    dots = 2 * x.detach().double().sum(-1, keepdim=True) * there
    close(weight.grad, dots, 66 * U * 2 * x.detach().double().abs().sum(-1, keepdim=True).expand(dots.shape), "dw")


def test_wide_experts_do_not_wrap(adaln):
    """int64 values that are experts in their lower 32 bits only are out of range."""
    from adaln_video_dit_gb300.autograd import route
    for e in (2 ** 32 + 1, 2 ** 40, -2 ** 32, 2 ** 32 - 1, 2 ** 63 - 1):
        r = route(torch.tensor([[1, e]], device="cuda"), 5)
        assert adaln.adaln_get_status() == (adaln.ADALN_ERR_EXPERT, adaln.ADALN_DEV_EXPERT_RANGE)
        assert r.row.tolist() == [[0, -1]] and r.counts.tolist() == [0, 1, 0, 0, 0]
    for dt in (torch.float32, torch.bool, torch.uint8):
        with pytest.raises(TypeError):
            route(torch.zeros(4, 2, device="cuda", dtype=dt), 5)


def test_trace_counts_the_launches(adaln):
    expert = torch.from_numpy(choices(70000, 2, 5, 4)).cuda()
    x, w = torch.randn(70000, 64, device="cuda"), torch.rand(70000, 2, device="cuda")
    adaln.adaln_trace_begin(16)
    r = adaln.adaln_route(expert, 5)
    small = adaln.adaln_route(expert[:8], 5)
    xs = adaln.adaln_expert_sort_fwd(x, r)
    adaln.adaln_expert_sort_bwd(xs, r)
    adaln.adaln_expert_combine_fwd(xs, w, r)
    adaln.adaln_expert_combine_bwd(x, xs, w, r)
    adaln.adaln_trace_end()
    assert adaln.adaln_trace_get(adaln.ADALN_KERNEL_EXPERTS)[0] == 7
    assert small.rows == 16 + 5 * 63 - (16 + 5 * 63) % 64


def test_binding_refuses(adaln):
    expert = torch.from_numpy(choices(20, 2, 5, 4)).cuda()
    with pytest.raises(TypeError):
        adaln.adaln_route(expert.long(), 5)
    with pytest.raises(ValueError):
        adaln.adaln_route(expert[:, 0], 5)
    with pytest.raises(ValueError):
        adaln.adaln_route(expert.t(), 5)
    for bad in (dict(E=0), dict(E=257), dict(E=-3), dict(E=5, align=0), dict(E=2 ** 40)):
        with pytest.raises(adaln.AdalnError) as e:
            adaln.adaln_route(expert, **bad)
        assert e.value.code == adaln.ADALN_ERR_DIM
    with pytest.raises(adaln.AdalnError):
        adaln.adaln_route(expert[:, :1].expand(20, 33).contiguous(), 5)
    r = adaln.adaln_route(expert, 5)
    x, w = torch.randn(20, 64, device="cuda"), torch.rand(20, 2, device="cuda")
    xs = adaln.adaln_expert_sort_fwd(x, r)
    for call in (lambda: adaln.adaln_expert_sort_fwd(x[:19], r), lambda: adaln.adaln_expert_sort_fwd(x.cpu(), r),
                 lambda: adaln.adaln_expert_sort_fwd(x, r, xs=xs[:-1]),
                 lambda: adaln.adaln_expert_sort_bwd(xs[:-1], r),
                 lambda: adaln.adaln_expert_combine_fwd(xs, w[:, :1], r),
                 lambda: adaln.adaln_expert_combine_fwd(xs, w.t(), r),
                 lambda: adaln.adaln_expert_combine_bwd(x[:, :32].contiguous(), xs, w, r),
                 lambda: adaln.adaln_expert_sort_fwd(x, r._replace(starts=r.starts[:-1]))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: adaln.adaln_expert_combine_fwd(xs, w.bfloat16(), r),
                 lambda: adaln.adaln_expert_combine_bwd(x.bfloat16(), xs, w, r),
                 lambda: adaln.adaln_expert_sort_fwd(x.half(), r), lambda: adaln.adaln_expert_sort_fwd(x, r[:3])):
        with pytest.raises(TypeError):
            call()
