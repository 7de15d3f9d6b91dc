"""The residual branch's operators together: in the example's block, in a captured
training step, from two threads, on given streams."""
import gc
import sys
import threading

import pytest
import torch

from gpu_helpers import status_ok
from test_gpu_block import example

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def test_example_block_of_experts_runs_and_has_gradients(adaln):
    m = example()
    losses = m.main(["--dim", "256", "--heads", "4", "--hidden", "512", "--steps", "3", "--experts", "6",
                     "--dropout", "0.1"])
    assert len(losses) == 3 and all(v == v for v in losses)
    torch.manual_seed(1)
    block = m.MixtureDiTBlock(128, 2, 256, 20, experts=4, dropout=0.2)
    x = torch.randn(100, 128, device="cuda", dtype=BF16, requires_grad=True)
    cond = torch.randn(2, 128, device="cuda", dtype=BF16)
    torch.nn.init.normal_(block.modulation.weight, std=0.02)
    seg = (torch.arange(100, device="cuda") >= 40).int()
    pos = torch.randint(0, 20, (100, 3), device="cuda", dtype=torch.int32)
    block(x, cond, seg, pos, [40, 60]).float().square().mean().backward()
    for name, p in [("x", x), *block.named_parameters()]:
        assert p.grad is not None and bool(p.grad.isfinite().all()) and bool(p.grad.any()), name
    status_ok()


def make(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()  # noqa: E731
    T, D, F, E, k = 700, 256, 512, 6, 2
    return dict(x=r(T, D), h=r(T, D), dy=r(T, D), gate=r(3, D), few=r(9, D),
                seg=torch.sort(torch.randint(0, 3, (T,), device="cuda", generator=g))[0].int(),
                expert=torch.rand(T, E, device="cuda", generator=g).topk(k)[1].int(),
                weight=torch.rand(T, k, device="cuda", generator=g),
                w=(r(E, F, D) / 16, r(E, F, D) / 16, r(E, D, F) / 16))


def work(L, s, stream=None):
    """Every call of the branch; the sorted arrays up to the last expert's rows."""
    how = dict(gate=s["gate"], seg_id=s["seg"], stream=stream)
    out = [L.adaln_dropout_fwd(s["h"], 0.3, (5, 6), x=s["x"], **how),
           *L.adaln_dropout_bwd(s["dy"], 0.3, (5, 6), h=s["h"], **how)]
    for n in (700, 9):
        r = L.adaln_route(s["expert"][:n], 6, stream=stream)
        x, w, dy = s["x"][:n], s["weight"][:n], s["dy"][:n]
        zeros = [torch.zeros(r.rows, 256, device="cuda", dtype=BF16) for _ in range(4)]
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        xs = L.adaln_expert_sort_fwd(x, r, xs=zeros[0], stream=stream)
        ys, saved = L.adaln_experts_ffn_fwd(xs, *s["w"], r.starts, save=True, ys=zeros[1], stream=stream)
        y = L.adaln_expert_combine_fwd(ys, w, r, stream=stream)
        dys, dw = L.adaln_expert_combine_bwd(dy, ys, w, r, dys=zeros[2], stream=stream)
        dxs, *grads = L.adaln_experts_ffn_bwd(dys, xs, *s["w"], r.starts, saved, dxs=zeros[3], stream=stream)
        out += [r.row, r.starts, r.counts, xs, ys, y, dys, dw, dxs, *grads,
                L.adaln_expert_sort_bwd(dxs, r, stream=stream)]
    return out


def test_calls_from_two_threads_on_two_streams(adaln):
    states = [make(1), make(2)]
    want = [[t.clone() for t in work(adaln, s)] for s in states]
    torch.cuda.synchronize()
    wrong = []

    def run(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(15):
                    got = work(adaln, states[i])
                    stream.synchronize()
                    wrong.extend(k for k, (a, b) in enumerate(zip(got, want[i])) if not torch.equal(a, b))
        except Exception as e:  # noqa: BLE001 (reported by the assertion below)
            wrong.append(repr(e))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:5]
    status_ok()


def test_what_a_call_on_a_given_stream_allocates_is_that_streams(adaln):
    """On a stream that is busy, given as an argument; the current stream then
    overwrites whatever memory its allocator has free."""
    s = make(3)
    want = work(adaln, s)
    torch.cuda.synchronize()
    side, busy = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda", dtype=BF16)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(40):
            busy @ busy
    got = work(adaln, s, side)
    junk = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
            for n in (512, 4096, 1 << 17, 1 << 19, 1 << 20, 3 << 20, 8 << 20) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    del junk
    status_ok()


def test_inputs_written_by_the_previous_kernel_are_seen(adaln):
    """Tokens, routes and weights written on the stream just before the calls."""
    s = make(4)
    want = work(adaln, s)
    bufs = {k: [torch.empty_like(t) for t in v] if isinstance(v, tuple) else torch.empty_like(v)
            for k, v in s.items()}
    pairs = [(b, t) for k in s for b, t in (zip(bufs[k], s[k]) if k == "w" else [(bufs[k], s[k])])]
    for i in range(10):
        for b, _ in pairs:
            b.zero_()
        work(adaln, bufs)
        for b, t in pairs:
            b.copy_(t)
        got = work(adaln, bufs)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
    status_ok()


def test_a_training_step_in_a_cuda_graph(adaln):
    """A mixture and the end of its branch, forward and backward, captured as torch
    documents it (warmed up on another stream, gradients made in the graph) and
    replayed on other tokens: as the same step without a graph."""
    from adaln_video_dit_gb300.autograd import GatedResidual, MixtureFFN
    torch.manual_seed(2)
    m, end = MixtureFFN(128, 256, 4, device="cuda"), GatedResidual(0.0)
    x = torch.randn(300, 128, device="cuda", dtype=BF16)
    gate = torch.randn(1, 128, device="cuda", dtype=BF16)
    seg = torch.zeros(300, dtype=torch.int32, device="cuda")

    def step():
        y = end(x, m(x), gate, seg)
        y.float().square().mean().backward()
        return y

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            m.zero_grad(set_to_none=True)
            step()
    torch.cuda.current_stream().wait_stream(side)
    m.zero_grad(set_to_none=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    captured = [p.grad for p in m.parameters()]
    for seed in range(2):
        x.copy_(torch.randn(300, 128, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        got = [y.clone(), *(g.clone() for g in captured)]
        m.zero_grad(set_to_none=True)
        want = [step(), *(p.grad for p in m.parameters())]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        m.zero_grad(set_to_none=True)
    status_ok()


def test_masks_of_a_captured_dropout_change_with_the_replays(adaln):
    from adaln_video_dit_gb300.autograd import dropout
    h = torch.ones(64, 512, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = dropout(h, 0.5)
    masks = []
    for _ in range(2):
        graph.replay()
        masks.append(y.clone())
    assert not torch.equal(*masks) and all(bool(((m == 0) | (m == 2)).all()) for m in masks)


def test_a_mixture_of_no_tokens(adaln):
    from adaln_video_dit_gb300.autograd import GatedResidual, MixtureFFN
    m = MixtureFFN(64, 96, 4, device="cuda")
    x = torch.randn(0, 64, device="cuda", dtype=BF16, requires_grad=True)
    y = GatedResidual(0.1)(x, m(x), torch.ones(1, 64, device="cuda", dtype=BF16),
                           torch.zeros(0, dtype=torch.int32, device="cuda"))
    y.sum().backward()
    assert y.shape == (0, 64) and not any(bool(p.grad.any()) for p in m.parameters())
    none = m(torch.randn(2, 5, 64, device="cuda", dtype=BF16), torch.zeros(2, 5, dtype=torch.bool, device="cuda"))
    assert none.shape == (2, 5, 64) and not bool(none.any())
    status_ok()


def test_masked_tokens_take_part_in_nothing(adaln):
    """NaN and infinities in masked tokens: outputs and gradients, the router's among
    them, are those of the other tokens alone."""
    from adaln_video_dit_gb300.autograd import MixtureFFN
    torch.manual_seed(5)
    m = MixtureFFN(64, 96, 4, device="cuda")
    x = torch.randn(3, 40, 64, device="cuda", dtype=BF16)
    mask = torch.rand(3, 40, device="cuda") < 0.6
    clean, foul = torch.where(mask[..., None], x, 0.0), torch.where(mask[..., None], x, float("nan"))
    foul[:, ::2] = torch.where(mask[:, ::2, None], x[:, ::2], float("inf"))
    results = []
    for t in (clean.requires_grad_(), foul.requires_grad_()):
        y = m(t, mask)
        results.append([y.detach(), *torch.autograd.grad(y.float().square().sum(), [t, *m.parameters()])])
    assert not any(bool(t.isnan().any()) for t in results[0])
    assert all(torch.equal(a, b) for a, b in zip(*results))
    assert not bool(results[0][0][~mask].any()) and not bool(results[0][1][~mask].any())
    status_ok()


def test_the_router_computes_in_32_bits(adaln):
    """Under autocast a mixture's bits are those without; one cast to bf16 as a whole runs,
    with its rounded router's."""
    from adaln_video_dit_gb300.autograd import MixtureFFN
    torch.manual_seed(6)
    m = MixtureFFN(64, 96, 4, device="cuda")
    x = torch.randn(100, 64, device="cuda", dtype=BF16)
    want = m(x)
    with torch.autocast("cuda", dtype=BF16):
        got = m(x)
    assert torch.equal(got, want)
    m.router.data = m.router.data.bfloat16().float()
    want = m(x)
    m.to(BF16)
    got = m(x)
    assert torch.equal(got, want)
    got.float().sum().backward()
    assert m.router.grad.dtype == BF16 and bool(m.router.grad.any())
    status_ok()


def test_calls_and_refusals_keep_no_references(adaln):
    s = make(5)
    r = adaln.adaln_route(s["expert"], 6)
    xs = adaln.adaln_expert_sort_fwd(s["x"], r)
    rng = torch.tensor([1, 2], device="cuda")
    how = dict(gate=s["gate"], seg_id=s["seg"])

    def calls():
        adaln.adaln_dropout_fwd(s["h"], 0.1, rng, x=s["x"], **how)
        adaln.adaln_dropout_bwd(s["dy"], 0.1, rng, h=s["h"], **how)
        work(adaln, s)
        for bad in (lambda: adaln.adaln_dropout_fwd(s["h"], 0.1, (1, "2")),
                    lambda: adaln.adaln_dropout_fwd(s["h"], 0.1, rng, gate=s["gate"]),
                    lambda: adaln.adaln_dropout_fwd(s["h"], "p", rng),
                    lambda: adaln.adaln_dropout_fwd(s["h"], 2.0, rng),
                    lambda: adaln.adaln_dropout_bwd(s["dy"], 0.1, rng, h=s["h"]),
                    lambda: adaln.adaln_route(s["expert"], 0),
                    lambda: adaln.adaln_route(s["expert"], "6"),
                    lambda: adaln.adaln_expert_sort_fwd(s["x"], r[:4]),
                    lambda: adaln.adaln_expert_sort_fwd(s["x"], r._replace(row=3)),
                    lambda: adaln.adaln_expert_combine_fwd(xs, s["weight"].half(), r),
                    lambda: adaln.adaln_expert_combine_bwd(s["dy"], xs[1:], s["weight"], r),
                    lambda: adaln.adaln_experts_ffn_fwd(xs, s["w"][0], s["w"][1], s["w"][1], r.starts),
                    lambda: adaln.adaln_experts_ffn_bwd(xs, xs, *s["w"], r.starts, None)):
            with pytest.raises((AttributeError, TypeError, ValueError, adaln.AdalnError)):
                bad()

    tensors = [rng, xs, r.row, r.starts, r.counts, *s["w"], *(v for v in s.values() if torch.is_tensor(v))]

    def state():
        torch.cuda.synchronize()
        gc.collect()
        return (torch.cuda.memory_allocated(), *map(sys.getrefcount, (
            *tensors, torch.float32, torch.bfloat16, torch.int32, torch.int64, torch.uint8, adaln.AdalnError)))

    calls()
    before = state()
    for _ in range(10):
        calls()
    assert state() == before


def test_gradients_of_shared_leaves_add_up(adaln):
    """The same experts and tokens used twice in one graph, and a gate used by two
    branches: gradients are the sums of those of each use."""
    from adaln_video_dit_gb300.autograd import MixtureFFN, gated_residual
    torch.manual_seed(4)
    m = MixtureFFN(64, 128, 3, device="cuda")
    x = torch.randn(50, 64, device="cuda", dtype=BF16, requires_grad=True)
    gate = torch.randn(1, 64, device="cuda", requires_grad=True)
    seg = torch.zeros(50, dtype=torch.int32, device="cuda")
    # Each of these is used once in `once`, so its two gradients meet in one sum.  (x is
    # used four times, in bf16: its parts are rounded as often and cancel in between.)
    leaves = [gate, *m.parameters()]

    def once(scale):
        h = m(x * scale).float()
        return gated_residual(x.float(), h, gate, seg, 0.25, (1, int(scale))).square().sum()

    parts = [torch.autograd.grad(once(s), leaves) for s in (1.0, 2.0)]
    both = torch.autograd.grad(once(1.0) + once(2.0), leaves)
    for a, b, c in zip(*parts, both):  # (one rounding of the sum)
        total = a.double() + b.double()
        assert bool(((total - c.double()).abs() <= torch.finfo(c.dtype).eps / 2 * total.abs() + 1e-30).all())
    status_ok()


def test_a_mixtures_step_under_anomaly_detection(adaln):
    """With NaN in all memory that is allocated, anomaly detection finds none in a step's
    gradients, sorted ones among them, and the step's bits are those without it."""
    from adaln_video_dit_gb300.autograd import MixtureFFN
    torch.manual_seed(8)
    m = MixtureFFN(64, 96, 4, device="cuda")
    x = torch.randn(37, 64, device="cuda", dtype=BF16, requires_grad=True)

    def step():
        y = m(x)
        return [y.detach(), *torch.autograd.grad(y.float().square().sum(), [x, *m.parameters()])]

    want = step()
    torch.use_deterministic_algorithms(True, warn_only=True)  # (fills what is allocated)
    try:
        assert bool(torch.empty(1000, device="cuda").isnan().all())
        with torch.autograd.detect_anomaly():
            got = step()
    finally:
        torch.use_deterministic_algorithms(False)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    status_ok()
