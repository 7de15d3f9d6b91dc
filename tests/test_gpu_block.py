"""The operators as autograd nodes, and together in the example block."""
import importlib.util
import os

import pytest
import torch

from gpu_helpers import status_ok

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("dit_block",
                                                  os.path.join(ROOT, "examples", "dit_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_qk_norm_rope_node_is_the_calls(adaln):
    from adaln_video_dit_gb300 import autograd as A
    from adaln_video_dit_gb300 import rotary
    T, h, dh = 50, 4, 64
    qkv = torch.randn(T, 3, h, dh, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    wq = torch.randn(dh, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    wk = torch.randn(dh, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    pairs = rotary.split_pairs(dh // 2)
    table = rotary.rope_table(10, pairs, device="cuda")
    pos = rotary.grid_positions([(2, 2, 4, 6)], device="cuda")
    q, k, _ = qkv.unbind(1)
    qo, ko = A.qk_norm_rope(q, k, wq, wk, table, pos, pairs)
    dqo, dko = torch.randn_like(qo), torch.randn_like(ko)
    (qo * dqo + ko * dko).float().sum().backward()
    with torch.no_grad():
        q, k, _ = qkv.unbind(1)
        want = adaln.adaln_qk_rope_fwd(q, k, table, pos, pairs, norm=True, wq=wq, wk=wk)
        dq, dk, dwq, dwk = adaln.adaln_qk_rope_bwd(dqo, dko, table, pos, pairs, norm=True, q=q, k=k,
                                                   wq=wq, wk=wk)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    assert torch.equal(qkv.grad[:, 0], dq) and torch.equal(qkv.grad[:, 1], dk)
    assert not qkv.grad[:, 2].any()
    assert torch.equal(wq.grad, dwq.bfloat16()) and torch.equal(wk.grad, dwk.bfloat16())
    # plain rotation: its gradient turns back, so q comes back to a bf16 rounding
    x = torch.randn(T, h, dh, device="cuda", requires_grad=True)
    y, _ = A.qk_rope(x, x, table, pos, pairs, interleaved=False)
    (y * y.detach()).sum().backward()
    assert float((x.grad - x.detach()).abs().max()) < 1e-5
    z, none = A.qk_rope(x, None, table, pos, pairs, interleaved=False)  # queries alone
    z.sum().backward()
    assert none is None and torch.equal(z, y)
    status_ok()


def test_gated_ffn_node_is_the_calls(adaln):
    from adaln_video_dit_gb300 import autograd as A
    m = A.GatedFFN(96, 160, act="gelu", device="cuda")
    x = torch.randn(3, 21, 96, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    y = m(x)
    dy = torch.randn_like(y)
    y.backward(dy)
    x2 = x.detach().reshape(-1, 96)
    want, saved = adaln.adaln_ffn_fwd(x2, m.wg, m.wu, m.wd, act="gelu", save=True)
    grads = adaln.adaln_ffn_bwd(dy.reshape(-1, 96), x2, m.wg, m.wu, m.wd, saved, act="gelu")
    assert torch.equal(y.reshape(-1, 96), want)
    for got, ref in zip((x.grad.reshape(-1, 96), m.wg.grad, m.wu.grad, m.wd.grad), grads):
        assert torch.equal(got, ref)
    with torch.no_grad():
        assert torch.equal(m(x), y)
    with pytest.raises(ValueError):
        A.GatedFFN(8, 8, act="relu", device="cuda")
    status_ok()


def test_example_block_trains(adaln):
    losses = example().main(["--dim", "256", "--heads", "4", "--hidden", "512", "--steps", "8"])
    assert all(map(lambda v: v == v, losses))
    assert losses[-1] < losses[0]
    status_ok()


def test_calls_and_refusals_keep_no_references(adaln):
    """The compiled marshalling owns what it takes and no more: after many calls,
    refused ones among them, no tensor and no byte of device memory is left over."""
    import gc
    import sys

    q = torch.randn(4, 2, 64, device="cuda")
    table = torch.zeros(3, 32, 2, device="cuda")
    pos = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    x = torch.randn(4, 64, device="cuda").bfloat16()
    w = [torch.randn(*s, device="cuda").bfloat16() for s in ((96, 64), (96, 64), (64, 96))]

    def calls():
        adaln.adaln_qk_rope_fwd(q, q, table, pos, (32,))
        adaln.adaln_qk_rope_bwd(q, q, table, pos, (32,), norm=True, q=q, k=q)
        _, saved = adaln.adaln_ffn_fwd(x, *w, save=True)
        adaln.adaln_ffn_bwd(x, x, *w, saved)
        for bad in (lambda: adaln.adaln_qk_rope_fwd(q.half(), None, table, pos, (32,)),
                    lambda: adaln.adaln_qk_rope_fwd(q, None, table, pos, (31,)),
                    lambda: adaln.adaln_qk_rope_fwd(q, None, table, pos, 7),
                    lambda: adaln.adaln_qk_rope_fwd(q, "no tensor", table, pos, (32,)),
                    lambda: adaln.adaln_qk_rope_fwd(q, None, table, pos, (32,), norm=True, eps=-1.0),
                    lambda: adaln.adaln_qk_rope_bwd(q, q, table, pos, (32,), norm=True, q=q),
                    lambda: adaln.adaln_ffn_fwd(x, w[0], w[1], w[1]),
                    lambda: adaln.adaln_ffn_fwd(x.float(), *(t.float() for t in w)),
                    lambda: adaln.adaln_ffn_bwd(x, x, *w, None)):
            with pytest.raises((AttributeError, TypeError, ValueError, adaln.AdalnError)):
                bad()

    def state():
        torch.cuda.synchronize()
        gc.collect()
        return (torch.cuda.memory_allocated(), *map(sys.getrefcount, (
            q, table, pos, x, *w, torch.float32, torch.bfloat16, torch.uint8, adaln.AdalnError)))

    calls()
    before = state()
    for _ in range(20):
        calls()
    assert state() == before


def test_calls_from_two_threads_on_two_streams(adaln):
    """Both operators at once on two streams, each thread with its own tensors:
    every result equals the serial one."""
    import threading

    def make(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()  # noqa: E731
        return dict(q=r(900, 6, 64), k=r(900, 2, 64), dq=r(900, 6, 64), dk=r(900, 2, 64),
                    w=r(64), table=torch.randn(9, 32, 2, device="cuda", generator=g),
                    pos=torch.randint(-1, 9, (900, 1), device="cuda", generator=g).int(),
                    x=[r(t, 256) for t in (1, 20, 300)], dy=[r(t, 256) for t in (1, 20, 300)],
                    ffn=(r(512, 256), r(512, 256), r(256, 512)))

    def work(s):
        out = [*adaln.adaln_qk_rope_fwd(s["q"], s["k"], s["table"], s["pos"], (32,), norm=True,
                                        wq=s["w"])]
        out += adaln.adaln_qk_rope_bwd(s["dq"], s["dk"], s["table"], s["pos"], (32,), norm=True,
                                       q=s["q"], k=s["k"], wq=s["w"])
        for x, dy in zip(s["x"], s["dy"]):
            y, saved = adaln.adaln_ffn_fwd(x, *s["ffn"], save=True)
            out += [y, *adaln.adaln_ffn_bwd(dy, x, *s["ffn"], saved)]
        return out

    states = [make(1), make(2)]
    want = [[t.clone() for t in work(s)] for s in states]
    torch.cuda.synchronize()
    wrong = []

    def run(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(15):
                    got = work(states[i])
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
    """Each call on a stream that is busy, given as an argument; the current
    stream then overwrites whatever memory its allocator has free."""
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()  # noqa: E731
    q, dq, w = r(900, 6, 64), r(900, 6, 64), r(64)
    table, pos = torch.randn(9, 32, 2, device="cuda", generator=g), torch.zeros(
        900, 1, dtype=torch.int32, device="cuda")
    x, dy, ffn = r(300, 256), r(300, 256), (r(512, 256), r(512, 256), r(256, 512))
    saved = adaln.adaln_ffn_fwd(x, *ffn, save=True)[1]
    calls = [lambda s: adaln.adaln_qk_rope_fwd(q, None, table, pos, (32,), norm=True, wq=w, stream=s),
             lambda s: adaln.adaln_qk_rope_bwd(dq, None, table, pos, (32,), norm=True, q=q, wq=w,
                                               stream=s),
             lambda s: adaln.adaln_ffn_fwd(x, *ffn, save=True, stream=s)[:1],
             lambda s: adaln.adaln_ffn_bwd(dy, x, *ffn, saved, stream=s)]
    side, busy = torch.cuda.Stream(), r(4096, 4096)
    for call in calls:
        want = [t for t in call(None) if t is not None]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(20):
                busy @ busy
        got = [t for t in call(side) if t is not None]
        junk = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
                for n in (512, 4096, 1 << 17, 1 << 19, 1 << 20, 3 << 20, 8 << 20) for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        del junk
    status_ok()


TWO_THREADS = r"""
#include <thread>
#include "adaln.h"
struct Call {
  adaln_heads_t in, out;
  int32_t heads;
  void* stream;
};
// `times` forward calls of each on a thread of its own; how many were refused.
extern "C" int two_threads(decltype(&adaln_qk_rope_fwd) fwd, const Call* calls, int64_t T, int32_t dh,
                           const adaln_rope_t* rope, const void* w, int times) {
  int refused[2] = {};
  auto run = [&](int i) {
    const Call& c = calls[i];
    for (int n = 0; n < times; ++n)
      refused[i] += fwd(&c.in, nullptr, T, c.heads, 0, dh, ADALN_BF16, rope, 1, w, nullptr, 1e-6f,
                        &c.out, nullptr, c.stream) != ADALN_OK;
  };
  std::thread a(run, 0), b(run, 1);
  a.join();
  b.join();
  return refused[0] + refused[1];
}
"""


def test_calls_of_two_sizes_from_two_threads(adaln, tmp_path):
    """Calls that share a kernel but need different amounts of shared memory (one
    and two heads, several tokens to a warp: 98,816 and 49,664 bytes), from two
    native threads at once (Python's would take turns): every launch is allowed
    its own."""
    import ctypes
    import subprocess

    (tmp_path / "two.cpp").write_text(TWO_THREADS)
    so = str(tmp_path / "two.so")
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-shared", "-fPIC", "-pthread",
                    "-I" + os.path.join(ROOT, "include"), str(tmp_path / "two.cpp"), "-o", so],
                   check=True)
    two = ctypes.CDLL(so).two_threads

    class Call(ctypes.Structure):
        _fields_ = [("inp", adaln.Heads), ("out", adaln.Heads), ("heads", ctypes.c_int32),
                    ("stream", ctypes.c_void_p)]

    T, dh = 5000, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()  # noqa: E731
    table = torch.randn(9, 64, 2, device="cuda", generator=g)
    pos = torch.randint(-1, 9, (T, 1), device="cuda", generator=g).int()
    w = r(dh)
    rope = adaln.Rope(table.data_ptr(), pos.data_ptr(), 9, 1, (ctypes.c_int32 * 4)(64, 0, 0, 0), 1)
    q = [r(T, h, dh) for h in (1, 2)]
    out = [torch.zeros_like(t) for t in q]
    streams = [torch.cuda.Stream() for _ in q]
    heads = lambda t: adaln.Heads(t.data_ptr(), t.stride(0), t.stride(1))  # noqa: E731
    calls = (Call * 2)(*(Call(heads(a), heads(b), a.shape[1], s.cuda_stream)
                         for a, b, s in zip(q, out, streams)))
    want = [adaln.adaln_qk_rope_fwd(t, None, table, pos, (64,), norm=True, wq=w)[0] for t in q]
    torch.cuda.synchronize()
    refused = two(ctypes.cast(adaln.raw.adaln_qk_rope_fwd, ctypes.c_void_p), calls,
                  ctypes.c_int64(T), dh, ctypes.byref(rope), ctypes.c_void_p(w.data_ptr()), 5000)
    torch.cuda.synchronize()
    assert refused == 0
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    status_ok()


def test_rotary_nodes_take_leading_dimensions(adaln):
    from adaln_video_dit_gb300 import autograd as A
    from adaln_video_dit_gb300 import rotary
    B, N, h, dh = 3, 48, 2, 64
    qkv = torch.randn(B, N, 3, h, dh, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(dh, device="cuda", dtype=torch.bfloat16)
    pairs = rotary.split_pairs(dh // 2)
    table = rotary.rope_table(10, pairs, device="cuda")
    pos = rotary.grid_positions([(0, 2, 4, 6)] * B, device="cuda")
    results = []
    for shape, p in (((B, N, 3, h, dh), pos.view(B, N, 3)), ((B * N, 3, h, dh), pos)):
        x = qkv.clone().view(shape).requires_grad_()
        q, k, _ = x.unbind(-3)
        qo, ko = A.qk_norm_rope(q, k, w, w, table, p, pairs)
        assert qo.shape == q.shape and ko.shape == k.shape
        (qo.float().square().sum() + ko.float().sum()).backward()
        results.append([t.reshape(-1) for t in (qo, ko, x.grad)])
    assert all(torch.equal(a, b) for a, b in zip(*results))
    status_ok()


def test_what_an_adaln_call_on_a_given_stream_allocates_is_that_streams(adaln):
    """As above, for the AdaLN's calls."""
    T, D = 900, 256
    g = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()  # noqa: E731
    x, dy, shift, scale, busy = r(T, D), r(T, D), r(2, D), r(2, D), r(4096, 4096)
    seg = (torch.arange(T, device="cuda") >= 400).int()
    _, mean, rstd = adaln.adaln_fwd(x, shift, scale, seg, 1e-6)
    side = torch.cuda.Stream()
    for call in (lambda s: adaln.adaln_fwd(x, shift, scale, seg, 1e-6, stream=s),
                 lambda s: adaln.adaln_bwd(dy, x, mean, rstd, scale, seg, stream=s)):
        want = call(None)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(20):
                busy @ busy
        got = call(side)
        junk = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda")
                for n in (512, 4096, 1 << 17, 1 << 19, 1 << 20, 3 << 20, 8 << 20) for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        del junk
    status_ok()
