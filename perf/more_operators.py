"""Cases of the residual branch of a video DiT block whose feed-forward is a mixture
of experts.

Three operators that stand between the modulated tokens and the residual stream:

  res_*, drop_*  dropout from a counter-based generator, whose mask is never stored,
                 with the adaLN-Zero gate of the token's segment and the residual
                 (res_*: y = x + gate[seg] * drop(h)) or on its own (drop_*);
  sort_*         tokens sorted by expert, and the experts' outputs brought back with
                 the router's weights applied;
  experts_*      the gated feed-forward of each expert on its rows,
                 y = (act(x Wg') * (x Wu')) Wd'.

Each case is one use as a program makes it: `*_fwd` the forward, `*_step` a forward
and its backward.  `run` computes it in a plain form (32-bit torch operations,
rounded once at the end), or, where `own` is true, with this library's entry points.
`exact` computes it in 64 bits.

The generator is Philox-4x32 with 10 rounds (Salmon, Moraes, Dror, Shaw: "Parallel
random numbers: as easy as 1, 2, 3", 2011).  Elements 8 c .. 8 c + 7 of token t take
the eight 16-bit parts, lowest first, of its output at key = seed and counter =
(t ceil(D / 8) + c, offset); an element is dropped where its part is below
round(65536 p), and the others are divided by the share that is kept.

A sorted array holds expert 0's rows first, in the order of their (token, choice)
pairs, then expert 1's, each expert's start rounded up to a multiple of 64 rows; the
rows between are zeros, and those past the last expert's, up to what any choices might
need, are left as they were (zeros here).  Expert -1 marks a choice that goes nowhere (a
padded token).
"""
import math

import numpy as np
import torch

own = False

ALIGN = 64
ACTS = ("silu", "gelu_tanh", "gelu")
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _res(name, op, T, D, nseg=1, p=0.1, dtype="bf16"):
    c = dict(op=op, T=T, D=D, nseg=nseg, p=p, dtype=dtype)
    return dict(c, name=name) if name else c


def _sort(name, op, T, D, E, k, padded=0.0, dtype="bf16"):
    c = dict(op=op, T=T, D=D, E=E, k=k, padded=padded, dtype=dtype)
    return dict(c, name=name) if name else c


def _experts(name, op, T, D, F, E, k, act="silu"):
    c = dict(op=op, T=T, D=D, F=F, E=E, k=k, act=act, padded=0.0, dtype="bf16")
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token's residual: the latency of a call
        _res("res_token_f32", "res_fwd", 1, 128, dtype="f32"),
        # the long-video bucket's residual in training: 21 x 30 x 52 tokens, one segment
        _res("res_long_step", "res_step", 32760, 5120),
        # small images and clips packed, a ragged row width, fp32
        _res("res_mixed_f32_step", "res_step", 5003, 1000, nseg=37, p=0.3, dtype="f32"),
        # plain dropout on the hidden values of two samples of 4096 tokens
        _res("drop_hidden_step", "drop_step", 8192, 4096, p=0.2),
        # one token to its experts and back
        _sort("sort_token", "sort_fwd", 1, 1536, 8, 2),
        # a training step at D = 1536: two samples of 4096 tokens
        _sort("sort_1536_step", "sort_step", 8192, 1536, 16, 2),
        # many small experts, a ragged batch with padded tokens, fp32
        _sort("sort_ragged_f32_step", "sort_step", 1111, 1000, 64, 6, padded=0.1, dtype="f32"),
        # the long-video bucket in training
        _sort("sort_long_step", "sort_step", 32760, 5120, 8, 2),
        # a few tokens: the weights of the experts they meet are read once
        _experts("experts_few", "experts_fwd", 8, 1536, 4096, 8, 2),
        # a training step at sizes that no tile divides
        _experts("experts_ragged_step", "experts_step", 1111, 1000, 2728, 16, 2, "gelu_tanh"),
        # a training step at D = 1536
        _experts("experts_1536_step", "experts_step", 8192, 1536, 4096, 8, 2),
        # the long-video bucket's forward
        _experts("experts_long", "experts_fwd", 32760, 5120, 13824, 8, 2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("res", "sort", "experts"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if kind == "experts":
        op = rng.choice(("experts_fwd", "experts_step"))
        D = 8 * _log(rng, 16, 640)
        F = 8 * max(8, min(1728, int(D * rng.choice((1 / 3, 4 / 3, 8 / 3)) / 8) + rng.randint(0, 8)))
        E = min(_log(rng, 2, 96), max(2, 8 * 5120 * 13824 // (D * F)))
        k = rng.randint(1, min(8, E))
        most = 2 * 32760 * 5120 * 13824 // (3 * k if op == "experts_step" else k)
        return _experts(None, op, max(1, min(_log(rng, 1, 32760), most // (D * F))), D, F, E, k,
                        rng.choice(ACTS))
    D = 8 * _log(rng, 8, 640) + (4 if dtype == "f32" and rng.random() < 0.5 else 0)
    if dtype == "f32":
        D = min(D, 4096)
    if kind == "sort":
        E = _log(rng, 1, 256)
        k = rng.randint(1, min(8, E))
        T = min(_log(rng, 1, 65536), 2 * 32760 * 5120 // (k * D * (2 if dtype == "f32" else 1)))
        return _sort(None, rng.choice(("sort_fwd", "sort_step")), T, D, E, k,
                     rng.choice((0.0, 0.0, 0.2)), dtype)
    T = min(_log(rng, 1, 262144), 32760 * 5120 // (D * (2 if dtype == "f32" else 1)))
    op = rng.choice(("res_fwd", "res_step", "res_step", "drop_step"))
    nseg = 1 if op == "drop_step" or rng.random() < 0.3 else _log(rng, 1, max(2, T // 8))
    return _res(None, op, T, D, nseg, round(rng.uniform(0.0, 0.5), 3), dtype)


# ----- inputs ---------------------------------------------------------------------


def _choices(c, g):
    """int32 [T, k]: distinct experts of every token, the most likely first under
    logits that favour some experts over others; -1 for a padded token's."""
    logits = torch.randn(c["T"], c["E"], device="cuda", generator=g)
    logits += 0.7 * torch.randn(c["E"], device="cuda", generator=g)
    score, expert = logits.topk(c["k"], dim=1)
    gone = torch.rand(c["T"], device="cuda", generator=g) < c["padded"]
    return torch.where(gone[:, None], -1, expert).int().contiguous(), score.softmax(1).contiguous()


def _layout(expert, E):
    """(row [T, k], starts [E + 1], counts [E]) of a sorted array."""
    e = expert.reshape(-1).long()
    counts = (e[:, None] == torch.arange(E, device=e.device)).sum(0)
    starts = torch.zeros(E + 1, dtype=torch.long, device=e.device)
    starts[1:] = ((counts + ALIGN - 1) // ALIGN * ALIGN).cumsum(0)
    order = torch.where(e < 0, E, e).argsort(stable=True)
    at = torch.empty_like(order)
    at[order] = torch.arange(len(e), device=e.device)
    row = starts[e.clamp(min=0)] + at - (counts.cumsum(0) - counts)[e.clamp(min=0)]
    row = torch.where(e < 0, -1, row).reshape(expert.shape)
    return row.int(), starts.int(), counts.int()


def _capacity(c):
    """Rows that a sorted array may take whatever the choices are."""
    pairs = c["T"] * c["k"]
    return (pairs + min(c["E"], pairs) * (ALIGN - 1)) // ALIGN * ALIGN


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def n(*shape, std=1.0):
        return (torch.randn(*shape, device=dev, generator=g) * std).to(dt)

    T, D, op, s = case["T"], case["D"], case["op"], {"case": case}
    if op.startswith(("res", "drop")):
        s["rng"] = torch.tensor([seed * 0x9E3779B97F4A7C15 % (1 << 63), seed % 1000], device=dev)
        s["h"] = n(T, D)
        if op != "res_fwd":
            s["dy"] = n(T, D, std=1e-2)
        if op.startswith("res"):
            s["x"], s["gate"] = n(T, D), n(case["nseg"], D, std=0.5)
            ends = torch.rand(case["nseg"] - 1, device=dev, generator=g).mul(T + 1).long().sort()[0]
            s["seg"] = torch.bucketize(torch.arange(T, device=dev), ends, right=True).int()
        return s
    expert, weight = _choices(case, g)
    row, starts, counts = _layout(expert, case["E"])
    rows = _capacity(case)
    kept_rows = [torch.zeros(rows, D, device=dev, dtype=dt) for _ in range(2)]  # for sorted outputs
    if op.startswith("sort"):
        s["expert"], s["weight"] = expert, weight
        s["x"], s["ys"] = n(T, D), n(rows, D)
        s["xs"] = kept_rows[0]
        if op == "sort_step":
            s["dy"], s["dxs"], s["dys"] = n(T, D, std=1e-2), n(rows, D, std=1e-2), kept_rows[1]
        return s
    s["ys"] = kept_rows[0]
    E, F = case["E"], case["F"]
    s["starts"], s["most"] = starts, int(counts.max())
    tokens, kept = torch.arange(T, device=dev).repeat_interleave(case["k"]), row.reshape(-1) >= 0
    at = row.reshape(-1)[kept].long()
    s["xs"] = torch.zeros(rows, D, device=dev, dtype=dt)
    s["xs"][at] = n(T, D)[tokens[kept]]
    s["wg"], s["wu"] = n(E, F, D, std=D ** -0.5), n(E, F, D, std=D ** -0.5)
    s["wd"] = n(E, D, F, std=F ** -0.5)
    if op == "experts_step":
        s["dxs"] = kept_rows[1]
        s["dys"] = torch.zeros(rows, D, device=dev, dtype=dt)
        s["dys"][at] = n(len(at), D, std=1e-2)
    return s


# ----- the plain forms --------------------------------------------------------------


def _philox(counter, offset, seed):
    """Four int64 tensors of 32-bit outputs for the counters of an int64 tensor."""
    low = 0xFFFFFFFF
    c = [counter & low, counter >> 32, offset & low, offset >> 32 & low]
    k0, k1 = seed & low, seed >> 32 & low
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]  # modulo 2^64: the bits are right
        c = [(b >> 32 & low) ^ c[1] ^ k0, b & low, (a >> 32 & low) ^ c[3] ^ k1, a & low]
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    return c


def _kept(s):
    """(truth values [T, D] of what is kept, the factor that makes up for the rest)."""
    c = s["case"]
    T, D, parts = c["T"], c["D"], (c["D"] + 7) // 8
    drop = math.floor(65536 * c["p"] + 0.5)
    words = _philox(torch.arange(T * parts, device="cuda"), s["rng"][1], s["rng"][0])
    bits = torch.stack([w >> 16 * i & 0xFFFF for w in words for i in range(2)], 1)
    return bits.reshape(T, 8 * parts)[:, :D] >= drop, 65536 / max(1, 65536 - drop)


def _run_residual(s):
    c = s["case"]
    dt, seg = s["h"].dtype, s["seg"].long() if "seg" in s else None
    keep, factor = _kept(s)
    h = torch.where(keep, s["h"].float() * factor, 0.0)
    if c["op"] == "drop_step":
        return [h.to(dt), torch.where(keep, s["dy"].float() * factor, 0.0).to(dt)]
    gate = s["gate"].float()
    y = (s["x"].float() + gate[seg] * h).to(dt)
    if c["op"] == "res_fwd":
        return [y]
    dy = s["dy"].float()
    dgate = torch.zeros_like(gate).index_add_(0, seg, dy * h)
    return [y, torch.where(keep, gate[seg] * dy * factor, 0.0).to(dt), dgate]


def _run_sort(s):
    dt = s["x"].dtype
    row, starts, counts = _layout(s["expert"], s["case"]["E"])
    kept, at = (row >= 0)[..., None], row.clamp(min=0).long()
    tokens, pairs = kept.nonzero()[:, 0], at[row >= 0]
    xs = torch.zeros_like(s["ys"])
    xs[pairs] = s["x"][tokens]
    ys = torch.where(kept, s["ys"][at].float(), 0.0)
    out = [row, starts, counts, xs, (s["weight"][..., None] * ys).sum(1).to(dt)]
    if s["case"]["op"] == "sort_fwd":
        return out
    dx = torch.where(kept, s["dxs"][at].float(), 0.0).sum(1).to(dt)
    dy = s["dy"].float()[:, None]
    dys = torch.zeros_like(xs)
    dys[pairs] = (s["weight"][..., None] * dy).to(dt)[row >= 0]
    return out + [dx, dys, (dy * ys).sum(2)]


def _act(act, g):
    """act(g) and act'(g)."""
    if act == "silu":
        q = torch.sigmoid(g)
        return g * q, q * (1 + g * (1 - q))
    if act == "gelu":
        q = 0.5 * torch.erfc(-g * math.sqrt(0.5))
        return g * q, q + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    a = 2 * math.sqrt(2 / math.pi)
    q = torch.sigmoid(a * (g + 0.044715 * g * g * g))
    return g * q, q + g * q * (1 - q) * a * (1 + 3 * 0.044715 * g * g)


def _run_experts(s):
    """Every expert's rows side by side, as many as the largest has; rows past an
    expert's own are zeros, and what they give goes nowhere."""
    c, dt = s["case"], s["xs"].dtype
    starts = s["starts"].long()
    deep = -(-s["most"] // ALIGN) * ALIGN
    rows = starts[:-1, None] + torch.arange(deep, device="cuda")
    mine = rows < starts[1:, None]
    at = rows[mine]
    rows = torch.where(mine, rows, 0)

    def spread(t):
        return torch.where(mine[..., None], t[rows], 0.0)

    x, wg, wu, wd = spread(s["xs"].float()), s["wg"].float(), s["wu"].float(), s["wd"].float()
    g, u = x @ wg.transpose(1, 2), x @ wu.transpose(1, 2)
    a, da = _act(c["act"], g)
    ys = torch.zeros_like(s["xs"])
    ys[at] = ((a * u) @ wd.transpose(1, 2))[mine].to(dt)
    if c["op"] == "experts_fwd":
        return [ys]
    dy = spread(s["dys"].float())
    dh = dy @ wd
    dg, du = dh * u * da, dh * a
    dxs = torch.zeros_like(ys)
    dxs[at] = (dg @ wg + du @ wu)[mine].to(dt)
    return [ys, dxs, (dg.transpose(1, 2) @ x).to(dt), (du.transpose(1, 2) @ x).to(dt),
            (dy.transpose(1, 2) @ (a * u)).to(dt)]


# ----- the library's calls ------------------------------------------------------------


def _own(s):
    from adaln_video_dit_gb300 import _lib as L
    c, op = s["case"], s["case"]["op"]
    if op.startswith(("res", "drop")):
        how = dict(p=c["p"], rng=s["rng"], gate=s.get("gate"), seg_id=s.get("seg"))
        y = L.adaln_dropout_fwd(s["h"], x=s.get("x"), **how)
        if op == "res_fwd":
            return [y]
        dh, dgate = L.adaln_dropout_bwd(s["dy"], h=s["h"] if op == "res_step" else None, **how)
        return [y, dh] + ([dgate] if op == "res_step" else [])
    if op.startswith("sort"):
        r = L.adaln_route(s["expert"], c["E"], align=ALIGN)
        out = [r.row, r.starts, r.counts, L.adaln_expert_sort_fwd(s["x"], r, xs=s["xs"]),
               L.adaln_expert_combine_fwd(s["ys"], s["weight"], r)]
        if op == "sort_fwd":
            return out
        dx = L.adaln_expert_sort_bwd(s["dxs"], r)
        dys, dw = L.adaln_expert_combine_bwd(s["dy"], s["ys"], s["weight"], r, dys=s["dys"])
        return out + [dx, dys, dw]
    x, weights, act = s["xs"], (s["wg"], s["wu"], s["wd"]), c["act"]
    if op == "experts_fwd":
        return [L.adaln_experts_ffn_fwd(x, *weights, s["starts"], act=act, ys=s["ys"])[0]]
    ys, saved = L.adaln_experts_ffn_fwd(x, *weights, s["starts"], act=act, save=True, ys=s["ys"])
    return [ys, *L.adaln_experts_ffn_bwd(s["dys"], x, *weights, s["starts"], saved, act=act, dxs=s["dxs"])]


def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    return (_run_experts if op.startswith("experts") else
            _run_sort if op.startswith("sort") else _run_residual)(s)


# ----- in 64 bits ------------------------------------------------------------------------


def _exact_bits(c, rng):
    """The generator's 16-bit parts, [T, D], with numpy's unsigned 64-bit arithmetic."""
    u64, low = np.uint64, np.uint64(0xFFFFFFFF)
    parts = (c["D"] + 7) // 8
    at = np.arange(c["T"] * parts, dtype=u64)
    seed, offset = (int(v) for v in rng.tolist())
    x = [at & low, at >> u64(32), np.full_like(at, offset & 0xFFFFFFFF), np.full_like(at, offset >> 32)]
    for i in range(10):
        a, b = x[0] * u64(0xD2511F53), x[2] * u64(0xCD9E8D57)
        key = (seed + i * 0x9E3779B9) & 0xFFFFFFFF, ((seed >> 32) + i * 0xBB67AE85) & 0xFFFFFFFF
        x = [b >> u64(32) ^ x[1] ^ u64(key[0]), b & low, a >> u64(32) ^ x[3] ^ u64(key[1]), a & low]
    words = np.stack([w.astype("<u4") for w in x], 1)
    return words.view("<u2").reshape(c["T"], 8 * parts)[:, :c["D"]]


def _exact_residual(c, s):
    drop = int(np.floor(np.float64(c["p"]) * 65536 + 0.5))
    kept = torch.from_numpy((_exact_bits(c, s["rng"]) >= drop).astype(np.uint8)).cuda().double()
    m = kept * (65536.0 / max(65536 - drop, 1))
    if c["op"] == "drop_step":
        return [m * s["h"].double(), m * s["dy"].double()]
    gate = s["gate"].double()[s["seg"].long()]
    y = torch.addcmul(s["x"].double(), gate * m, s["h"].double())
    if c["op"] == "res_fwd":
        return [y]
    each = m.mul_(s["dy"].double())
    dh = gate * each
    total = (each * s["h"].double()).cumsum(0)
    ends = torch.searchsorted(s["seg"].long(), torch.arange(c["nseg"], device="cuda"), right=True)
    total = torch.cat([torch.zeros_like(total[:1]), total])[ends]
    return [y, dh, torch.diff(total, dim=0, prepend=torch.zeros_like(total[:1]))]


def _exact_sort(c, s):
    """Pair by pair on the host for the layout; one-hot products for the rest."""
    expert = s["expert"].cpu().numpy()
    counts = np.bincount(expert[expert >= 0].reshape(-1), minlength=c["E"])
    starts = np.concatenate([[0], np.cumsum(-(-counts // ALIGN) * ALIGN)])
    row = np.full(expert.shape, -1)
    for e in range(c["E"]):
        row[expert == e] = starts[e] + np.arange(counts[e])
    source = np.full(len(s["ys"]), -1)
    t, j = np.nonzero(row >= 0)
    source[row[t, j]] = t
    source = torch.from_numpy(source).cuda()
    at, there = torch.from_numpy(row).cuda(), torch.from_numpy(row >= 0).cuda()
    w = s["weight"].double() * there

    def take(x, rows, factor):
        return x.double()[rows.clamp(min=0)] * factor[:, None]

    used = (source >= 0).double()
    y = sum(take(s["ys"], at[:, i], w[:, i]) for i in range(c["k"]))
    out = [None, None, None, take(s["x"], source, used), y]
    if c["op"] == "sort_fwd":
        return out
    dx = sum(take(s["dxs"], at[:, i], there[:, i].double()) for i in range(c["k"]))
    of_row = torch.zeros(len(s["ys"]), dtype=torch.float64, device="cuda")
    of_row[at[there]] = s["weight"].double()[there]
    dw = torch.stack([(take(s["ys"], at[:, i], there[:, i].double()) * s["dy"].double()).sum(1)
                      for i in range(c["k"])], 1)
    return out + [dx, take(s["dy"], source, of_row), dw]


def _exact_experts(c, s):
    step = c["op"] == "experts_step"
    parts = []
    act = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
           "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[c["act"]]
    edges = s["starts"].tolist()
    for e in range(c["E"]):
        lo, hi = edges[e], edges[e + 1]
        leaves = [t.double().requires_grad_(step) for t in (s["xs"][lo:hi], s["wg"][e], s["wu"][e], s["wd"][e])]
        x, wg, wu, wd = leaves
        y = torch.mm(act(torch.mm(x, wg.t())) * torch.mm(x, wu.t()), wd.t())
        grads = torch.autograd.grad(y, leaves, s["dys"][lo:hi].double()) if step else ()
        parts.append((y.detach(), *grads))
    left = s["xs"][edges[-1]:].double()  # past the last expert's rows: zeros
    return [torch.cat([*p, left]) if i < 2 else torch.stack(p) for i, p in enumerate(zip(*parts))]


def exact(case, seed):
    if case["op"].startswith("experts") and work(case)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    return (_exact_experts if case["op"].startswith("experts") else
            _exact_sort if case["op"].startswith("sort") else _exact_residual)(case, s)


# ----- what a pass cannot do without ---------------------------------------------------------


def work(case):
    T, D, op = case["T"], case["D"], case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op.startswith(("res", "drop")):
        # h (and x, the gate, the segments); y; then dy (and h); dh (and dgate)
        many = {"res_fwd": 3, "res_step": 6, "drop_step": 4}[op]
        gates = case["nseg"] * D * (e + 4 * (op == "res_step")) if op != "drop_step" else 0
        return {"bytes": many * T * D * e + gates + (4 * T if gates else 0), "flops": 2 * many * T * D}
    k = case["k"]
    if op.startswith("sort"):
        # the choices, weights and places; x and the sorted rows; the experts' rows and y;
        # then dxs, dx, dy, the experts' rows, dys and the weights' gradients
        fwd, bwd = (2 + 2 * k) * T * D * e + 12 * T * k, (2 + 3 * k) * T * D * e + 4 * T * k
        step = op == "sort_step"
        return {"bytes": fwd + step * bwd, "flops": (2 + 4 * step) * T * k * D}
    F, R = case["F"], T * k
    met = min(case["E"], R)  # experts whose weights are read, at most
    if op == "experts_fwd":
        return {"bytes": e * (2 * R * D + 3 * met * D * F), "flops": 6 * R * D * F}
    return {"bytes": e * (4 * R * D + 3 * (met + case["E"]) * D * F), "flops": 18 * R * D * F}
