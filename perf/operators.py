"""Cases of the attention front end and the feed-forward block of a video DiT.

Three operators that stand beside the fused AdaLN in a transformer block over
packed tokens:

  rope_*  rotary positions over several axes (time, height, width) applied to
          queries and keys;
  qk_*    the same with an RMS norm of every head first, in the same pass;
  ffn_*   the gated feed-forward block y = (act(x Wg') * (x Wu')) Wd'.

Each case is one call as a user makes it: `*_fwd` the forward, `*_bwd` the
backward alone, `*_step` a forward and its backward.  `run` computes it in a
plain form (32-bit torch operations, rounded once at the end), or, where `own`
is true, with this library's entry points.  `exact` computes it in 64 bits.

Positions are those of samples of `text` unrotated tokens (position -1 on
every axis) followed by gf x gh x gw video tokens in raster order, packed back
to back and cut at T tokens.
"""
import math

import torch

own = False

ACTS = ("silu", "gelu_tanh", "gelu")
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _qk(name, op, T, hq, hk, dh, rot, grid, text=0, half=False, dtype="bf16", packed=False):
    c = dict(op=op, T=T, hq=hq, hk=hk, dh=dh, rot=rot, text=text, gf=grid[0], gh=grid[1],
             gw=grid[2], half=half, dtype=dtype, packed=packed)
    return dict(c, name=name) if name else c


def _ffn(name, op, T, D, F, act="silu"):
    c = dict(op=op, T=T, D=D, F=F, act=act, dtype="bf16")
    return dict(c, name=name) if name else c


def listed():
    return [
        # one small fp32 image (256 tokens, D = 128): the latency of a call
        _qk("rope_image_f32", "rope_fwd", 256, 4, 4, 32, 32, (1, 16, 16), dtype="f32"),
        # the rotation's gradient in a joint text + video layer (8 samples of
        # 512 text and 4096 video tokens), halves layout
        _qk("rope_joint_bwd", "rope_bwd", 36864, 24, 24, 128, 128, (16, 16, 16), text=512,
            half=True),
        # a single token on its own
        _qk("qk_token", "qk_fwd", 1, 12, 12, 128, 128, (1, 1, 1)),
        # a training step's front end: two samples of 4096 tokens, D = 1536,
        # read out of the packed q|k|v projection
        _qk("qk_step_1536", "qk_step", 8192, 12, 12, 128, 128, (16, 16, 16), packed=True),
        # the long-video bucket's forward: 21 x 30 x 52 tokens, D = 5120
        _qk("qk_long_video", "qk_fwd", 32760, 40, 40, 128, 128, (21, 30, 52), packed=True),
        # grouped keys, a head width that is no power of two, fp32, ragged T
        _qk("qk_grouped_f32_step", "qk_step", 5003, 32, 8, 80, 80, (5, 25, 40), text=3,
            half=True, dtype="f32"),
        # the feed-forward block of one token: every weight is read once
        _ffn("ffn_token", "ffn_fwd", 1, 1536, 4096),
        # one image's tokens through the widest block
        _ffn("ffn_image", "ffn_fwd", 256, 5120, 13824),
        # a training step at sizes that no tile divides
        _ffn("ffn_ragged_step", "ffn_step", 1111, 1000, 2728, "gelu_tanh"),
        # a training step at D = 1536
        _ffn("ffn_step_1536", "ffn_step", 8192, 1536, 4096),
        # the long-video bucket's forward
        _ffn("ffn_long_video", "ffn_fwd", 32760, 5120, 13824),
        # a training step at D = 5120
        _ffn("ffn_step_5120", "ffn_step", 8192, 5120, 13824, "gelu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        op = rng.choice(("rope_fwd", "rope_bwd", "qk_fwd", "qk_step"))
        dh = rng.choice((32, 64, 72, 80, 96, 128, 128, 192, 256))
        hk = _log(rng, 1, 40)
        hq = hk * rng.choice((1, 1, 2, 3, 4, 8))
        if hq > 64:
            hq = hk
        most = 32760 * 80 * 128 // (3 if op == "qk_step" else 1)
        T = max(1, min(_log(rng, 1, 65536), most // ((hq + hk) * dh)))
        rot = dh if rng.random() < 0.7 else dh // 2
        return _qk(None, op, T, hq, hk, dh, rot,
                   (_log(rng, 1, 24), _log(rng, 1, 64), _log(rng, 1, 64)),
                   text=rng.choice((0, 0, 7, 77, 512)), half=rng.random() < 0.5,
                   dtype=rng.choice(("bf16", "bf16", "f32")), packed=rng.random() < 0.5)
    op = rng.choice(("ffn_fwd", "ffn_fwd", "ffn_step"))
    D = 8 * _log(rng, 16, 640)
    F = 8 * max(8, min(1728, int(D * rng.choice((4 / 3, 8 / 3, 4)) / 8) + rng.randint(0, 8)))
    most = 32760 * 5120 * 13824 // (3 if op == "ffn_step" else 1)
    T = max(1, min(_log(rng, 1, 32760), most // (D * F)))
    return _ffn(None, op, T, D, F, rng.choice(ACTS))


def _axis_pairs(rot):
    """Pairs of the (time, height, width) axes: height and width take a third
    each, time the rest."""
    p = rot // 2
    return (p - 2 * (p // 3), p // 3, p // 3)


def _table(rows, rot, device):
    """(cos, sin) of position * 10000^(-i/n) for pair i of an axis of n pairs:
    [rows, rot/2, 2], computed in 64 bits, held in 32."""
    f = torch.cat([10000.0 ** (-torch.arange(n, dtype=torch.float64) / max(n, 1))
                   for n in _axis_pairs(rot)]).to(device)
    a = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).float()


def _positions(c, device):
    i = torch.arange(c["T"], device=device) % (c["text"] + c["gf"] * c["gh"] * c["gw"]) - c["text"]
    p = torch.stack([i // (c["gh"] * c["gw"]), i // c["gw"] % c["gh"], i % c["gw"]], 1)
    return torch.where(i[:, None] < 0, -1, p).int().contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def n(*shape, std=1.0):
        return torch.randn(*shape, device=dev, generator=g) * std

    T, s = case["T"], {"case": case}
    if case["op"].startswith("ffn"):
        D, F = case["D"], case["F"]
        s["x"] = n(T, D).to(dt)
        s["wg"], s["wu"] = n(F, D, std=D ** -0.5).to(dt), n(F, D, std=D ** -0.5).to(dt)
        s["wd"] = n(D, F, std=F ** -0.5).to(dt)
        if case["op"] == "ffn_step":
            s["dy"] = n(T, D, std=1e-2).to(dt)
        return s
    hq, hk, dh = case["hq"], case["hk"], case["dh"]
    s["table"] = _table(max(case["gf"], case["gh"], case["gw"]), case["rot"], dev)
    s["pos"] = _positions(case, dev)
    s["pairs"] = _axis_pairs(case["rot"])
    s["axis"] = torch.tensor([a for a, m in enumerate(s["pairs"]) for _ in range(m)], device=dev)
    if case["packed"]:  # views of the projection's output, q | k | v
        qkv = n(T, hq + 2 * hk, dh, std=1.5).to(dt)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
    else:
        s["q"], s["k"] = n(T, hq, dh, std=1.5).to(dt), n(T, hk, dh, std=1.5).to(dt)
    if case["op"] in ("rope_bwd", "qk_step"):
        s["dq"], s["dk"] = n(T, hq, dh, std=1e-2).to(dt), n(T, hk, dh, std=1e-2).to(dt)
    if case["op"].startswith("qk"):
        s["wq"], s["wk"] = (1 + n(dh, std=0.1)).to(dt), (1 + n(dh, std=0.1)).to(dt)
    return s


# ----- plain forms -------------------------------------------------------------


def _rows(s):
    """cos and sin of every token and pair, [T, 1, pairs]."""
    axis = s["axis"]
    p = s["pos"].long()[:, axis]
    cs = s["table"][p.clamp(min=0), torch.arange(axis.numel(), device=axis.device)]
    on = p >= 0
    return (torch.where(on, cs[..., 0], 1.0)[:, None], torch.where(on, cs[..., 1], 0.0)[:, None])


def _turn(x, cos, sin, rot, half):
    """The rotation of 32-bit x [T, heads, dh]; minus sin turns it back."""
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., :rot // 2], r[..., rot // 2:]) if half else (r[..., 0::2], r[..., 1::2])
    u, v = a * cos - b * sin, b * cos + a * sin
    r = torch.cat([u, v], -1) if half else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([r, rest], -1)


def _plain_qk(s):
    c = s["case"]
    op, rot, half = c["op"], c["rot"], c["half"]
    dt = DTYPES[c["dtype"]]
    cos, sin = _rows(s)
    if op == "rope_bwd":
        return [_turn(s[n].float(), cos, -sin, rot, half).to(dt) for n in ("dq", "dk")]
    if op == "rope_fwd":
        return [_turn(s[n].float(), cos, sin, rot, half).to(dt) for n in ("q", "k")]
    out, grads = [], []

    def one(x, w, dy):
        x, w = x.float(), w.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        out.append(_turn(x * r * w, cos, sin, rot, half).to(dt))
        if op == "qk_step":
            g = _turn(dy.float(), cos, -sin, rot, half)
            h = g * w
            dx = r * (h - x * r * r * (h * x).mean(-1, keepdim=True))
            grads.extend([dx.to(dt), (g * x * r).sum((0, 1))])

    one(s["q"], s["wq"], s.get("dq"))
    one(s["k"], s["wk"], s.get("dk"))
    return out + grads


def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        p = 1 / (1 + torch.exp(-g))
        return g * p, p * (1 + g * (1 - p))
    if act == "gelu":
        p = 0.5 * (1 + torch.erf(g * 0.5 ** 0.5))
        return g * p, p + g * torch.exp(-0.5 * g * g) * (2 * math.pi) ** -0.5
    k = (2 / math.pi) ** 0.5
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


def _plain_ffn(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    x, wg, wu, wd = (s[n].float() for n in ("x", "wg", "wu", "wd"))
    g, u = x @ wg.t(), x @ wu.t()
    a, da = _act(g, c["act"])
    h = a * u
    y = (h @ wd.t()).to(dt)
    if c["op"] == "ffn_fwd":
        return [y]
    dy = s["dy"].float()
    dh = dy @ wd
    dg, du = dh * u * da, dh * a
    dx = dg @ wg + du @ wu
    return [y, dx.to(dt), (dg.t() @ x).to(dt), (du.t() @ x).to(dt), (dy.t() @ h).to(dt)]


# ----- the library's calls -----------------------------------------------------


def _own(s):
    from adaln_video_dit_gb300 import lib
    L = lib()
    c = s["case"]
    op = c["op"]
    if op.startswith("ffn"):
        w = (s["wg"], s["wu"], s["wd"])
        y, saved = L.adaln_ffn_fwd(s["x"], *w, act=c["act"], save=op == "ffn_step")
        if op == "ffn_fwd":
            return [y]
        return [y, *L.adaln_ffn_bwd(s["dy"], s["x"], *w, saved, act=c["act"])]
    how = dict(axis_pairs=s["pairs"], interleaved=not c["half"])
    if op == "rope_fwd":
        return list(L.adaln_qk_rope_fwd(s["q"], s["k"], s["table"], s["pos"], **how))
    if op == "rope_bwd":
        return list(L.adaln_qk_rope_bwd(s["dq"], s["dk"], s["table"], s["pos"], **how)[:2])
    how.update(norm=True, wq=s["wq"], wk=s["wk"], eps=EPS)
    qo, ko = L.adaln_qk_rope_fwd(s["q"], s["k"], s["table"], s["pos"], **how)
    if op == "qk_fwd":
        return [qo, ko]
    dq, dk, dwq, dwk = L.adaln_qk_rope_bwd(s["dq"], s["dk"], s["table"], s["pos"], q=s["q"],
                                           k=s["k"], **how)
    return [qo, ko, dq, dwq, dk, dwk]


def run(state):
    if own:
        return _own(state)
    return _plain_ffn(state) if state["case"]["op"].startswith("ffn") else _plain_qk(state)


# ----- the definition in 64 bits ------------------------------------------------


def _exact_qk(s):
    c = s["case"]
    T, rot, op = c["T"], c["rot"], c["op"]
    P = rot // 2
    # the unit complex number that pair p of token t is multiplied by
    z = torch.ones(T, P, dtype=torch.complex128, device=s["pos"].device)
    at = 0
    for a, n in enumerate(s["pairs"]):
        p = s["pos"][:, a].long()
        rows = torch.view_as_complex(s["table"][:, at:at + n].double().contiguous())
        z[:, at:at + n] = torch.where((p >= 0)[:, None], rows[p.clamp(min=0)], 1.0)
        at += n

    def turn(x):
        r = x[..., :rot]
        r = r.reshape(*r.shape[:2], 2, P).transpose(2, 3) if c["half"] else \
            r.reshape(*r.shape[:2], P, 2)
        r = torch.view_as_real(torch.view_as_complex(r.contiguous()) * z[:, None])
        r = (r.transpose(2, 3) if c["half"] else r).reshape(*x.shape[:2], rot)
        return torch.cat([r, x[..., rot:]], 2)

    if op == "rope_fwd":
        return [turn(s["q"].double()), turn(s["k"].double())]
    if op == "rope_bwd":  # the map is linear: its gradient from the chain rule at any point
        res = []
        for n in ("dq", "dk"):
            x = torch.zeros(s[n].shape, dtype=torch.float64, device=z.device, requires_grad=True)
            res.append(torch.autograd.grad(turn(x), x, s[n].double())[0])
        return res
    out, grads = [], []
    for n in ("q", "k"):
        x = s[n].double().requires_grad_(op == "qk_step")
        w = s["w" + n].double().requires_grad_(op == "qk_step")
        y = turn(x / ((x * x).sum(-1, keepdim=True) / c["dh"] + EPS).sqrt() * w)
        out.append(y.detach())
        if op == "qk_step":
            grads.extend(torch.autograd.grad(y, (x, w), s["d" + n].double()))
    return out + grads


def exact(case, seed):
    s = prepare(case, seed)
    if not case["op"].startswith("ffn"):
        return _exact_qk(s)
    if work(case)["flops"] > 4e12:
        return None
    step = case["op"] == "ffn_step"
    x, wg, wu, wd = (s[n].double().requires_grad_(step) for n in ("x", "wg", "wu", "wd"))
    act = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
           "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[case["act"]]
    y = torch.mm(act(torch.mm(x, wg.t())) * torch.mm(x, wu.t()), wd.t())
    if not step:
        return [y]
    return [y.detach(), *torch.autograd.grad(y, (x, wg, wu, wd), s["dy"].double())]


def work(case):
    T = case["T"]
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("ffn"):
        D, F = case["D"], case["F"]
        if case["op"] == "ffn_fwd":  # x, three weights; y
            return {"bytes": e * (2 * T * D + 3 * D * F), "flops": 6 * T * D * F}
        # x, dy, three weights; y, dx, three weight gradients
        return {"bytes": e * (4 * T * D + 6 * D * F), "flops": 18 * T * D * F}
    n = T * (case["hq"] + case["hk"]) * case["dh"]
    other = 12 * T + 4 * max(case["gf"], case["gh"], case["gw"]) * case["rot"]
    if case["op"].startswith("rope"):
        return {"bytes": 2 * n * e + other, "flops": 3 * n}
    # the norm's gradient needs the head whole: the forward's read and write, then
    # both inputs read and the gradient written
    k = 2 if case["op"] == "qk_fwd" else 5
    return {"bytes": k * n * e + other, "flops": (7 if k == 2 else 24) * n}
