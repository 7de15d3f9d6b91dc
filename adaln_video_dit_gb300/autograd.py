"""The operators as autograd nodes: the fused AdaLN, the rotary positions and
norm of queries and keys, the gated feed-forward block, dropout with the gate and
the residual of a branch, and feed-forward blocks that are mixtures of experts.

AdaptiveLoad (Technical summary, section 2.B, "graph simplification"): the
LayerNorm -> multiply -> add chain of an adaLN modulation site collapses into
a single node whose intermediate statistics never become framework tensors.
`AdaLNModulateFunction` is that node: its forward is `adaln_fwd`, it saves
only x, the per-row mean and rstd (8 bytes per token), the modulation scale
and the segment ids, and its backward is `adaln_bwd`.  The unfused chain
instead keeps the normalised activations and the gathered (1 + scale) rows.

Layout: x is [..., D] (flattened to tokens [T, D]); shift and scale are
[nseg, D]; seg_id is int32 [T], non-decreasing, mapping each token to its
modulation row.  For a batch x [B, N, D] with one modulation row per sample,
`sample_seg_ids(B, N)` gives seg_id.  The other operators' tensors may have any
leading dimensions as well.
"""
import torch
from torch.autograd.function import once_differentiable

from . import _lib


def sample_seg_ids(B, N, device=None):
    """seg_id for B samples of N tokens each, packed back to back."""
    return torch.arange(B, device=device, dtype=torch.int32).repeat_interleave(N)


class AdaLNModulateFunction(torch.autograd.Function):
    """y = LayerNorm(x) * (1 + scale[seg_id]) + shift[seg_id], fused."""

    @staticmethod
    def forward(ctx, x, shift, scale, seg_id, eps):
        shape = x.shape
        D = shape[-1]
        x2 = x.reshape(-1, D)
        if not x2.is_contiguous():
            x2 = x2.contiguous()
        y, mean, rstd = _lib.adaln_fwd(x2, shift.contiguous(), scale.contiguous(),
                                       seg_id, eps)
        ctx.save_for_backward(x2, mean, rstd, scale.contiguous(), seg_id)
        ctx.shape = shape
        ctx.mod_dtypes = (shift.dtype, scale.dtype)
        return y.reshape(shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x2, mean, rstd, scale, seg_id = ctx.saved_tensors
        dy2 = dy.reshape(x2.shape)
        if dy2.dtype != x2.dtype:
            dy2 = dy2.to(x2.dtype)
        if not dy2.is_contiguous():
            dy2 = dy2.contiguous()
        dx, dshift, dscale = _lib.adaln_bwd(dy2, x2, mean, rstd, scale, seg_id)
        return (dx.reshape(ctx.shape), dshift.to(ctx.mod_dtypes[0]),
                dscale.to(ctx.mod_dtypes[1]), None, None)


def adaln_modulate(x, shift, scale, seg_id, eps=1e-6):
    """Functional form of the fused operator (differentiable in x, shift, scale)."""
    return AdaLNModulateFunction.apply(x, shift, scale, seg_id, float(eps))


class AdaLNModulate(torch.nn.Module):
    """Module form: forward(x, shift, scale, seg_id) -> y."""

    def __init__(self, eps=1e-6):
        super().__init__()
        self.eps = float(eps)

    def forward(self, x, shift, scale, seg_id):
        return adaln_modulate(x, shift, scale, seg_id, self.eps)

    def extra_repr(self):
        return f"eps={self.eps}"


class QKNormRopeFunction(torch.autograd.Function):
    """Rotary positions of queries and keys, with an optional RMS norm of every
    head first.  Saves q and k themselves (they may be views of a packed
    projection), the weights, the table and the positions; nothing else."""

    @staticmethod
    def forward(ctx, q, k, wq, wk, table, pos, axis_pairs, interleaved, norm, eps):
        wq = wq.contiguous() if wq is not None else None
        wk = wk.contiguous() if wk is not None else None
        ctx.how = (tuple(axis_pairs), interleaved, norm)
        ctx.eps = eps
        ctx.save_for_backward(*((q, k) if norm else (None, None)), wq, wk, table, pos)
        return _lib.adaln_qk_rope_fwd(q, k, table, pos, *ctx.how, wq=wq, wk=wk, eps=eps)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, wq, wk, table, pos = ctx.saved_tensors
        dq_out, dk_out = (d if d is None or d.stride(-1) == 1 else d.contiguous()
                          for d in (dq_out, dk_out))
        dq, dk, dwq, dwk = _lib.adaln_qk_rope_bwd(dq_out, dk_out, table, pos, *ctx.how, q=q, k=k,
                                                  wq=wq, wk=wk, eps=ctx.eps)
        # (The keys' weight has no gradient where there are no keys.)
        return (dq, dk, dwq.to(wq.dtype) if wq is not None else None,
                dwk.to(wk.dtype) if wk is not None and dwk is not None else None) + (None,) * 6


def _by_token(q, k, wq, wk, table, pos, *how):
    """The node on tokens [T, heads, dh], from any leading dimensions and back."""
    if q.dim() == 3 and pos.dim() == 2:
        return QKNormRopeFunction.apply(q, k, wq, wk, table, pos, *how)

    def flat(x):
        return x.reshape(-1, *x.shape[-2:]) if x is not None else None

    qo, ko = QKNormRopeFunction.apply(flat(q), flat(k), wq, wk, table, pos.reshape(-1, pos.shape[-1]),
                                      *how)
    return qo.reshape(q.shape), ko.reshape(k.shape) if k is not None else None


def qk_rope(q, k, table, pos, axis_pairs, interleaved=True):
    """Rotary positions of q [..., hq, dh] and k [..., hk, dh] (or None) with pos
    [..., axes], flattened to tokens (differentiable)."""
    return _by_token(q, k, None, None, table, pos, axis_pairs, interleaved, False, 0.0)


def qk_norm_rope(q, k, wq, wk, table, pos, axis_pairs, interleaved=True, eps=1e-6):
    """RMS norm of every head (weights wq, wk [dh] in q's dtype, or None for ones),
    then the rotary positions, in one pass (differentiable in q, k, wq, wk); shapes
    as for qk_rope."""
    return _by_token(q, k, wq, wk, table, pos, axis_pairs, interleaved, True, float(eps))


class QKNormRope(torch.nn.Module):
    """Module form: holds the two weights, in the queries' and keys' dtype;
    forward(q, k, table, pos) -> (q, k)."""

    def __init__(self, head_dim, axis_pairs, interleaved=True, eps=1e-6, device=None, dtype=None):
        super().__init__()
        self.wq = torch.nn.Parameter(torch.ones(head_dim, device=device, dtype=dtype))
        self.wk = torch.nn.Parameter(torch.ones(head_dim, device=device, dtype=dtype))
        self.axis_pairs, self.interleaved, self.eps = tuple(axis_pairs), interleaved, float(eps)

    def forward(self, q, k, table, pos):
        return qk_norm_rope(q, k, self.wq, self.wk, table, pos, self.axis_pairs, self.interleaved,
                            self.eps)

    def extra_repr(self):
        return f"axis_pairs={self.axis_pairs}, interleaved={self.interleaved}, eps={self.eps}"


class GatedFFNFunction(torch.autograd.Function):
    """y = (act(x wg') * (x wu')) wd', saving x and the two projections (24 bits
    a value); without a gradient to come, nothing.  `grad` is whether gradients
    were on at the call: in here they are always off, and needs_input_grad is
    True for a parameter under no_grad() too."""

    @staticmethod
    def forward(ctx, x, wg, wu, wd, act, grad):
        shape = x.shape
        x2 = x.reshape(-1, shape[-1]).contiguous()
        wg, wu, wd = wg.contiguous(), wu.contiguous(), wd.contiguous()
        y, saved = _lib.adaln_ffn_fwd(x2, wg, wu, wd, act=act,
                                      save=grad and any(ctx.needs_input_grad))
        ctx.save_for_backward(x2, wg, wu, wd, saved)
        ctx.act, ctx.shape = act, shape
        return y.reshape(shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x2, wg, wu, wd, saved = ctx.saved_tensors
        dy2 = dy.reshape(x2.shape).to(x2.dtype).contiguous()
        dx, dwg, dwu, dwd = _lib.adaln_ffn_bwd(dy2, x2, wg, wu, wd, saved, act=ctx.act)
        return dx.reshape(ctx.shape), dwg, dwu, dwd, None, None


def gated_ffn(x, wg, wu, wd, act="silu"):
    """The gated feed-forward block of bf16 x [..., D] with wg, wu [F, D], wd
    [D, F], at 16-byte alignment; act "silu", "gelu_tanh" or "gelu"
    (differentiable)."""
    return GatedFFNFunction.apply(x, wg, wu, wd, act, torch.is_grad_enabled())


class GatedFFN(torch.nn.Module):
    """Module form of the gated feed-forward block (bf16, no biases)."""

    def __init__(self, dim, hidden, act="silu", device=None):
        super().__init__()
        if act not in _lib.ACTS:
            raise ValueError(f"act must be one of {sorted(_lib.ACTS)}, got {act!r}")

        def weight(rows, cols):
            w = torch.empty(rows, cols, device=device, dtype=torch.bfloat16)
            return torch.nn.Parameter(torch.nn.init.normal_(w, std=cols ** -0.5))

        self.wg, self.wu, self.wd = weight(hidden, dim), weight(hidden, dim), weight(dim, hidden)
        self.act = act

    def forward(self, x):
        return gated_ffn(x, self.wg, self.wu, self.wd, self.act)

    def extra_repr(self):
        return f"dim={self.wg.shape[1]}, hidden={self.wg.shape[0]}, act={self.act!r}"


class DropoutFunction(torch.autograd.Function):
    """y = [x +] [gate[seg_id] *] dropout(h).  Saves the gate and, for its gradient,
    h; the mask is made again from p and rng."""

    @staticmethod
    def forward(ctx, h, x, gate, seg_id, p, rng):
        shape = h.shape
        h2 = h.reshape(-1, shape[-1]).contiguous()
        x2 = x.reshape(h2.shape).contiguous() if x is not None else None
        gate = gate.contiguous() if gate is not None else None
        of_gate = gate is not None and ctx.needs_input_grad[2]
        held = torch.is_tensor(rng)
        ctx.save_for_backward(h2 if of_gate else None, gate, seg_id, rng if held else None)
        ctx.shape, ctx.p, ctx.rng = shape, p, None if held else rng
        ctx.x_shape = x.shape if x is not None else None
        return _lib.adaln_dropout_fwd(h2, p, rng, x=x2, gate=gate, seg_id=seg_id).reshape(shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        h, gate, seg_id, rng = ctx.saved_tensors
        dh = dgate = None
        if ctx.needs_input_grad[0] or h is not None:
            dy2 = dy.reshape(-1, ctx.shape[-1]).contiguous()
            dh, dgate = _lib.adaln_dropout_bwd(dy2, ctx.p, ctx.rng if rng is None else rng, h=h, gate=gate,
                                               seg_id=seg_id)
            dh = dh.reshape(ctx.shape)
        return (dh, dy.reshape(ctx.x_shape) if ctx.needs_input_grad[1] else None,
                dgate.to(gate.dtype) if dgate is not None else None, None, None, None)


def _draw(p, rng, device):
    """The (seed, offset) of a mask: the given one, or one drawn on the device from
    torch's generator there, which torch.manual_seed seeds, checkpointing restores
    for a recomputation and a captured graph advances at each replay."""
    if rng is not None or p == 0.0:
        return rng
    return torch.randint(1 << 62, (2,), device=device, dtype=torch.int64)


def dropout(h, p, rng=None):
    """Dropout of h [..., D] (differentiable): the same p and rng give the same mask.
    rng is (seed, offset), an int64 CUDA tensor of the two (which may not be
    changed before the backward), or None: drawn from torch's generator."""
    return DropoutFunction.apply(h, None, None, None, float(p), _draw(p, rng, h.device))


def gated_residual(x, h, gate, seg_id, p=0.0, rng=None):
    """x + gate[seg_id] * dropout(h): the end of a branch of an adaLN-Zero block, for
    x, h [..., D] and gate [nseg, D] of one dtype (differentiable in x, h, gate)."""
    return DropoutFunction.apply(h, x, gate, seg_id, float(p), _draw(p, rng, h.device))


class GatedResidual(torch.nn.Module):
    """Module form: forward(x, h, gate, seg_id); drops in training mode only."""

    def __init__(self, p=0.0):
        super().__init__()
        if not 0.0 <= p <= 1.0:
            raise ValueError(f"p must be in [0, 1], got {p}")
        self.p = float(p)

    def forward(self, x, h, gate, seg_id, rng=None):
        return gated_residual(x, h, gate, seg_id, self.p if self.training else 0.0, rng)

    def extra_repr(self):
        return f"p={self.p}"


def route(expert, num_experts, align=64):
    """Where tokens go: expert [..., k], of a signed integer type, holds each token's choices
    (-1 for none), and the Route sorts the (token, choice) pairs by expert, for
    expert_sort and expert_combine."""
    if expert.dtype not in (torch.int8, torch.int16, torch.int32, torch.int64):
        raise TypeError(f"expert must be of a signed integer type, got {expert.dtype}")
    if expert.dtype == torch.int64:  # none wraps to an expert: what is none is refused as it is
        expert = expert.clamp(-2, num_experts)
    return _lib.adaln_route(expert.reshape(-1, expert.shape[-1]).to(torch.int32).contiguous(), num_experts,
                            align)


def _seen_whole(name, like):
    """{name: zeros} for a call that leaves a gradient's rows behind the last expert as they
    were, while anomaly detection looks at whole gradients for NaN; else nothing."""
    return {name: torch.zeros_like(like)} if torch.is_anomaly_enabled() else {}


class ExpertSortFunction(torch.autograd.Function):
    """xs[route.row[t, j]] = x[t].  Saves the route's indices."""

    @staticmethod
    def forward(ctx, x, row, starts, counts, rows, align):
        x2 = x.reshape(-1, x.shape[-1]).contiguous()
        ctx.save_for_backward(row, starts, counts)
        ctx.rows, ctx.align, ctx.shape = rows, align, x.shape
        return _lib.adaln_expert_sort_fwd(x2, _lib.Route(row, starts, counts, rows, align))

    @staticmethod
    @once_differentiable
    def backward(ctx, dxs):
        r = _lib.Route(*ctx.saved_tensors, ctx.rows, ctx.align)
        return (_lib.adaln_expert_sort_bwd(dxs.contiguous(), r).reshape(ctx.shape),) + (None,) * 5


class ExpertCombineFunction(torch.autograd.Function):
    """y[t] = sum_j weight[t, j] ys[route.row[t, j]].  Saves ys, the weights and the
    route's indices."""

    @staticmethod
    def forward(ctx, ys, weight, row, starts, counts, rows, align):
        w2 = weight.reshape(row.shape).float().contiguous()
        ys = ys.contiguous()
        ctx.save_for_backward(ys, w2, row, starts, counts)
        ctx.rows, ctx.align, ctx.weight = rows, align, (weight.shape, weight.dtype)
        y = _lib.adaln_expert_combine_fwd(ys, w2, _lib.Route(row, starts, counts, rows, align))
        return y.reshape(*weight.shape[:-1], y.shape[-1])

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        ys, weight, *indices = ctx.saved_tensors
        dys, dw = _lib.adaln_expert_combine_bwd(dy.reshape(-1, dy.shape[-1]).contiguous(), ys, weight,
                                                _lib.Route(*indices, ctx.rows, ctx.align),
                                                **_seen_whole("dys", ys))
        return (dys, dw.reshape(ctx.weight[0]).to(ctx.weight[1])) + (None,) * 5


def expert_sort(x, route):
    """Tokens x [..., D] sorted by expert: [route.rows, D], each at the rows of its
    choices, zeros between the experts' rows (differentiable).  Rows from
    route.starts[-1] on hold nothing: they are not written, here or in a gradient, and
    may hold NaN (a hook on a sorted array's gradient sees them; zeros under
    torch.autograd.detect_anomaly)."""
    return ExpertSortFunction.apply(x, *route)


def expert_combine(ys, weight, route):
    """The experts' outputs ys [route.rows, D] brought back to their tokens, each
    weighted with its choice's weight [..., k], and summed: [..., D]
    (differentiable in ys and weight)."""
    return ExpertCombineFunction.apply(ys, weight, *route)


class ExpertsFFNFunction(torch.autograd.Function):
    """ys = (act(xs wg[e]') * (xs wu[e]')) wd[e]' on each expert's rows, saving xs and the
    two projections; without a gradient to come, nothing (`grad`: as for the block)."""

    @staticmethod
    def forward(ctx, xs, wg, wu, wd, starts, act, grad):
        xs, wg, wu, wd = xs.contiguous(), wg.contiguous(), wu.contiguous(), wd.contiguous()
        ys, saved = _lib.adaln_experts_ffn_fwd(xs, wg, wu, wd, starts, act=act,
                                               save=grad and any(ctx.needs_input_grad))
        ctx.save_for_backward(xs, wg, wu, wd, starts, saved)
        ctx.act = act
        return ys

    @staticmethod
    @once_differentiable
    def backward(ctx, dys):
        xs, wg, wu, wd, starts, saved = ctx.saved_tensors
        return (*_lib.adaln_experts_ffn_bwd(dys.to(xs.dtype).contiguous(), xs, wg, wu, wd, starts, saved,
                                            act=ctx.act, **_seen_whole("dxs", xs)), None, None, None)


def experts_ffn(xs, wg, wu, wd, route, act="silu"):
    """The gated feed-forward block of each expert on its rows of bf16 xs [route.rows,
    D], as expert_sort gives them (align a multiple of 64), with wg, wu [E, F, D], wd
    [E, D, F] (differentiable).  Rows between the experts' are zeros, here and in the
    gradients; rows from route.starts[-1] on hold nothing."""
    if route.align % 64:
        raise ValueError(f"the experts' rows must start at multiples of 64, not of {route.align}")
    return ExpertsFFNFunction.apply(xs, wg, wu, wd, route.starts, act, torch.is_grad_enabled())


class MixtureFFN(torch.nn.Module):
    """A mixture of `experts` gated feed-forward blocks (bf16, no biases), of which every
    token of x [..., D] takes the top_k that a linear router gives the largest
    softmax probabilities, weighted with those, scaled to a sum of one.  Tokens whose
    `mask` [...] is false go to no expert: their output is zero.  The router's product is
    torch's, of fp32 values: torch's setting of fp32 products applies to it, and with TF32
    (set_float32_matmul_precision("high")) tokens between two experts may take the other.

    The whole runs on the device: how many tokens an expert gets is never asked for."""

    def __init__(self, dim, hidden, experts, top_k=2, act="silu", device=None):
        super().__init__()
        if act not in _lib.ACTS:
            raise ValueError(f"act must be one of {sorted(_lib.ACTS)}, got {act!r}")
        if not 1 <= top_k <= experts:
            raise ValueError(f"top_k must be in [1, {experts}], got {top_k}")

        def weight(rows, cols):
            w = torch.empty(experts, rows, cols, device=device, dtype=torch.bfloat16)
            return torch.nn.Parameter(torch.nn.init.normal_(w, std=cols ** -0.5))

        self.wg, self.wu, self.wd = weight(hidden, dim), weight(hidden, dim), weight(dim, hidden)
        self.router = torch.nn.Parameter(
            torch.nn.init.normal_(torch.empty(experts, dim, device=device), std=dim ** -0.5))
        self.experts, self.top_k, self.act = experts, top_k, act

    def forward(self, x, mask=None):
        # (The router's few products in 32 bits, under autocast too: its probabilities choose
        # the experts.  Where torch is told to use TF32 they are TF32's: of 32760 tokens of
        # 5120 values with two of 8 experts 13 took another one.  A product with
        # exact parts of the weights would hold them, at up to 3 times the default's time.
        # What is masked stays out of them: a NaN there would be in the router's gradient.)
        seen = x.float()
        if mask is not None:
            seen = torch.where(mask[..., None], seen, 0.0)
        with torch.autocast(x.device.type, enabled=False):
            p, expert = (seen @ self.router.float().t()).softmax(-1).topk(self.top_k, -1)
        expert = expert.int()
        if mask is not None:
            expert = torch.where(mask[..., None], expert, -1)
        r = route(expert, self.experts)
        ys = experts_ffn(expert_sort(x, r), self.wg, self.wu, self.wd, r, self.act)
        return expert_combine(ys, p / p.sum(-1, keepdim=True), r)

    def extra_repr(self):
        return (f"dim={self.wg.shape[2]}, hidden={self.wg.shape[1]}, experts={self.experts}, "
                f"top_k={self.top_k}, act={self.act!r}")
