"""The operators as autograd nodes: the fused AdaLN, the rotary positions and
norm of queries and keys, and the gated feed-forward block.

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
