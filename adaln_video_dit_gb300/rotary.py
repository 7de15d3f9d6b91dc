"""Tables and positions of the rotary operator (host-side helpers).

A table holds, for each position (row) and each pair of a head's elements, the
cosine and sine of position * theta^(-i / n), i counting an axis's n pairs.
The angles are computed in 64 bits and rounded once: at position 10,000 an
angle computed in 32 bits would be off by up to 5e-4.
"""
import torch


def split_pairs(pairs, axes=3):
    """`pairs` shared out over the axes: equal parts, the rest to the first
    (time); 64 pairs over (time, height, width) are (22, 21, 21)."""
    if axes < 1 or pairs < 1:
        raise ValueError("axes and pairs must be positive")
    part = pairs // axes
    return (pairs - (axes - 1) * part,) + (part,) * (axes - 1)


def rope_table(rows, axis_pairs, theta=10000.0, scale=None, device=None):
    """fp32 [rows, sum(axis_pairs), 2]: cosine and sine of the positions
    0 .. rows - 1.  `scale` (one factor per axis) multiplies the positions, for
    images or clips larger or smaller than those trained on."""
    if rows < 1 or len(axis_pairs) < 1 or min(axis_pairs) < 0 or sum(axis_pairs) < 1:
        raise ValueError("rows and the sum of axis_pairs must be positive, its counts >= 0")
    scale = (1.0,) * len(axis_pairs) if scale is None else scale
    if len(scale) != len(axis_pairs):
        raise ValueError("scale needs one factor per axis")
    freq = torch.cat([s * theta ** (-torch.arange(n, dtype=torch.float64) / max(n, 1))
                      for n, s in zip(axis_pairs, scale)])
    angle = torch.arange(rows, dtype=torch.float64)[:, None] * freq
    return torch.stack([angle.cos(), angle.sin()], -1).float().to(device)


def grid_positions(samples, device=None):
    """int32 [T, 3] positions of packed samples, each (text, frames, height,
    width): `text` unrotated tokens (-1 on every axis), then the video tokens in
    raster order, time slowest."""
    parts = []
    for text, f, h, w in samples:
        grid = torch.cartesian_prod(torch.arange(f), torch.arange(h), torch.arange(w)).view(-1, 3)
        parts += [torch.full((text, 3), -1), grid]
    pos = torch.cat(parts) if parts else torch.empty(0, 3)
    return pos.to(torch.int32).contiguous().to(device)
