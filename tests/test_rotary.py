"""Rotary tables and positions (host side)."""
import math

import pytest
import torch

from adaln_video_dit_gb300 import rotary


def test_split_pairs():
    assert rotary.split_pairs(64) == (22, 21, 21)
    assert rotary.split_pairs(64, 2) == (32, 32)
    assert rotary.split_pairs(1, 3) == (1, 0, 0)
    with pytest.raises(ValueError):
        rotary.split_pairs(0)


def test_table_is_the_rounded_definition():
    t = rotary.rope_table(300, (3, 2, 1), theta=100.0, scale=(1.0, 0.5, 2.0))
    assert t.shape == (300, 6, 2) and t.dtype == torch.float32
    want = [(n, i, s) for n, s in ((3, 1.0), (2, 0.5), (1, 2.0)) for i in range(n)]
    for p in (0, 1, 17, 299):
        for j, (n, i, s) in enumerate(want):
            a = p * s * 100.0 ** (-i / n)
            for got, ref in zip(t[p, j].tolist(), (math.cos(a), math.sin(a))):
                # one rounding to 32 bits, and the angle's own in 64
                assert abs(got - ref) <= 2.0 ** -24 * abs(ref) + 1e-13 * max(1.0, a)
    for bad in (dict(rows=0, axis_pairs=(1,)), dict(rows=1, axis_pairs=(0,)),
                dict(rows=1, axis_pairs=(1, 1), scale=(1.0,))):
        with pytest.raises(ValueError):
            rotary.rope_table(**bad)


def test_grid_positions():
    p = rotary.grid_positions([(2, 2, 1, 2), (0, 1, 2, 1), (1, 0, 3, 3)])
    assert p.dtype == torch.int32 and p.tolist() == [
        [-1, -1, -1], [-1, -1, -1], [0, 0, 0], [0, 0, 1], [1, 0, 0], [1, 0, 1],
        [0, 0, 0], [0, 1, 0], [-1, -1, -1]]
    assert rotary.grid_positions([]).shape == (0, 3)
