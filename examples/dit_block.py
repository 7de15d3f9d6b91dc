"""A video DiT block over packed samples, with the library's operators together.

    python examples/dit_block.py [--dim 1536] [--heads 12] [--hidden 4096] [--steps 5]

Packed samples of text and video tokens go through adaLN modulation, the
query/key norm with rotary positions over (time, height, width) (text tokens
unrotated), attention within each sample, a second modulation and the gated
feed-forward block; the projections and the attention are torch's.  The
example trains the block on synthetic data for a few steps, in bf16, and then
runs one forward without gradients.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from adaln_video_dit_gb300 import rotary  # noqa: E402
from adaln_video_dit_gb300.autograd import GatedFFN, QKNormRope, adaln_modulate  # noqa: E402


class DiTBlock(torch.nn.Module):
    """One block; `cond` [samples, dim] makes the six modulation vectors of each
    sample (shift, scale and gate for both halves)."""

    def __init__(self, dim, heads, hidden, rows, device="cuda"):
        super().__init__()
        bf16 = dict(device=device, dtype=torch.bfloat16)
        self.heads, self.head_dim = heads, dim // heads
        self.modulation = torch.nn.Linear(dim, 6 * dim, **bf16)
        self.qkv = torch.nn.Linear(dim, 3 * dim, bias=False, **bf16)
        self.out = torch.nn.Linear(dim, dim, bias=False, **bf16)
        pairs = rotary.split_pairs(self.head_dim // 2)
        self.rope = QKNormRope(self.head_dim, pairs, **bf16)
        self.ffn = GatedFFN(dim, hidden, device=device)
        self.register_buffer("table", rotary.rope_table(rows, pairs, device=device))
        torch.nn.init.zeros_(self.modulation.weight)  # adaLN-Zero: starts as the identity
        torch.nn.init.zeros_(self.modulation.bias)

    def attend(self, q, k, v, lengths):
        """Attention within each packed sample; [T, heads, head_dim] each."""
        outs, at = [], 0
        for n in lengths:
            s = [t[at:at + n].transpose(0, 1)[None] for t in (q, k, v)]
            outs.append(torch.nn.functional.scaled_dot_product_attention(*s)[0].transpose(0, 1))
            at += n
        return torch.cat(outs)

    def forward(self, x, cond, seg_id, pos, lengths):
        shift1, scale1, gate1, shift2, scale2, gate2 = self.modulation(
            torch.nn.functional.silu(cond)).chunk(6, dim=1)
        h = adaln_modulate(x, shift1, scale1, seg_id)
        q, k, v = self.qkv(h).view(len(x), 3, self.heads, self.head_dim).unbind(1)
        q, k = self.rope(q, k, self.table, pos)  # strided views in, contiguous out
        a = self.attend(q, k, v, lengths).reshape(x.shape)
        rows = seg_id.long()
        x = x + gate1[rows] * self.out(a)
        h = adaln_modulate(x, shift2, scale2, seg_id)
        return x + gate2[rows] * self.ffn(h)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--dim", type=int, default=1536)
    ap.add_argument("--heads", type=int, default=12)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=5)
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    samples = [(77, 4, 16, 16), (77, 1, 16, 16), (0, 2, 12, 20)]  # text, frames, height, width
    lengths = [t + f * h * w for t, f, h, w in samples]
    pos = rotary.grid_positions(samples, device="cuda")
    seg_id = torch.repeat_interleave(torch.arange(len(samples), dtype=torch.int32),
                                     torch.tensor(lengths)).cuda()
    block = DiTBlock(a.dim, a.heads, a.hidden, rows=20)
    x = torch.randn(sum(lengths), a.dim, device="cuda", dtype=torch.bfloat16)
    cond = torch.randn(len(samples), a.dim, device="cuda", dtype=torch.bfloat16)
    target = torch.randn_like(x)
    opt = torch.optim.AdamW(block.parameters(), lr=1e-3)
    losses = []
    for step in range(a.steps):
        loss = (block(x, cond, seg_id, pos, lengths).float() - target.float()).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
        print(f"step {step}: loss {losses[-1]:.5f}")
    with torch.no_grad():
        y = block(x, cond, seg_id, pos, lengths)
    print(f"{sum(lengths)} packed tokens, output rms {y.float().square().mean().sqrt():.4f}")
    return losses


if __name__ == "__main__":
    main()
