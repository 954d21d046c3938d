"""A network of a WTConv stage and token blocks on images of different sizes,
and a training loop on synthetic ones:

    python -m memory_bound_cnn_amd.hybrid [--steps N] [--channels C] [--blocks B] [--scan]

Each image goes through the WTConv stage as a channels-last plane; its pixels
are then tokens, packed with those of the other images, for blocks of norm,
rotary attention and dropout (``tokens.TokenBlock``), which see each image
alone, or with --scan for blocks of layer norm, gated recurrence and experts
(``tokens.ScanBlock``), whose work grows with the tokens and not with their
square.  A norm, a mean over each image's tokens and a linear layer classify it.
"""

import argparse

import torch

from . import tokens
from .autograd import WTConv2d

__all__ = ["HybridNet", "train"]


class HybridNet(torch.nn.Module):
    """images [3, H, W] float32, a list of any sizes -> logits [n, classes]."""

    def __init__(self, channels=96, heads=3, kv_heads=None, blocks=2, patch=4, levels=2, classes=10, p=0.1, device=None,
                 dtype=torch.bfloat16, scan=False, experts=4):
        super().__init__()
        self.dtype = dtype
        self.stem = torch.nn.Conv2d(3, channels, patch, patch, device=device)
        self.conv = WTConv2d(channels, kernel_size=5, levels=levels, device=device)
        self.scan = scan
        f = dict(device=device, dtype=dtype)
        self.blocks = torch.nn.ModuleList(
            tokens.ScanBlock(channels, experts=experts, **f) if scan else
            tokens.TokenBlock(channels, heads, kv_heads, p=p, seed=i, **f) for i in range(blocks))
        self.norm = tokens.RMSNorm(channels, device=device)
        self.head = torch.nn.Linear(channels, classes, device=device, dtype=dtype)

    def forward(self, images):
        planes = []
        for image in images:
            x = self.stem(image[None]).contiguous(memory_format=torch.channels_last)
            planes.append(x + self.conv(x))
        sizes = [tuple(x.shape[2:]) for x in planes]
        positions, cu_seqlens = tokens.image_positions(sizes, device=planes[0].device)
        t = torch.cat([x.permute(0, 2, 3, 1).reshape(-1, x.shape[1]) for x in planes]).to(self.dtype)
        for block in self.blocks:
            t = block(t, cu_seqlens) if self.scan else block(t, positions, cu_seqlens)
        t = self.norm(t).float()
        pooled = torch.stack([part.mean(0) for part in t.split([h * w for h, w in sizes])])
        return self.head(pooled.to(self.dtype)).float()


def train(steps=20, channels=96, blocks=2, images=8, seed=0, device="cuda", dtype=torch.bfloat16, log=print, scan=False):
    """Losses of `steps` steps on the same synthetic images of 28 to 64 pixels a
    side, whose class is in their mean colour."""
    torch.manual_seed(seed)
    net = HybridNet(channels, heads=channels // 32, blocks=blocks, device=device, dtype=dtype, scan=scan)
    labels = torch.arange(images, device=device) % 10
    batch = [torch.randn(3, 4 * (7 + i % 10), 4 * (16 - i % 8), device=device) + 0.3 * (int(labels[i]) - 5)
             for i in range(images)]
    opt = torch.optim.AdamW(net.parameters(), lr=1e-3)
    losses = []
    for step in range(steps):
        loss = torch.nn.functional.cross_entropy(net(batch), labels)
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
        if log:
            log(f"step {step}: loss {losses[-1]:.4f}")
    return losses


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--channels", type=int, default=96, help="a multiple of 32 (heads of 32 channels)")
    p.add_argument("--blocks", type=int, default=2)
    p.add_argument("--scan", action="store_true", help="gated recurrence and experts instead of attention and one branch")
    a = p.parse_args()
    train(a.steps, a.channels, a.blocks, scan=a.scan)


if __name__ == "__main__":
    main()
