"""Plain 64-bit forms of the operators beside the 4-bit linears in a decoder: rotary positions, the vocabulary
loss with its gradient, and the product of a few tokens with a codebook-quantized weight. Written from their
definitions with elementary float64 torch operations (any device); shares no code with the library.
"""
from __future__ import annotations

import math

import torch


def rope_frequencies(R, base=10000.0, scaling="none", factor=1.0, original_length=0.0, low=None, high=None):
    """(angle per position of each pair, the scale of the result), one pair at a time."""
    low = 1.0 if low is None else low
    high = (32.0 if scaling == "yarn" else 4.0) if high is None else high
    theta, m = [], 1.0
    if scaling == "ntk":
        base = base * factor ** (R / (R - 2))
    for i in range(R // 2):
        t = 1.0 / base ** (2 * i / R)
        if scaling == "linear":
            t = t / factor
        elif scaling == "banded":
            turns = original_length * t / (2 * math.pi)
            if turns <= low:
                t = t / factor
            elif turns < high:
                mix = (turns - low) / (high - low)
                t = (1 - mix) * t / factor + mix * t
        elif scaling == "yarn":
            at = [R * math.log(original_length / (2 * math.pi * b)) / (2 * math.log(base)) for b in (high, low)]
            lo, hi = min(max(math.floor(at[0]), 0), R - 1), min(max(math.ceil(at[1]), 0), R - 1)
            ramp = min(max((i - lo) / (hi - lo if hi > lo else 0.001), 0.0), 1.0)
            t = (t / factor) * ramp + t * (1 - ramp)
            m = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
        theta.append(t)
    return torch.tensor(theta, dtype=torch.float64), m


def rope(x, positions, theta, m=1.0, layout="half", inverse=False):
    """x (B, T, heads, D) turned by positions (B, T); float64 result."""
    x = x.double()
    R = 2 * len(theta)
    angle = positions.double()[:, :, None, None] * theta.to(x.device)
    cos, sin = angle.cos() * m, angle.sin() * (-m if inverse else m)
    y = x.clone()
    a, b = (slice(0, R // 2), slice(R // 2, R)) if layout == "half" else (slice(0, R, 2), slice(1, R, 2))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def vocab_loss(X, W, targets, g=None, ignore=-100):
    """(loss per token, dX for the tokens' loss gradients g), float64."""
    X, W = X.double(), W.double()
    used = targets != ignore
    y = torch.where(used, targets, 0).long()
    rows = torch.arange(X.shape[0], device=X.device)
    X = torch.where(used[:, None], X, 0.0)
    l = X @ W.t()
    lse = torch.logsumexp(l, 1)
    # log(1 + sum of the others) where the target leads: lse - l_y loses a small loss's digits even in 64 bits
    rest = (l - l[rows, y][:, None]).exp()
    rest[rows, y] = 0.0
    small = torch.log1p(rest.sum(1))
    loss = torch.where(lse - l[rows, y] < 0.5, small, lse - l[rows, y])
    loss = torch.where(used, loss, 0.0)
    p = (l - lse[:, None]).exp()
    p[rows, y] = -(-torch.expm1(-loss))
    g = torch.ones_like(loss) if g is None else g.double()
    return loss, (p @ W) * torch.where(used, g, 0.0)[:, None]


def codebook_weight(codes, absmax, N, K, levels):
    """The N x K weight, float64: level[code] * absmax of its block of 64."""
    lv = torch.tensor(list(levels) + [0.0] * (16 - len(levels)), dtype=torch.float32, device=codes.device).double()
    both = torch.stack([codes.view(-1) >> 4, codes.view(-1) & 15], 1).view(-1)[:N * K].long()
    return (lv[both].view(-1, 64) * absmax.view(-1, 1).double()).view(N, K)
