"""Plain 64-bit norm, rotation and append of new tokens, written from the definitions in
include/pkv.h, and the bounds of the kernel's distance from them."""
import math

import torch

E32 = 2.0 ** -24   # half a step of 32-bit values, relative
BF16 = 2.0 ** -8   # of bf16


def frequencies(rot, base=10000.0, factor=1.0, original=0, low=1.0, high=4.0):
    out = []
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        keep = 0.0
        if original:
            keep = min(1.0, max(0.0, (original * f / (2 * math.pi) - low) / (high - low)))
        out.append(f if factor == 1 else f * (keep + (1 - keep) / factor))
    return torch.tensor(out, dtype=torch.float64)


def norm_rope(x, w, eps, pos, freq, factor, interleaved):
    """(values, bounds) of heads x [T, H, D], in double.

    Before the rounding to bf16 (half a step of the value) the kernel is off by, in units of
    2^-24 of the pair's size: the sum of squares 11 (8 products in turn and up to 4 partial
    sums, less 1 as they are all positive), half of it under the root, the reciprocal root 4,
    three products 3; the angle's fraction and its rounding pi (1 + 2^-8), sine and cosine 2 and
    the factor 1 of each of two products, their sum 2: less than 32 together."""
    y, D = x.double(), x.shape[-1]
    if w is not None:
        y = w.double() * y / torch.sqrt((y ** 2).mean(-1, keepdim=True) + eps)
    size = y.abs()
    if freq is not None:
        n = 2 * len(freq)
        t = torch.outer(pos.double(), freq)[:, None]
        i = torch.arange(len(freq))
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + len(freq))
        u, v = y[..., a], y[..., b]
        y, size = y.clone(), size.clone()
        y[..., a] = factor * (u * t.cos() - v * t.sin())
        y[..., b] = factor * (v * t.cos() + u * t.sin())
        size[..., a] = size[..., b] = abs(factor) * torch.hypot(u, v)
        assert n <= D
    off = 32 * E32 * size
    return y, off + BF16 * (y.abs() + off) + 2.0 ** -130


def places(lens, cu, T, table, P, blocks, positions=None):
    """Per token (rotary position or None, page or None, slot)."""
    out = [(None, None, 0)] * T
    B = len(lens)
    cu = [b * (T // B) for b in range(B + 1)] if cu is None else [int(c) for c in cu]
    for b in range(B):
        for t in range(cu[b], cu[b + 1]):
            pos = int(lens[b]) - (cu[b + 1] - t)
            rot = pos if positions is None else int(positions[t])
            if pos < 0 or rot < 0:
                continue
            page = int(table[b, pos // P]) if pos // P < table.shape[1] else -1
            out[t] = (rot, page if 0 <= page < blocks else None, pos % P)
    return out
