"""Plain 64-bit models of the operators that make a selection (CPU), and the bounds that their rounding gives. Nothing here
shares code with the HIP library."""
from __future__ import annotations

import math

import numpy as np
import torch

F32 = 2.0 ** -24   # half a step of float32, relative
BF16 = 2.0 ** -8   # of bf16

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E4M3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()  # 0 .. 448, ascending


def grid_of(bits):
    return E4M3 if bits == 8 else E2M1


def decode(codes, scales, bits):
    """float64 values of bytes (4-bit ones in pairs, the even one in the low bits) and e8m0 scales, on the CPU."""
    codes, scales = codes.cpu(), scales.cpu()
    if bits == 8:
        v = codes.contiguous().view(torch.float8_e4m3fn).double()
    else:
        c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
        v = E2M1[c & 7] * torch.where(c >= 8, -1.0, 1.0).double()
    s = torch.exp2(scales.double() - 127)
    s[scales == 255] = math.nan
    return (v.unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)


def head(v, norm, weight, bias, eps, pos, freqs, at, rope, halves):
    """(y, bound of its error in 32 bits) of heads v [n, heads, dim] (float64) of tokens at pos [n]."""
    dim = v.shape[-1]
    w = torch.ones(dim).double() if weight is None else weight.double()
    b = torch.zeros(dim).double() if bias is None else bias.double()
    err = torch.zeros_like(v)
    if norm == "none":
        y = v
    else:
        mean = v.mean(-1, keepdim=True) if norm == "layer" else torch.zeros_like(v[..., :1])
        e_mean = (dim + 2) * F32 * v.abs().mean(-1, keepdim=True) if norm == "layer" else torch.zeros_like(mean)
        c = v - mean
        std = torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
        z = c / std
        y = z * w + b
        # the mean's sum, the sum of squares (half of it under the root), root, division, products; a mean that is off by
        # e adds e^2 to the mean of squares
        err = (z.abs() * (dim + 24) * F32 + e_mean / std + z.abs() * (e_mean / std) ** 2) * w.abs() * 1.01
        err = err + y.abs() * 2 * F32 + b.abs() * F32
    if rope and freqs is not None:
        part, pe = y[..., at:at + rope], err[..., at:at + rope]
        P = rope // 2
        split = (lambda x: (x[..., :P], x[..., P:])) if halves else (lambda x: (x[..., 0::2], x[..., 1::2]))
        (p, q), (ep, eq) = split(part), split(pe)
        turn = (pos.double().clamp(min=0)[:, None] * freqs)[:, None]
        c, s = torch.cos(turn), torch.sin(turn)
        size = torch.sqrt(p * p + q * q)
        # the angle rounded to 32 bits (of half a turn), before that in 64 bits; sine and cosine two steps; two products
        # and a sum
        e = ep + eq + size * (12 * F32 + turn.abs() * 2.0 ** -51)
        join = (lambda a, b: torch.cat([a, b], -1)) if halves else (lambda a, b: torch.stack([a, b], -1).flatten(-2))
        y = torch.cat([y[..., :at], join(p * c - q * s, p * s + q * c), y[..., at + rope:]], -1)
        err = torch.cat([err[..., :at], join(e, e), err[..., at + rope:]], -1)
    return y, err


def check_quantised(values, scales, y, err, bits, what):
    """Codes' values (without their scale) and scale bytes against unrounded values y that may be off by err: each block's
    scale the least power of two that keeps it within the largest value, each value rounded to the nearest."""
    largest = 448.0 if bits == 8 else 6.0
    y, err = y.reshape(-1, 32), err.reshape(-1, 32)
    values, e = values.reshape(-1, 32).double(), scales.reshape(-1).double() - 127
    assert torch.isfinite(values).all() and (e >= -100).all(), what
    scale = torch.exp2(e)
    low, high = (y.abs() - err).amax(1), (y.abs() + err).amax(1)
    assert (low <= largest * scale).all(), f"{what}: a block does not fit its scale"
    assert ((e == -100) | (high > largest / 2 * scale)).all(), f"{what}: a block's scale is not the least"
    grid = grid_of(bits)
    mid = torch.cat([torch.zeros(1).double(), (grid[1:] + grid[:-1]) / 2, torch.tensor([largest * 1.0000001]).double()])
    at = torch.searchsorted(grid, values.abs())
    assert (grid[at] == values.abs()).all(), f"{what}: not a value of the type"
    size, slack = y.abs() / scale[:, None], err / scale[:, None]
    assert (size + slack >= mid[at]).all() and (size - slack <= mid[at + 1]).all(), f"{what}: not the nearest value"
    wrong = (values * y < 0) & (y.abs() > err)
    assert not wrong.any(), f"{what}: signs differ"


def quantise(y, bits):
    """Bytes and scale bytes for y (float64, finite), ties to even: for inputs that 32 bits compute exactly."""
    largest, grid = (448.0, E4M3) if bits == 8 else (6.0, E2M1)
    blocks = y.double().unflatten(-1, (-1, 32))
    top = blocks.abs().amax(-1)
    e = torch.full_like(top, -100.0)
    for _ in range(400):  # the least power of two, counted up
        e = torch.where(top > largest * torch.exp2(e), e + 1, e)
    size = blocks.abs() / torch.exp2(e).unsqueeze(-1)
    low = (torch.searchsorted(grid, size, right=True) - 1).clamp(max=grid.numel() - 2)
    down, up = size - grid[low], grid[low + 1] - size
    code = torch.where((up < down) | ((up == down) & (low % 2 == 1)), low + 1, low)
    code = (code + torch.signbit(blocks) * (128 if bits == 8 else 8)).flatten(-2).to(torch.uint8)
    if bits == 4:
        code = code[..., 0::2] | (code[..., 1::2] << 4)
    return code, (e + 127).to(torch.uint8)


def score(q, weights, keys):
    """(scores [L], bound) of one token: q [heads, dim], weights [heads], keys [L, dim], float64. Sums of dim exact products in
    32 bits, a product with the weight and a sum over the heads."""
    dots = q @ keys.T
    s = weights @ torch.where(dots < 0, torch.zeros_like(dots), dots)
    size = weights.abs() @ (q.abs() @ keys.abs().T)
    return s, size * (q.shape[1] + q.shape[0] + 4) * F32 * 1.01 + 1e-37


def select(scores, k, recent):
    """Ids of one row (float32 on the CPU, its valid positions alone): the k best, ties to the lowest, ascending, -1 behind."""
    s = scores.double()
    m = s.numel()
    bad = torch.isnan(s) | (s == -math.inf)
    rank = s.clone()
    last = torch.arange(m) >= m - recent
    rank[bad] = -math.inf
    group = torch.where(last, 0, torch.where(bad, 2, 1)).numpy()  # recent ones first, what is never selected last
    key = np.where(group == 1, -rank.numpy(), 0.0)
    order = np.lexsort((np.arange(m), key, group))[:k]
    best = sorted(int(i) for i in order if group[i] < 2)
    return best + [-1] * (k - len(best))
