"""Plain 64-bit models of the latent-attention operators (CPU, loops over requests), and the bounds that their
rounding gives. Nothing here shares code with the HIP library."""
from __future__ import annotations

import math

import torch

BF16_HALF = 2.0 ** -8     # half a step of bf16, relative
E4M3_HALF = 2.0 ** -4     # half a step of e4m3, relative; below 2^-6 half the subnormal step, 2^-10
F32_HALF = 2.0 ** -24


def row_layout(latent, rope, mx):
    """(byte offset of the scales, byte offset of the rope part, bytes of a row)."""
    if not mx:
        return 0, 2 * latent, 2 * latent + 2 * rope
    at = latent + -(-(latent // 32) // 16) * 16
    return latent, at, at + 2 * rope


def unpack(rows, latent, rope, mx):
    """float64 [..., latent + rope] of rows (uint8 [..., bytes]) on the CPU."""
    rows = rows.cpu()
    if not mx:
        return rows.contiguous().view(torch.bfloat16).double()
    s, at, _ = row_layout(latent, rope, True)
    v = rows[..., :latent].contiguous().view(torch.float8_e4m3fn).double()
    e = rows[..., s:s + latent // 32].double() - 127
    v = (v.reshape(*v.shape[:-1], latent // 32, 32) * torch.exp2(e).unsqueeze(-1)).reshape(v.shape)
    return torch.cat([v, rows[..., at:].contiguous().view(torch.bfloat16).double()], -1)


def random_rows(shape, latent, rope, mx, gen, spread=1.0):
    """Rows (uint8) of normal values; 8-bit ones from random e4m3 values and scales near one."""
    if not mx:
        return (torch.randn(*shape, latent + rope, generator=gen) * spread).bfloat16().view(torch.uint8)
    q = (torch.randn(*shape, latent, generator=gen) * 64).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    e = torch.randint(119, 123, (*shape, latent // 32), generator=gen, dtype=torch.uint8)
    s, at, _ = row_layout(latent, rope, True)
    fill = torch.randint(0, 256, (*shape, at - s - latent // 32), generator=gen, dtype=torch.uint8)
    r = torch.randn(*shape, rope, generator=gen).bfloat16().view(torch.uint8)
    return torch.cat([q, e, fill, r], -1)


def softmax_rows(s, v):
    """(o, lse, sum of p |v|) for scores [n, keys] and values [keys, m]; zeros and -inf without keys."""
    if s.shape[1] == 0:
        z = torch.zeros(s.shape[0], v.shape[1], dtype=torch.float64)
        return z, torch.full((s.shape[0],), -math.inf, dtype=torch.float64), z
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    return p @ v, lse, p @ v.abs()


def score_error(q, keys, scale):
    """Bound of a score's error in 32 bits, per query: a sum of D products of exact factors, each addition and the
    scaling (to base 2) rounded."""
    if keys.shape[0] == 0:
        return torch.zeros(q.shape[0], dtype=torch.float64)
    mag = (q.abs() @ keys.abs().T).amax(1) * abs(scale)
    return mag * (q.shape[1] + 4) * F32_HALF


def attention_bounds(o, lse, pv, ds, n):
    """Bounds of o [n, m] and lse [n] for weights rounded to bf16 and divided by their own sum, a score error ds, and
    32-bit sums over n keys. exp in 32 bits is off by at most 4 half steps here, its argument by one of the score's
    magnitude (in ds)."""
    p_err = ds * 1.01 + 8 * F32_HALF  # of a weight, relative
    sums = (n + 16) * F32_HALF
    bo = BF16_HALF * o.abs() * 1.01 + pv * (2 * (BF16_HALF + p_err[:, None]) + 2 * sums) * 1.02
    bl = p_err + sums + 4 * F32_HALF * lse.abs().clamp(max=1e30) + 1e-7
    return bo, bl


def attend(q, rows, latent, scale):
    """One request: q float64 [heads, D], rows float64 [m, D] of the selection's valid rows. (o, lse, bounds)."""
    s = q @ rows.T * scale
    o, lse, pv = softmax_rows(s, rows[:, :latent])
    return (o, lse) + attention_bounds(o, lse, pv, score_error(q, rows, scale), rows.shape[0])


def prompt(q, kv, rope, nope, scale, causal):
    """One sequence and head: q [m, nope + rope], kv [n, nope + value], rope [n, rope], all float64."""
    m, n = q.shape[0], kv.shape[0]
    keys = torch.cat([kv[:, :nope], rope], 1)
    v = kv[:, nope:]
    s = q @ keys.T * scale
    if causal:
        seen = torch.arange(n)[None, :] <= (n - m) + torch.arange(m)[:, None]
        s = s.masked_fill(~seen, -math.inf)
    if n == 0:
        o, lse, pv = softmax_rows(s, v)
    else:
        lse = torch.logsumexp(s, 1)
        p = torch.exp(s - lse.clamp(min=-1e300)[:, None])
        o, pv = p @ v, p @ v.abs()
    return (o, lse) + attention_bounds(o, lse, pv, score_error(q, keys, scale), n)


def map_tokens(new, length, tail0, n, B, T, H):
    """The map by a loop over requests and tokens."""
    R = len(new)
    cu, req, pos, slot, status = [0] * (R + 1), [-1] * n, [-1] * n, [-1] * n, [0] * R
    at = 0
    for r in range(R):
        cu[r] = at
        if new[r] < 0:
            status[r] = 1
        for j in range(max(0, min(new[r], n - at))):
            x = length[r] + j
            t = at + j
            req[t] = r
            ok = 0 <= x < H
            if ok and T > 0 and x >= tail0[r]:
                if x < tail0[r] + T:
                    slot[t] = B + x % T
                else:
                    ok = False
            if ok:
                pos[t] = x
            else:
                status[r] = 1
        at = min(n, at + max(0, new[r]))
    cu[R] = at
    return cu, req, pos, slot, status


def store_values(x, weight, eps, pos, freqs, halves, latent):
    """float64 (y [latent], z [rope]) of one token's input x (float64)."""
    y = x[:latent] / math.sqrt(float((x[:latent] ** 2).mean()) + eps) * weight
    z = x[latent:].clone()
    P = z.numel() // 2
    if freqs is not None:
        a, b = (z[:P], z[P:]) if halves else (z[0::2], z[1::2])
        c, s = torch.cos(pos * freqs), torch.sin(pos * freqs)
        u, v = a * c - b * s, a * s + b * c
        z = torch.cat([u, v]) if halves else torch.stack([u, v], 1).flatten()
    return y, z
