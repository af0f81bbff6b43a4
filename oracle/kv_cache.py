"""Plain 64-bit forms of the serving operators over a paged key-value cache (test infrastructure;
shares no code with the library): token by token, page by page, from the definitions in
include/cm.h.  Tensors are on the CPU."""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def rotate(x, cos, sin, interleaved):
    """x [heads, d], cos, sin [rot / 2] -> rotated x, and the magnitudes the rotation summed."""
    x, cos, sin = x.to(F64), cos.to(F64), sin.to(F64)
    n = cos.numel()
    out, size = x.clone(), x.abs()
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        out[:, a] = x[:, a] * cos[i] - x[:, b] * sin[i]
        out[:, b] = x[:, b] * cos[i] + x[:, a] * sin[i]
        size[:, a] = (x[:, a] * cos[i]).abs() + (x[:, b] * sin[i]).abs()
        size[:, b] = (x[:, b] * cos[i]).abs() + (x[:, a] * sin[i]).abs()
    return out, size


def exponent(a: float) -> int:
    """e of the smallest 2^e with a <= 127 * 2^e, held to [-50, 50]."""
    if math.isinf(a):
        return 50
    e = -50
    while e < 50 and a > 127 * 2.0 ** e:
        e += 1
    return e


def summary(keys):
    """keys [tokens, d] as the cache holds them -> (largest, smallest) in 8 bits, scale."""
    ok = ~torch.isnan(keys)
    high = torch.where(ok, keys, -math.inf).amax(0)
    low = torch.where(ok, keys, math.inf).amin(0)
    e = exponent(torch.maximum(high.abs(), low.abs()).max().item())
    up = torch.ceil(high.to(F64) * 2.0 ** -e).clamp(-127, 127)
    down = torch.floor(low.to(F64) * 2.0 ** -e).clamp(-127, 127)
    return torch.stack([up, down]).to(torch.int8), 2.0 ** e


def rows(pool, scale, table, h, positions):
    """Values [n, d] in 64 bits of one head's tokens at the given positions of a sequence."""
    P = pool.shape[2]
    at = table[positions // P].long()
    if pool.element_size() == 1:  # e4m3 is indexed by its bytes
        x = pool.view(torch.uint8)[at, h, positions % P].view(pool.dtype).float()
    else:
        x = pool[at, h, positions % P].float()
    return x.to(F64) if scale is None else (x * scale[h]).to(F64)


def decode(q, k, v, scale):
    """q [g, d], k, v [n, d] of the visible keys -> o [g, d], lse [g], and the bounds' terms: the
    largest sum of magnitudes of a score, and sum_j p_j |v_j|."""
    q = q.to(F64)
    if k.shape[0] == 0:
        z = torch.zeros(q.shape, dtype=F64)
        return z, torch.full((q.shape[0],), -math.inf, dtype=F64), 0.0, z
    s = scale * q @ k.T
    size = abs(scale) * (q.abs() @ k.abs().T).max().item()
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    return p @ v, lse, size, p @ v.abs()


def scores(q, summaries, scales):
    """q [g, d], summaries [pages, 2, d], scales [pages] -> score of each page."""
    best = [-math.inf] * len(scales)
    for x in q.to(F64):
        f = exponent(x.abs().max().item())
        x = torch.round(x * 2.0 ** -f).clamp(-127, 127)
        for n, (s, e) in enumerate(zip(summaries.to(F64), scales)):
            best[n] = max(best[n], (torch.where(x > 0, x * s[0], x * s[1]).sum() * 2.0 ** f * float(e)).item())
    return best


def pick(score, n, keep_first, keep_last):
    """The n best pages, ascending: forced ones first, then by score, the lowest page first."""
    total = len(score)
    forced = [i < keep_first or i >= total - keep_last for i in range(total)]
    order = sorted(range(total), key=lambda i: (not forced[i], -score[i] if not forced[i] else 0, i))
    return sorted(order[:n])
