"""Plain definitions of the cache operators in 64 bits on the CPU, and the
error each result may have.  Shares no code with the library."""
import math

import numpy as np
import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
Q = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}


def e4m3_table():
    """The 127 non-negative values, by code."""
    out = [m / 8 * 2.0 ** -6 for m in range(8)]
    out += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return np.array(out[:127])


def quantise(x, kind):
    """Codes' values (float64) and scales of rows x (16-bit), by exact integer
    arithmetic for int8 and by the table of codes for e4m3."""
    x64 = x.double().numpy()
    flat = x64.reshape(-1, x64.shape[-1])
    codes, scales = np.zeros_like(flat), np.zeros(flat.shape[0], np.float32)
    table = e4m3_table()
    for r, row in enumerate(flat):
        if not np.isfinite(row).all():
            scales[r] = np.nan
            continue
        top = np.abs(row).max(initial=0.0)
        if top == 0.0:
            continue
        scales[r] = np.float32(top) / np.float32(Q[kind])
        n = np.abs(row) * Q[kind]                      # exact: at most 11 + 7 bits
        if kind == torch.int8:
            lo = np.floor(n / top)
            for d in (-1.0, 1.0):                      # the division may be off by one at a whole number
                lo = np.where((lo + d) * top <= n, np.maximum(lo, lo + d), lo)
                lo = np.where(lo * top > n, lo - 1, lo)
            twice = 2 * (n - lo * top)                 # against top: exact
            up = (twice > top) | ((twice == top) & (lo % 2 == 1))
            c = lo + up
        else:
            hi = np.clip(np.searchsorted(table, n / top), 1, 126)
            for d in (-1, 1):
                j = np.clip(hi + d, 1, 126)
                better = np.abs(table[j - 1] + table[j] - 2 * n / top) < np.abs(table[hi - 1] + table[hi] - 2 * n / top)
                hi = np.where(better, j, hi)
            mid = (table[hi - 1] + table[hi]) / 2 * top  # exact: 5 bits times 11
            up = (n > mid) | ((n == mid) & (hi % 2 == 0))
            c = np.where(up, table[hi], table[hi - 1])
        codes[r] = np.sign(row) * c
    return codes.reshape(x64.shape), scales.reshape(x64.shape[:-1])


def held(pages, scales):
    """Values of a cache as float64 [pages, heads, places, dim]."""
    x = pages.cpu().float().double()
    return x if scales is None else x * scales.cpu().double()[..., None]


def attention(q, k, v, table, page, q_lens, ctx, group, window, scale, held_type, dtype):
    """(out, lse, out's allowed error, lse's) over float64 values [pages,
    heads, places, dim].  The error counts: the rounding of each weight to the
    second product's type, of the result to the output's, 32-bit sums of dim
    products and of the keys, and fp16's smallest step."""
    total, heads, dim = q.shape
    out = torch.zeros(total, heads, dim, dtype=torch.float64)
    lse = torch.full((total, heads), -math.inf, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros(total, heads, dtype=torch.float64)
    u_w = UNIT[held_type]
    tiny_w = TINY[held_type]
    at = 0
    for s, (n, c) in enumerate(zip(q_lens, ctx)):
        for r in range(n):
            pos = c - n + r
            lo = max(0, pos - window + 1) if window else 0
            hi = min(pos + 1, c)
            if hi > lo:
                t = torch.arange(lo, hi)
                pages, place = table[s][t // page].long(), t % page
                for h in range(heads):
                    kk, vv = k[pages, h // group, place], v[pages, h // group, place]
                    qq = q[at + r, h].double()
                    x = kk @ qq * scale
                    out[at + r, h] = torch.softmax(x, 0) @ vv
                    lse[at + r, h] = torch.logsumexp(x, 0)
                    near = torch.softmax(x, 0) @ vv.abs()
                    size = (kk.abs() @ qq.abs()).max().item() * abs(scale)
                    d = (dim + 8) * 2.0 ** -24 * size
                    rest = near * (u_w + 2 * d + (hi - lo + 16) * 2.0 ** -23) + tiny_w * vv.abs().sum(0)
                    tol[at + r, h] = rest + UNIT[dtype] * (out[at + r, h].abs() + rest) + TINY[dtype]
                    ltol[at + r, h] = d + (hi - lo + 16) * 2.0 ** -23 + abs(lse[at + r, h].item()) * 2.0 ** -22
        at += n
    return out, lse, tol, ltol


def rope(x, positions, freqs, interleaved, factor, inverse):
    """(result, allowed error): products and their sum in 32 bits (three
    roundings of each product's size, cosines to 2^-21), rounded once."""
    rot = 2 * len(freqs)
    a = positions.double()[:, None, None] * freqs.double() * (-1 if inverse else 1)
    c, s = torch.cos(a) * factor, torch.sin(a) * factor
    y = x.double().clone()
    i0 = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    i1 = i0 + 1 if interleaved else i0 + rot // 2
    p, q = y[..., i0].clone(), y[..., i1].clone()
    y[..., i0], y[..., i1] = p * c - q * s, q * c + p * s
    tol = torch.zeros_like(y)
    size = (p.abs() + q.abs()) * abs(factor) * 2.0 ** -21
    tol[..., i0] = size
    tol[..., i1] = size
    tol += (y.abs() + tol) * UNIT[x.dtype] + TINY[x.dtype]
    tol[..., rot:] = 0
    return y, tol
