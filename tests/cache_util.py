"""Inputs and plain 64-bit references of the operators on small caches.

Tolerance of an attention output in bf16 against the 64-bit result, per element, from the
arithmetic the kernels may use (u = 2^-8: half a step of a bf16 value, e = 2^-23: a whole
step of an fp32 one), with A = sum_p softmax_p |V_p|, n visible positions:
  * the output is rounded once:                        u |out|
  * each probability enters the product rounded:       pu A,  pu = u (bf16), u^2 (two bf16 terms) or
    2^-11 (fp16), there also an absolute 2^-25 of the largest one:  n 2^-25 max|V|
  * a score is a sum of 128 products in fp32:          ds = 128 e scale sum_d |q_d K_d|
    and its exponent is formed in fp32:                dx = 4 e max|x|, x = score * log2(e)
    both move numerator and denominator:               2 (ds + dx) A
  * over 4-bit rows q enters in fp16, scaled so that its largest value is at least 2^8, where a
    value is off by at most 2^-25 below 2^-14: 2^-33 of the largest, in 128 products:
                                                       ds += 128 2^-33 scale max|q| max|K|
  * exp2 within 2 steps, sums over n terms in fp32:    2 (n + 4) e A
A weight is a sum over G heads of probabilities p: each off by (2 (ds + dx) + (n + 8) e) p, the
sum and what it is added to by (G + 1) e of it.
"""
import math

import torch

D = 128
U, E = 2.0 ** -8, 2.0 ** -23
GRID = [0, .5, 1, 1.5, 2, 3, 4, 6]


def paged(x, page, table, pages, fill):
    """Logical rows [B][Hkv][N][w] into pages [pages][Hkv][page][w]; every other row is `fill`."""
    B, Hkv, N, w = x.shape
    out = torch.full((pages, Hkv, page, w), fill, dtype=x.dtype)
    for b in range(B):
        for p0 in range(0, N, page):
            n = min(page, N - p0)
            out[table[b, p0 // page], :, :n] = x[b, :, p0:p0 + n]
    return out


def quantise(x):
    """td_q4_append's codes (bytes [..., 64]) and scales (bytes [..., 8]) of rows [..., 128], value by
    value in 64 bits: every candidate's distance is compared."""
    y = x.double().view(*x.shape[:-1], 8, 16)
    nan = y.isnan().any(-1, keepdim=True)
    z = torch.nan_to_num(y, nan=0.0, posinf=1e300, neginf=-1e300)
    every = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    s, sbyte = nearest(z.abs().amax(-1, keepdim=True) / 6, every)
    t = torch.where(s > 0, z.abs() / torch.where(s > 0, s, 1.0), 0.0)
    _, code = nearest(t, torch.tensor(GRID, dtype=torch.float64))
    code = torch.where((s > 0) & ~nan, code | (torch.signbit(y).long() << 3), 0)
    sbyte = torch.where(nan, 0x7f, sbyte)
    code = code.view(*x.shape[:-1], 64, 2)
    return (code[..., 0] | code[..., 1] << 4).to(torch.uint8), sbyte.squeeze(-1).to(torch.uint8)


def nearest(t, grid):
    """The grid's value nearest to t (ties: the even number; beyond its end the last one) and its number."""
    hi = torch.searchsorted(grid, t.contiguous()).clamp(1, len(grid) - 1)
    lo = hi - 1
    a, b = t - grid[lo], grid[hi] - t
    n = torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)
    return grid[n], n


def values(codes, scales):
    """What 4-bit rows stand for, in 64 bits."""
    grid = torch.tensor(GRID + [-v for v in GRID], dtype=torch.float64)
    half = torch.stack([codes & 15, codes >> 4], -1).long()
    s = scales.contiguous().view(torch.float8_e4m3fn).double()
    return (grid[half].view(*codes.shape[:-1], 8, 16) * s[..., None]).flatten(-2)


def visible(n, p, window, sinks):
    """Positions below n that a token at position p sees."""
    return [j for j in range(min(n, p + 1)) if j < sinks or not window or p - j < window]


def attend(q, k, v, sees, pu, q4=False, scale=None):
    """Rows q [T][d] over k, v [n][d] in 64 bits, sees bool [T][n]: out, tolerance, probabilities and
    the relative error of those."""
    scale = 1 / math.sqrt(D) if scale is None else scale
    q, k, v = q.double(), k.double(), v.double()
    if len(k) == 0:
        return torch.zeros_like(q), torch.zeros_like(q), sees.double(), sees.double()
    z = (q @ k.T) * scale
    some = sees.any(-1, keepdim=True)
    a = torch.where(some, torch.softmax(z.masked_fill(~sees, -math.inf).where(some, 0.0), -1), 0.0)
    out, A = a @ v, a @ v.abs()
    n = sees.sum(-1, keepdim=True)
    cut = torch.where(sees, q.abs() @ k.abs().T, 0.0).amax(-1, keepdim=True)
    ds = D * E * scale * cut
    if q4:
        top = torch.where(sees, k.abs().amax(-1)[None], 0.0).amax(-1, keepdim=True)
        ds = ds + D * 2.0 ** -33 * scale * q.abs().amax(-1, keepdim=True) * top
    dx = 4 * E * torch.where(sees, z.abs(), 0.0).amax(-1, keepdim=True) * 1.4427
    tol = U * out.abs() + (pu + 2 * (ds + dx) + 2 * (n + 4) * E) * A * (1 + U)
    if q4:
        big = torch.where(sees[..., None], v.abs()[None], 0.0).amax(1)
        tol = tol + n * 2.0 ** -25 * big
    return out, tol, a, 2 * (ds + dx) + (n + 8) * E


def evict(w, n, budget, sinks, recent):
    """Positions kept of n, from weights w (list): td_evict step by step."""
    if n <= budget:
        return list(range(n))
    fixed = [i for i in range(n) if i < sinks or i >= n - recent]
    key = lambda i: (-math.inf if math.isnan(w[i]) else -w[i], i)
    # a NaN ranks before an infinity
    rest = sorted((i for i in range(sinks, n - recent)), key=lambda i: (not math.isnan(w[i]),) + key(i))
    return sorted(fixed + rest[:budget - sinks - recent])
