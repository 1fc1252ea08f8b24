"""Inputs and plain 64-bit references of the speculative-decoding operators.

Tolerance of the tree attention's bf16 output against the 64-bit result, per
element, from the arithmetic the kernel may use (u = 2^-8: half a step of a
bf16 value, e = 2^-23: a whole step of an fp32 one, so that truncating
accumulation counts too), with A = sum_p softmax_p |V_p|:
  * the output is rounded once:                       u |out|
  * each probability enters the product in bf16:      u A
  * a score is a sum of 128 exact products in fp32:   ds = 128 e scale sum_d |q_d K_d|
    and its exponent is formed in fp32:               dx = 4 e max|x|, x = score * log2(e)
    both move numerator and denominator:              2 (ds + dx) A
  * exp2 within 2 steps, sums over n terms in fp32:   2 (n + 4) e A
"""
import math

import torch

D = 128
U, E = 2.0 ** -8, 2.0 ** -23


def pack_mask(seen):
    """bool [B][T][T] -> int32 words [B][T][ceil(T/32)]."""
    B, T, _ = seen.shape
    W = (T + 31) // 32
    bits = torch.zeros(B, T, W * 32, dtype=torch.int64)
    bits[:, :, :T] = seen
    words = (bits.view(B, T, W, 32) << torch.arange(32)).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def make_mask(kind, B, T, gen):
    if kind == "chain":
        return torch.ones(T, T, dtype=torch.bool).tril().expand(B, T, T)
    if kind == "empty":
        return torch.zeros(B, T, T, dtype=torch.bool)
    if kind == "random":                       # any bits: rows that see nothing, rows that see later nodes
        return torch.rand(B, T, T, generator=gen) < 0.4
    seen = torch.zeros(B, T, T, dtype=torch.bool)
    par = torch.arange(T) - torch.randint(1, 5, (B, T), generator=gen)
    for b in range(B):
        for t in range(T):
            if par[b, t] >= 0:
                seen[b, t] = seen[b, par[b, t]]
            seen[b, t, t] = True
    return seen


def paged(K, page, table, pages, fill=float("nan")):
    """Logical rows [B][Hkv][N][D] into pages [pages][Hkv][page][D]; every other row is `fill`."""
    B, Hkv, N, _ = K.shape
    out = torch.full((pages, Hkv, page, D), fill, dtype=K.dtype)
    for b in range(B):
        for p0 in range(0, N, page):
            n = min(page, N - p0)
            out[table[b, p0 // page], :, :n] = K[b, :, p0:p0 + n]
    return out


def reference(q, K, V, lens, sizes, seen, idx=None, scale=None):
    """out [B][T][Hq][D] in 64 bits (rows t >= sizes[b] are zero) and its tolerance;
    K, V are the logical rows [B][Hkv][N][D]."""
    B, T, Hq, _ = q.shape
    Hkv = K.shape[1]
    G = Hq // Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for b in range(B):
        nt = sizes[b]
        c = lens[b] - nt
        for g in range(Hkv):
            rows = list(range(c))
            if idx is not None:
                rows = [int(p) for p in idx[b, g] if 0 <= p < c]
            for t in range(nt):
                pos = rows + [c + j for j in range(nt) if seen[b, t, j]]
                if not pos:
                    continue
                k, v = K[b, g, pos].double(), V[b, g, pos].double()
                for h in range(g * G, (g + 1) * G):
                    qr = q[b, t, h].double()
                    z = (k @ qr) * scale
                    w = torch.softmax(z, 0)
                    o = w @ v
                    A = w @ v.abs()
                    n = len(pos)
                    ds = D * E * scale * float((k.abs() @ qr.abs()).max())
                    dx = 4 * E * float(z.abs().max()) * 1.4427
                    out[b, t, h] = o
                    tol[b, t, h] = U * o.abs() + (U + 2 * (ds + dx) + 2 * (n + 4) * E) * A * (1 + U)
    return out, tol


def tables_reference(page, max_blocks, num_pages, lens, new, table, held, free, count, max_new):
    """td_block_tables on Python lists, step by step; returns the outputs and whether it ran out."""
    table = [list(r) for r in table]
    stack = list(free[:count])
    target = [-(-n // page) for n in lens]
    for b, t in enumerate(target):
        for j in range(t, held[b]):
            stack.append(table[b][j])
    out_held, ran_out = list(held), False
    for b, t in enumerate(target):
        if held[b] >= t:
            out_held[b] = t
            continue
        if ran_out or t - held[b] > len(stack):
            ran_out = True
            continue
        for j in range(held[b], t):
            table[b][j] = stack.pop()
        out_held[b] = t
    cu, slots = [0], []
    for b, n in enumerate(lens):
        for p in range(n - new[b], n):
            page_id = table[b][p // page] if p // page < out_held[b] else -1
            slots.append(page_id * page + p % page if 0 <= page_id < num_pages else -1)
        cu.append(cu[-1] + new[b])
    slots = (slots + [-1] * max_new)[:max_new]
    return table, out_held, stack, cu, slots, ran_out or cu[-1] > max_new
