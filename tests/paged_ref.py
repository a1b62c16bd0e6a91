"""Plain 64-bit forms of the paged cache's operators, one sequence and head at
a time, on the CPU, and the error bounds that the kernels' roundings give."""
import math

import numpy as np
import torch

E4M3 = torch.float8_e4m3fn


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def values(codes, scale=None):
    """A cache's values in 64 bits (codes [pages, tokens, heads, D])."""
    x = codes.cpu().to(torch.float32).double()
    return x if scale is None else x * scale.cpu().double()[:, None, :, None]


def attend(q, k, v, table, lens, counts, scale=None, causal=False):
    """q [total, H, D]; k, v: 64-bit pages; counts: rows a sequence.  (out,
    lse, spread, reach): spread = sum p |v|, reach = the largest sum |q| |k|
    over a row's keys, for the bounds."""
    q = q.cpu().double()
    total, H, D = q.shape
    P, hkv = k.shape[1], k.shape[2]
    G, sc = H // hkv, (1.0 / math.sqrt(D) if scale is None else scale)
    out, spread = torch.zeros(total, H, D, dtype=torch.float64), torch.zeros(total, H, D, dtype=torch.float64)
    lse, reach = torch.full((total, H), -math.inf, dtype=torch.float64), torch.zeros(total, H, dtype=torch.float64)
    top = torch.zeros(total, H, D, dtype=torch.float64)
    row = 0
    for b, n in enumerate(counts):
        length = min(max(int(lens[b]), 0), table.shape[1] * P)
        for i in range(n):
            limit = min(max(length - n + i + 1, 0), length) if causal else length
            keys = [(int(table[b, j // P]), j % P) for j in range(limit)]
            keys = [(p, r) for p, r in keys if 0 <= p < k.shape[0]]
            if keys:
                pages, rows = torch.tensor([x[0] for x in keys]), torch.tensor([x[1] for x in keys])
                for h in range(H):
                    kk, vv = k[pages, rows, h // G], v[pages, rows, h // G]
                    s = sc * (kk @ q[row, h])
                    m = s.max()
                    e = torch.exp(s - m)
                    lse[row, h] = m + torch.log(e.sum())
                    p = e / e.sum()
                    out[row, h], spread[row, h] = p @ vv, p @ vv.abs()
                    reach[row, h] = abs(sc) * (kk.abs() @ q[row, h].abs()).max()
                    top[row, h] = vv.abs().max(0).values
            row += 1
    return out, lse, spread, reach, top


def attend_bounds(ref, n_keys, D, dtype, weight_dtype):
    """Elementwise bound on the output's error, and on the log-sum-exp's.

    A score is a sum of D products in 32 bits and a few multiplications: off
    by at most (D + 16) 2^-24 of sum |q| |k|, and so its weight by that much
    relatively, on both sides of the division; 2^-21 covers the base-2
    exponential (2 ulp) and its argument's rounding.  Each weight is then rounded to 16 bits (half a
    step, or half of fp16's least subnormal 2^-24 where the largest weight is
    at least 1), sums of n terms are off by n 2^-23 of the absolute sum, and
    the result is rounded once."""
    out, lse, spread, reach, top = ref
    e = (D + 16) * 2.0 ** -24 * reach + 2.0 ** -21 * (1 + reach)
    rel = half_step(weight_dtype) + 2 * e + 2 * n_keys * 2.0 ** -23
    tol = half_step(dtype) * out.abs() + rel[..., None] * spread * (1 + 2.0 ** -6)
    if weight_dtype == torch.float16:
        tol = tol + n_keys * 2.0 ** -25 * top
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25
    return tol + 1e-30, e + n_keys * 2.0 ** -23 + 2.0 ** -22 * (1 + lse.abs().nan_to_num(0, 0, 0))


def rotate(x, cos, sin, interleaved):
    """x [heads, D] in 64 bits."""
    half = cos.numel()
    y = x.clone()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    y[:, a] = x[:, a] * cos - x[:, b] * sin
    y[:, b] = x[:, b] * cos + x[:, a] * sin
    return y


def scale_for(amax):
    """The least power of two, in range, with amax <= 448 * scale."""
    if amax == 0:
        return 2.0 ** -50
    return 2.0 ** min(max(math.ceil(math.log2(amax / 448.0)), -50), 50)


def append(ck, cv, ks, vs, k, v, table, lens, counts, cos=None, sin=None, interleaved=False):
    """Appends to 64-bit pages ck, cv (values; with 8-bit scales ks, vs in 64
    bits) in place.  Returns {(page, row)} written and, for 8-bit caches,
    {(name, page, head)} whose scale grew."""
    P = ck.shape[1]
    token, written, grown = 0, set(), set()
    for b, n in enumerate(counts):
        fresh = {}
        for i in range(n):
            pos = int(lens[b]) - n + i
            t = token + i
            if pos < 0 or pos >= table.shape[1] * P or (cos is not None and pos >= cos.shape[0]):
                continue
            page = int(table[b, pos // P])
            if not 0 <= page < ck.shape[0]:
                continue
            kk, vv = k[t].cpu().double(), v[t].cpu().double()
            if cos is not None:
                kk = rotate(kk, cos[pos].cpu().double(), sin[pos].cpu().double(), interleaved)
            written.add((page, pos % P))
            fresh.setdefault(page, []).append((pos % P, kk, vv))
        for page, rows in fresh.items():
            for name, cache, scale, which in (("k", ck, ks, 1), ("v", cv, vs, 2)):
                for r in rows:
                    cache[page, r[0]] = r[which]
                if scale is None:
                    continue
                for h in range(cache.shape[2]):
                    new = torch.stack([r[which][h] for r in rows])
                    need = scale_for(float(new[torch.isfinite(new)].abs().max()) if torch.isfinite(new).any() else 0.0)
                    old = min(max(float(np.nan_to_num(scale[page, h].item(), nan=0.0)), 2.0 ** -50), 2.0 ** 50)
                    if rows[0][0] > 0 and need > old:
                        grown.add((name, page, h))
                    scale[page, h] = max(need, old) if rows[0][0] > 0 else need
        token += n
    return written, grown
