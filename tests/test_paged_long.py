"""The paged cache's operators where their loops run for long: many steps a CTA
(rings, notes, page windows and rescaling go round many times), many short
sequences a CTA, many sequences an append."""
import math

import numpy as np
import pytest
import torch

from tests import paged_ref as ref

E4M3 = torch.float8_e4m3fn
gpu = pytest.mark.gpu


def make(sdpa, n_pages, P, hkv, D, cache, seed, ramp=None):
    """A cache of random values; ramp: factors of the keys of each page."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    tensors, kw = [], {}
    for name in ("k", "v"):
        x = torch.randn(n_pages, P, hkv, D, generator=g, device="cuda")
        if name == "k" and ramp is not None:
            x *= ramp[:, None, None, None]
        if cache is E4M3:
            s = torch.exp2(torch.randint(-8, -4, (n_pages, hkv), generator=g, device="cuda").float())
            if seed % 2:
                s = s * (1 + torch.rand(n_pages, hkv, generator=g, device="cuda"))
            kw[name + "_scale"] = s
            x = (x / s[:, None, :, None]).clamp(-448, 448)
        tensors.append(x.to(cache))
    return sdpa.SdpaPagedCache(*tensors, **kw)


def attend64(q, c, table, lens, counts, causal):
    """In 64 bits on the GPU, a sequence and head at a time: (out, lse, spread, reach), the last two
    for the bounds: sum p |v|, and the largest sum |q| |k| over the keys; and sum p |v| of weights
    that may each be off by 2^-36 of the largest (all ones)."""
    total, H, D = q.shape
    P, hkv = c.page_size, c.n_kv_heads
    G = H // hkv
    shape = dict(dtype=torch.float64, device="cuda")
    out, spread, ones = (torch.zeros(total, H, D, **shape) for _ in range(3))
    lse, reach, loud = torch.full((total, H), -math.inf, **shape), torch.zeros(total, H, **shape), torch.zeros(total, H, **shape)
    row = 0
    for b, (n, length) in enumerate(zip(counts, lens)):
        if n == 0:
            continue
        ids = table[b, :-(-length // P)].long().cuda()
        here = ((ids >= 0) & (ids < c.n_pages)).repeat_interleave(P)[:length]
        ids = ids.clamp(0, c.n_pages - 1)
        kv = []
        for t, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
            x = t.view(torch.uint8 if s is not None else torch.int16)[ids].view(t.dtype).double()
            if s is not None:
                x = x * s[ids].double()[:, None, :, None]
            kv.append(x.flatten(0, 1)[:length])
        rows = slice(row, row + n)
        seen = here[None, :].expand(n, -1)
        if causal:
            last = torch.arange(n, device="cuda") + length - n
            seen = seen & (torch.arange(length, device="cuda")[None, :] <= last[:, None])
        seen = seen.repeat_interleave(G, 0)
        some = seen.any(1)
        for h in range(hkv):
            hs = slice(h * G, (h + 1) * G)
            k, v = kv[0][:, h], kv[1][:, h]
            qd = q[rows, hs].double().reshape(n * G, D)
            s = (qd @ k.T / math.sqrt(D)).masked_fill(~seen, -math.inf)
            lse[rows, hs] = torch.logsumexp(s, 1).view(n, G)
            p = torch.softmax(s, 1).nan_to_num(0.0)
            out[rows, hs], spread[rows, hs] = (p @ v).view(n, G, D), (p @ v.abs()).view(n, G, D)
            ones[rows, hs] = (v.abs() * here[:, None]).sum(0)
            size = k.abs() * here[:, None]
            reach[rows, hs] = ((qd.abs() @ size.T / math.sqrt(D)).amax(1) * some).view(n, G) if length else 0.0
            loud[rows, hs] = (qd.abs().amax(1) * size.sum(1).max() / math.sqrt(D)).view(n, G) if length else 0.0
        row += n
    return out, lse, spread, reach, ones, loud


def compare(sdpa, q, c, table, lens, counts, causal, max_q=None):
    """Scores: (D + 16) 2^-24 of sum |q| |k|, over 8-bit pages 2^-21 max |q| sum |k| for query elements
    below 2^-13 of the row's largest; 2^-21 (1 + that) for the exponential; on both sides of the
    division.  Weights: half a step of 16 bits, fp16 ones 2^-36 of the largest (times up to 2^5 for
    pages whose value scales lie that far apart).  Sums of n terms: n 2^-23.  The result: half a
    step, or 2^-25."""
    D = q.shape[2]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    args = (q, c, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), cu, max_q or max(counts))
    got, got_lse = sdpa.sdpa_paged_forward(*args, is_causal=causal, return_lse=True)
    assert sdpa.sdpa_last_device_status()[0] == 0
    again = sdpa.sdpa_paged_forward(*args, is_causal=causal, return_lse=True)
    assert torch.equal(got, again[0]) and torch.equal(got_lse, again[1])
    out, lse, spread, reach, ones, loud = attend64(q, c, table, lens, counts, causal)
    weight = torch.bfloat16 if c.k.dtype == torch.bfloat16 else torch.float16
    n = max(lens)
    e = (D + 16) * 2.0 ** -24 * reach + 2.0 ** -21 * (1 + reach)
    if c.k.dtype is E4M3:
        e = e + 2.0 ** -21 * loud
    tol = ref.half_step(q.dtype) * out.abs() + (ref.half_step(weight) + 2 * e + 2 * n * 2.0 ** -23)[..., None] * spread * (1 + 2.0 ** -6)
    if weight is torch.float16:
        tol = tol + 2.0 ** -31 * ones
    tol = tol + (2.0 ** -25 if q.dtype is torch.float16 else 1e-30)
    off = (got.double() - out).abs() / tol
    assert off.max() <= 1, f"out: worst by {off.max().item():.3g} at {(off == off.max()).nonzero()[0].tolist()}, {int((off > 1).sum())} of {off.numel()}"
    empty = torch.isinf(lse)
    assert torch.equal(torch.isinf(got_lse), empty) and (got[empty] == 0).all()
    off = ((got_lse.double() - lse).abs() / (e + n * 2.0 ** -23 + 2.0 ** -22 * (1 + lse.abs())))[~empty]
    assert off.max() <= 1, f"log-sum-exp: worst by {off.max().item():.3g}"


def long_tables(lens, P, seed, bad=0):
    """Page tables of sequences that fill a pool, in any order; ``bad`` entries of each are none."""
    g = torch.Generator().manual_seed(seed)
    per = [-(-n // P) for n in lens]
    pages = torch.randperm(sum(per), generator=g).to(torch.int32)
    table = torch.full((len(lens), max(per)), -1, dtype=torch.int32)
    for b, p in enumerate(pages.split(per)):
        table[b, :len(p)] = p
        for i in torch.randint(0, len(p), (bad,), generator=g).tolist():
            table[b, i] = -1 if i % 2 else sum(per) + i
    return table, sum(per)


LONG = [  # D, cache, dtype, page, kv heads, G, sequences, longest, rows, causal
    # few rows: four heads a unit, two, one (a warp each, two, four)
    (128, E4M3, torch.bfloat16, 16, 8, 4, 16, 13001, 1, True),
    (128, E4M3, torch.float16, 64, 2, 8, 64, 7003, 2, False),
    (128, torch.bfloat16, torch.bfloat16, 16, 1, 8, 64, 13000, 1, True),
    (64, E4M3, torch.bfloat16, 32, 4, 4, 40, 12345, 4, True),
    (64, torch.float16, torch.float16, 16, 4, 16, 40, 12345, 1, False),
    # half tiles: 17 to 64 rows a head
    (128, E4M3, torch.bfloat16, 16, 8, 8, 6, 12001, 5, True),
    (128, E4M3, torch.float16, 1024, 8, 4, 6, 13000, 16, False),
    (128, torch.bfloat16, torch.bfloat16, 16, 4, 16, 12, 12011, 3, True),
    (64, E4M3, torch.bfloat16, 64, 8, 6, 6, 14000, 7, True),
    (64, torch.float16, torch.float16, 16, 8, 8, 6, 12001, 4, True),
    # one full tile, both warpgroups in turn
    (128, E4M3, torch.bfloat16, 16, 8, 4, 6, 12001, 30, True),
    (128, torch.float16, torch.float16, 128, 4, 8, 12, 12345, 16, False),
    (64, E4M3, torch.float16, 32, 8, 4, 6, 13000, 32, True),
    (64, torch.bfloat16, torch.bfloat16, 16, 8, 4, 6, 12500, 17, True),
    # two, a warpgroup each; more than one unit a head
    (128, E4M3, torch.bfloat16, 64, 4, 8, 6, 12007, 70, True),
    (128, torch.bfloat16, torch.bfloat16, 16, 4, 4, 6, 13000, 100, True),
    (64, E4M3, torch.float16, 16, 4, 4, 6, 12001, 90, False),
    (64, torch.float16, torch.float16, 32, 4, 4, 6, 12003, 64, True),
]


@gpu
@pytest.mark.parametrize("case", LONG, ids=lambda c: f"D{c[0]}-{str(c[1])[6:]}-{str(c[2])[6:]}-P{c[3]}-{c[4]}x{c[5]}-{c[6]}x{c[7]}-{c[8]}")
def test_many_steps_a_cta(sdpa_lib, case):
    """24 steps a CTA and more; keys that grow along each sequence, so that the weights' base moves
    again and again; a few page entries that are none."""
    D, cache, dtype, P, hkv, G, B, longest, rows, causal = case
    g = torch.Generator().manual_seed(D + P + rows)
    lens = [longest - int(x) for x in torch.randint(0, longest // 8, (B,), generator=g)]
    counts = [rows] + [int(x) for x in torch.randint(max(1, rows // 2), rows + 1, (B - 1,), generator=g)]
    table, n_pages = long_tables(lens, P, 3, bad=3)
    ramp = torch.ones(n_pages)
    for b in range(B):
        ok = (table[b] >= 0) & (table[b] < n_pages)
        ramp[table[b][ok].long()] = (torch.arange(table.shape[1]).float() * P / longest * 2.5 + 0.25)[ok]
    c = make(sdpa_lib, n_pages, P, hkv, D, cache, rows, ramp.cuda())
    q = torch.randn(sum(counts), hkv * G, D, generator=g).to(dtype).cuda()
    compare(sdpa_lib, q, c, table, lens, counts, causal)


@gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,cache,dtype,hkv,G,big", [
    (128, E4M3, torch.bfloat16, 2, 4, 40), (128, torch.bfloat16, torch.bfloat16, 1, 8, 90),
    (64, E4M3, torch.float16, 1, 8, 6), (64, torch.float16, torch.float16, 2, 2, 300)])
@pytest.mark.parametrize("B", [100, 600, 1100])
def test_many_short_sequences(sdpa_lib, D, cache, dtype, hkv, G, big, B, causal):
    """More sequences than a block adds up at a time, several a CTA, in the forms for many rows: a
    few sequences have many rows, the others one or none."""
    g = torch.Generator().manual_seed(B + big)
    lens = [int(x) for x in torch.randint(0, 200, (B,), generator=g)]
    counts = [int(x) for x in torch.randint(0, 3, (B,), generator=g)]
    for b in (0, B // 2, B - 1):
        counts[b], lens[b] = big, big + 100 * (b % 3)
    table, n_pages = long_tables([max(n, 1) for n in lens], 16, 3)
    c = make(sdpa_lib, n_pages, 16, hkv, D, cache, B % 7)
    q = torch.randn(sum(counts), hkv * G, D, generator=g).to(dtype).cuda()
    compare(sdpa_lib, q, c, table, lens, counts, causal)


def turned(x, cos, sin, interleaved):
    """x [tokens, heads, D] in 32 bits: each product and each sum rounded on its own."""
    half = cos.shape[1]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    x1, x2, c, s = x[..., a], x[..., b], cos[:, None], sin[:, None]
    y = x.clone()
    p, r = x1 * c, x2 * s
    y[..., a] = p - r
    p, r = x2 * c, x1 * s
    y[..., b] = p + r
    return y


def append32(codes, scale, x, table, lens, counts, P):
    """x [tokens, heads, D] in 32 bits into pages on the CPU, in place."""
    t = 0
    for b, n in enumerate(counts):
        done, end = lens[b] - n, lens[b]
        while done < end:
            page, row = int(table[b, done // P]), done % P
            m = min(end - done, P - row)
            y = x[t:t + m]
            if scale is not None:
                need = torch.tensor([ref.scale_for(float(y[:, h].abs().max())) for h in range(x.shape[1])])
                now = torch.maximum(need, scale[page]) if row else need
                if row:
                    codes[page, :row] = (codes[page, :row].float() * (scale[page] / now)[:, None]).to(codes.dtype)
                scale[page] = now
                y = (y / now[:, None]).clamp(-448, 448)
            codes[page, row:row + m] = y.to(codes.dtype)
            done += m
            t += m


def same_append(sdpa, D, cache, dtype, P, hkv, H, rot, interleaved, lens, counts, seed):
    g = torch.Generator().manual_seed(seed)
    table, n_pages = long_tables([max(n, 1) for n in lens], P, seed)
    c = make(sdpa, n_pages, P, hkv, D, cache, 2 * seed)
    total = sum(counts)
    q, k, v = (torch.randn(total, n, D, generator=g).to(dtype) for n in (H, hkv, hkv))
    cos = sin = cos_t = sin_t = None
    if rot:
        at = torch.cat([torch.arange(L - n, L) for n, L in zip(counts, lens)])
        a = torch.rand(max(lens), rot // 2, generator=g) * 6.3
        cos, sin = a.cos(), a.sin()
        cos_t, sin_t = cos[at], sin[at]
    want_q, want_k = ((turned(x.float(), cos_t, sin_t, interleaved) if rot else x.float()) for x in (q, k))
    want = {}
    for name, x in (("k", want_k), ("v", v.float())):
        codes = getattr(c, name).cpu()
        scale = getattr(c, name + "_scale")
        scale = scale.cpu() if scale is not None else None
        append32(codes, scale, x, table, lens, counts, P)
        want[name] = codes, scale
    cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    got = sdpa.sdpa_cache_append(c, k.cuda(), v.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), cu,
                                 cos=cos.cuda() if rot else None, sin=sin.cuda() if rot else None, interleaved=interleaved, q=q.cuda())
    assert torch.equal(got.cpu(), want_q.to(dtype))
    for name, (codes, scale) in want.items():
        wide = torch.uint8 if cache is E4M3 else torch.int16
        assert torch.equal(getattr(c, name).cpu().view(wide), codes.view(wide)), name
        if scale is not None:
            assert torch.equal(getattr(c, name + "_scale").cpu(), scale), name


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,cache,dtype,rot", [(128, E4M3, torch.bfloat16, 128), (128, torch.bfloat16, torch.bfloat16, 128),
                                               (64, E4M3, torch.float16, 64), (64, torch.float16, torch.float16, 24),
                                               (128, E4M3, torch.float16, 40)])
def test_append_bit_for_bit(sdpa_lib, D, cache, dtype, rot, interleaved):
    """Rotated queries, keys, codes and scales equal those of separate 32-bit operations."""
    same_append(sdpa_lib, D, cache, dtype, 32, 3, 5, rot, interleaved, [70, 33, 500], [61, 33, 130], D + rot)


@gpu
@pytest.mark.parametrize("cache,dtype", [(E4M3, torch.bfloat16), (torch.float16, torch.float16)])
@pytest.mark.parametrize("B,most", [(33, 40), (64, 1), (200, 9), (1000, 2)])
def test_append_for_many_sequences(sdpa_lib, cache, dtype, B, most):
    """Ragged, some without new tokens: every token finds its sequence's pages."""
    g = torch.Generator().manual_seed(B)
    counts = [int(x) for x in torch.randint(0, most + 1, (B,), generator=g)]
    counts[0] = counts[-1] = 0
    counts[B // 2] = most
    lens = [n + int(x) for n, x in zip(counts, torch.randint(0, 50, (B,), generator=g))]
    same_append(sdpa_lib, 64, cache, dtype, 16, 2, 4, 64, False, lens, counts, B)


@gpu
@pytest.mark.parametrize("cache", ["e4m3", "16"])
def test_append_allocates_the_queries(sdpa_lib, cache):
    """q_out allocated by the call: rows of tokens that have a place are the rotated queries (the
    others are left as allocated); in place the others keep their queries."""
    from tests.test_paged import make_cache
    c = make_cache(sdpa_lib, 6, 16, 1, 64, cache, torch.bfloat16, 4)
    g = torch.Generator().manual_seed(1)
    k, v, q = (torch.randn(23, n, 64, generator=g).bfloat16().cuda() for n in (1, 1, 3))
    a = torch.rand(30, 32, generator=g)
    cos, sin = a.cos().cuda(), a.sin().cuda()
    table = torch.tensor([[4, 1], [2, 77]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([3, 35], dtype=torch.int32, device="cuda")           # positions -2 .. 2, 20 .. 34
    cu = torch.tensor([0, 5, 20], dtype=torch.int32, device="cuda")
    placed = list(range(2, 5)) + list(range(5, 15))                          # 30 is past the angles; a bad page has a place
    at = torch.tensor([0, 1, 2] + list(range(20, 30)))
    want = turned(q.float().cpu()[placed], a.cos()[at], a.sin()[at], False).bfloat16()
    got = sdpa_lib.sdpa_cache_append(c, k, v, table, lens, cu, cos=cos, sin=sin, q=q)
    assert torch.equal(got.cpu()[placed], want)
    before = q.clone()
    assert sdpa_lib.sdpa_cache_append(c, k, v, table, lens, cu, cos=cos, sin=sin, q=q, q_out=q) is q
    assert torch.equal(q.cpu()[placed], want)
    rest = [i for i in range(23) if i not in placed]
    assert torch.equal(q[rest], before[rest])
