"""Precision of the attention over a paged cache where it is easily lost: small
weights beside a large one, small query elements beside a large one."""
import math

import pytest
import torch

from tests import paged_ref as ref

E4M3 = torch.float8_e4m3fn
gpu = pytest.mark.gpu


def paged(sdpa, k, v, P, cache, scale, seed):
    """A cache of one sequence's k, v [tokens, heads, D], its pages in any order; (cache, table)."""
    n, hkv, D = k.shape
    pages = -(-n // P)
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    tensors, kw = [], {}
    for name, x in (("k", k), ("v", v)):
        full = torch.zeros(pages * P, hkv, D)
        full[:n] = x
        t = torch.empty(pages, P, hkv, D, dtype=cache)
        t[perm] = (full / scale).view(pages, P, hkv, D).to(cache)
        tensors.append(t.cuda())
        if cache is E4M3:
            kw[name + "_scale"] = torch.full((pages, hkv), scale, device="cuda")
    return sdpa.SdpaPagedCache(*tensors, **kw), perm.to(torch.int32)[None]


def held(t, table, scale, n):
    """The n tokens that a cache's tensor holds, in 64 bits on the GPU."""
    return (t.view(torch.uint8 if t.dtype is E4M3 else torch.int16)[table[0].long().cuda()].view(t.dtype).double() * scale).flatten(0, 1)[:n]


def call(sdpa, q, c, table, n, causal=False, copies=1):
    """Of ``copies`` sequences with the same queries and pages."""
    rows, H, D = q.shape
    lens = torch.full((copies,), n, dtype=torch.int32, device="cuda")
    out, lse = sdpa.sdpa_paged_forward(q.repeat(copies, 1, 1), c, table.repeat(copies, 1).cuda(), lens, is_causal=causal,
                                       return_lse=True)
    assert sdpa.sdpa_last_device_status()[0] == 0
    return out.view(copies, rows * H, D), lse.view(copies, rows * H)


# rows: the form for few rows, half tiles, one full tile, two; one sequence, cut
# between many CTAs, and so many that each CTA takes whole ones
@gpu
@pytest.mark.parametrize("rows", [1, 12, 30, 70])
@pytest.mark.parametrize("copies", [1, 500])
@pytest.mark.parametrize("cache,dtype", [(E4M3, torch.bfloat16), (E4M3, torch.float16), (torch.float16, torch.float16),
                                         (torch.bfloat16, torch.bfloat16)])
@pytest.mark.parametrize("D,above", [(128, 26), (64, 20)])
def test_a_key_far_above_the_rest(sdpa_lib, rows, copies, cache, dtype, D, above):
    """The first key's weight is about 2^above times any other's and its value is zero, so that the
    output is what the small weights give.

    Rounded to 16 bits a weight is off by half a step of its own size, or, in fp16, by half of the
    least subnormal where the row's largest weight is 2^11 or more: 2^-36 of that largest weight,
    and the sum of weights is no less than it.  Scores: (D + 16) 2^-24 of sum |q| |k|, and 2^-21 (1
    + that) for the exponential, on both sides of the division; sums of n terms n 2^-23; the result
    is rounded once (fp16: or to within 2^-25)."""
    n, G, P = 9000, 4, 64
    g = torch.Generator().manual_seed(D + rows)
    k, v = torch.randn(n, 1, D, generator=g), torch.randn(n, 1, D, generator=g)
    q = torch.zeros(rows, G, D)
    q[..., 0] = 4.0                                 # (the scores of the others stay within +- 2)
    q[..., 1:] = torch.randn(rows, G, D - 1, generator=g) * 0.5
    k[:, :, 0] = 0.0
    k[0, 0, :] = 0.0
    k[0, 0, 0] = above * math.log(2.0) * math.sqrt(D) / 4.0
    v[0] = 0.0
    q = q.to(dtype).cuda()
    scale = 2.0 ** -2 if cache is E4M3 else 1.0
    c, table = paged(sdpa_lib, k, v, P, cache, scale, 3)
    out, lse = call(sdpa_lib, q, c, table, n, copies=copies)
    kk, vv = held(c.k, table, scale, n)[:, 0], held(c.v, table, scale, n)[:, 0]
    qd = q.double().flatten(0, 1)
    s = qd @ kk.T / math.sqrt(D)
    reach = (qd.abs() @ kk.T.abs() / math.sqrt(D)).amax(1, keepdim=True)
    p = torch.softmax(s, 1)
    assert float(p[:, 0].min()) > 0.97
    want, spread = p @ vv, p @ vv.abs()
    weight = torch.bfloat16 if cache is torch.bfloat16 else torch.float16
    e = (D + 16) * 2.0 ** -24 * reach + 2.0 ** -21 * (1 + reach)
    tol = ref.half_step(dtype) * want.abs() + (ref.half_step(weight) + 2 * e + 2 * n * 2.0 ** -23) * spread * (1 + 2.0 ** -6)
    if weight is torch.float16:
        tol = tol + 2.0 ** -36 * vv.abs().sum(0)
    if dtype is torch.float16:
        tol = tol + 2.0 ** -25
    off = (out.double() - want).abs()
    worst, size = (off / tol).max().item(), (off.pow(2).mean().sqrt() / want.pow(2).mean().sqrt()).item()
    assert worst <= 1, f"worst by {worst:.3g}, relative to the output's size {size:.3g}"
    want_lse = torch.logsumexp(s, 1)
    assert ((lse.double() - want_lse).abs() <= e[:, 0] + n * 2.0 ** -23 + 2.0 ** -22 * (1 + want_lse.abs())).all()


def query_error(D, rows, G, dtype):
    """What of its row's largest element a query element may be off by over an 8-bit cache: none down
    to 2^-13 of it; below, with more than 16 rows a head, half a step of the last of the e4m3 and
    e5m2 terms that carry it (two for bf16, three for fp16); with fewer, a bf16 row is fp16 under a
    power of two that takes the largest element to 2^14 or more."""
    if rows * G > 16:
        return 2.0 ** -21 if dtype is torch.bfloat16 else 2.0 ** -24
    return 2.0 ** -39 if dtype is torch.bfloat16 else 0.0


@gpu
@pytest.mark.parametrize("rows", [4, 5, 12, 30, 70])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ratio,exact", [(2 ** 8, False), (2 ** 11, True), (2 ** 12, False)])
def test_a_query_channel_far_above_the_rest(sdpa_lib, rows, dtype, D, ratio, exact):
    """One channel of the queries is 2^8 to 2^12 times the others, where the keys are small: the
    others decide the scores.  exact: no element is below 2^-13 of its row's largest, so none is
    off.  (Otherwise a score is off by that error times the sum of |k|.)  Other terms as above."""
    n, G, P = 300, 4, 32
    g = torch.Generator().manual_seed(D + rows)
    q = torch.randn(rows, G, D, generator=g)
    q[..., 5] = ratio * (1 + torch.rand(rows, G, generator=g)) / 2
    if exact:
        q = torch.where(q.abs() < 0.25, torch.copysign(torch.tensor(0.25), q), q)
    q = q.to(dtype).cuda()
    k, v = torch.randn(n, 1, D, generator=g), torch.randn(n, 1, D, generator=g)
    k[..., 5] = torch.randn(n, 1, generator=g) / ratio
    c, table = paged(sdpa_lib, k, v, P, E4M3, 2.0 ** -6, 3)
    out, lse = call(sdpa_lib, q, c, table, n, True)
    kk, vv = held(c.k, table, 2.0 ** -6, n)[:, 0], held(c.v, table, 2.0 ** -6, n)[:, 0]
    qd = q.double().flatten(0, 1)
    top = qd.abs().amax(1)
    if exact:
        assert (qd.abs().amin(1) >= 2.0 ** -13 * top).all()
    s = qd @ kk.T / math.sqrt(D)
    last = torch.arange(rows, device="cuda").repeat_interleave(G) + n - rows
    s = s.masked_fill(torch.arange(n, device="cuda")[None] > last[:, None], -math.inf)
    reach = (qd.abs() @ kk.T.abs() / math.sqrt(D)).amax(1)
    e = (D + 16) * 2.0 ** -24 * reach + 2.0 ** -21 * (1 + reach)
    if not exact:
        e = e + query_error(D, rows, G, dtype) * top * kk.abs().sum(1).max() / math.sqrt(D)
    p = torch.softmax(s, 1)
    want, spread = p @ vv, p @ vv.abs()
    tol = ref.half_step(dtype) * want.abs() + (ref.half_step(torch.float16) + 2 * e + 2 * n * 2.0 ** -23)[:, None] * spread * (1 + 2.0 ** -6)
    tol = tol + 2.0 ** -36 * vv.abs().sum(0)
    if dtype is torch.float16:
        tol = tol + 2.0 ** -25
    want_lse = torch.logsumexp(s, 1)
    off = (lse[0].double() - want_lse).abs() / (e + n * 2.0 ** -23 + 2.0 ** -22 * (1 + want_lse.abs()))
    assert off.max() <= 1, f"log-sum-exp: worst by {off.max().item():.3g}"
    bad = (out[0].double() - want).abs() / tol
    assert bad.max() <= 1, f"worst by {bad.max().item():.3g}"
