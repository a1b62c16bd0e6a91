"""The paged cache's operators against their plain 64-bit forms: appending
(rotation, 16-bit and e4m3 pages), attention of a few or many new tokens, and
the two together as a decoding loop."""
import math

import numpy as np
import pytest
import torch

from tests import paged_ref as ref

E4M3 = torch.float8_e4m3fn
gpu = pytest.mark.gpu


def layout(shape, kind, dtype, gen):
    """An uninitialised [pages, tokens, heads, D] cache tensor in one of several memory orders."""
    n, P, H, D = shape
    if kind == "heads":          # [pages, heads, tokens, D]
        return torch.empty(n, H, P, D, dtype=dtype, device="cuda").transpose(1, 2)
    if kind == "padded":         # rows of a wider buffer
        return torch.empty(n, P, H, D + 64, dtype=dtype, device="cuda")[..., :D]
    return torch.empty(n, P, H, D, dtype=dtype, device="cuda")


def make_cache(sdpa, n_pages, P, hkv, D, cache, dtype, seed, kind="tokens", spread=1.0, stale=None):
    """A cache full of random values; ``stale``: what else it may hold (set by the caller)."""
    g = torch.Generator().manual_seed(seed)
    kw = {}
    tensors = []
    for name in ("k", "v"):
        x = torch.randn(n_pages, P, hkv, D, generator=g) * spread
        if cache == "e4m3":
            s = torch.exp2(torch.randint(-9, -5, (n_pages, hkv), generator=g).float())
            if seed % 2:   # scales need not be powers of two
                s = s * (1 + torch.rand(n_pages, hkv, generator=g))
            t = layout(x.shape, kind, E4M3, g)
            t.copy_((x / s[:, None, :, None]).clamp(-448, 448).to(E4M3))
            kw[name + "_scale"] = s.cuda()
        else:
            t = layout(x.shape, kind, dtype, g)
            t.copy_(x.to(dtype))
        tensors.append(t)
    return sdpa.SdpaPagedCache(*tensors, **kw)


def tables(B, max_pages, n_pages, seed):
    g = torch.Generator().manual_seed(seed + 5)
    return torch.randperm(n_pages, generator=g)[:B * max_pages].view(B, max_pages).to(torch.int32)


def check(got, want, tol, what):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst by "
                           f"{((got - want).abs() / tol)[bad].max().item():.3g} at {bad.nonzero()[0].tolist()}")


def run_attend(sdpa, cache, q, table, lens, counts, causal, scale=None, use_cu=True, max_q=None, **kw):
    cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda") if use_cu else None
    out, lse = sdpa.sdpa_paged_forward(q, cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), cu,
                                       (max(counts) if max_q is None else max_q) if use_cu else None,
                                       is_causal=causal, scale=scale, return_lse=True, **kw)
    k, v = ref.values(cache.k, cache.k_scale), ref.values(cache.v, cache.v_scale)
    want = ref.attend(q, k, v, table, lens, counts, scale, causal)
    weight = torch.bfloat16 if cache.k.dtype == torch.bfloat16 else torch.float16
    tol, lse_tol = ref.attend_bounds(want, max(1, max(lens)), q.shape[2], q.dtype, weight)
    check(out, want[0], tol, "out")
    empty = torch.isinf(want[1])
    assert torch.equal(torch.isinf(lse.cpu()), empty)
    assert torch.all(out.cpu()[empty] == 0)
    check(lse.cpu()[~empty], want[1][~empty], lse_tol[~empty], "lse")
    return out, lse


ATTEND = [  # D, cache, dtype, page, kv heads, G, memory order, causal, counts, lengths
    (128, "e4m3", torch.bfloat16, 16, 2, 4, "tokens", True, [1, 1, 1, 1, 1], [1, 0, 16, 17, 333]),
    (128, "e4m3", torch.float16, 64, 1, 16, "heads", True, [1, 1, 1], [63, 64, 65]),
    (128, "16", torch.bfloat16, 32, 2, 8, "tokens", False, [2, 1, 2], [100, 5, 257]),
    (128, "16", torch.float16, 16, 3, 1, "padded", True, [1, 7, 16], [130, 7, 9]),
    (64, "e4m3", torch.bfloat16, 128, 2, 7, "heads", True, [1, 3, 4], [200, 3, 500]),
    (64, "e4m3", torch.float16, 16, 4, 1, "padded", True, [1, 1], [1000, 31]),
    (64, "16", torch.bfloat16, 64, 1, 3, "heads", False, [5, 2], [129, 64]),
    (64, "16", torch.float16, 32, 2, 16, "tokens", True, [1, 2, 1], [700, 33, 2]),
    (128, "e4m3", torch.bfloat16, 32, 1, 5, "tokens", True, [40, 1, 9], [90, 300, 9]),
    (128, "e4m3", torch.bfloat16, 64, 2, 8, "tokens", True, [33, 70, 1], [33, 260, 150]),
    (128, "16", torch.bfloat16, 16, 1, 8, "heads", True, [130, 3], [400, 129]),
    (64, "16", torch.float16, 128, 1, 4, "tokens", True, [77, 5], [300, 64]),
    (64, "e4m3", torch.bfloat16, 16, 1, 64, "tokens", True, [5, 1], [129, 200]),
    (128, "e4m3", torch.float16, 16, 1, 33, "padded", False, [6, 2], [129, 640]),
    (64, "e4m3", torch.float16, 32, 2, 8, "heads", True, [20, 1, 260], [20, 700, 300]),
    (128, "16", torch.float16, 64, 1, 16, "heads", False, [9, 33], [513, 128]),
    (64, "16", torch.bfloat16, 16, 4, 4, "padded", True, [70, 11], [200, 11]),
    (128, "e4m3", torch.bfloat16, 16, 8, 4, "tokens", True, [1, 3, 1, 0], [130, 3, 77, 12]),
    (64, "e4m3", torch.float16, 256, 4, 8, "tokens", True, [4, 2], [600, 31]),
    (128, "16", torch.bfloat16, 1024, 4, 2, "tokens", True, [1, 16], [1500, 16]),
    (64, "16", torch.float16, 512, 6, 1, "heads", False, [1, 2], [515, 40]),
    (128, "e4m3", torch.float16, 32, 2, 8, "heads", True, [5, 8, 1, 0], [300, 8, 129, 4]),
    (128, "16", torch.bfloat16, 64, 3, 16, "tokens", True, [4, 3, 1], [1000, 3, 128]),
    (64, "16", torch.float16, 16, 1, 48, "padded", False, [1, 1], [257, 40]),
]


@gpu
@pytest.mark.parametrize("case", ATTEND, ids=lambda c: f"D{c[0]}-{c[1]}-{str(c[2])[6:]}-P{c[3]}-{c[4]}x{c[5]}-{c[6]}-{c[8]}")
def test_attend(sdpa_lib, case):
    D, cache, dtype, P, hkv, G, kind, causal, counts, lens = case
    seed = D + P + hkv * 10 + G
    mp = -(-max(lens) // P) + 1
    n_pages = len(lens) * mp + 2
    c = make_cache(sdpa_lib, n_pages, P, hkv, D, cache, dtype, seed, kind)
    q = torch.randn(sum(counts), hkv * G, D, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()
    run_attend(sdpa_lib, c, q, tables(len(lens), mp, n_pages, seed), lens, counts, causal)


@gpu
@pytest.mark.parametrize("cache", ["e4m3", "16"])
@pytest.mark.parametrize("rows", [1, 2, 40])
def test_attend_many_ctas_a_sequence(sdpa_lib, cache, rows):
    """One long sequence, cut between all CTAs and joined again; any max_seqlen_q gives the results."""
    lens, P = [9001], 64
    c = make_cache(sdpa_lib, 142, P, 1, 128, cache, torch.bfloat16, 7)
    q = torch.randn(rows, 4, 128, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    t = tables(1, 141, 142, 3)
    a = run_attend(sdpa_lib, c, q, t, lens, [rows], True)
    b = run_attend(sdpa_lib, c, q, t, lens, [rows], True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    run_attend(sdpa_lib, c, q, t, lens, [rows], True, max_q=1)
    run_attend(sdpa_lib, c, q, t, lens, [rows], True, max_q=5000)


@gpu
@pytest.mark.parametrize("hkv,G", [(4, 2), (8, 1), (2, 3)])
def test_attend_many_ctas_and_heads(sdpa_lib, hkv, G):
    """Units of several heads, cut between CTAs; any bound on the rows gives the results, with
    what sdpa_paged_workspace_bytes says for it."""
    lens = [2500, 1, 700]
    c = make_cache(sdpa_lib, 170, 32, hkv, 64, "e4m3", torch.bfloat16, 9)
    q = torch.randn(3, hkv * G, 64, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    t = tables(3, 79, 3 * 79, 3) % 170
    for max_q in (1, 7, 30, 4000):
        run_attend(sdpa_lib, c, q, t, lens, [1, 1, 1], True, max_q=max_q)


@gpu
@pytest.mark.parametrize("rows", [1, 40])
def test_shared_pages_and_lengths_out_of_range(sdpa_lib, rows):
    """Sequences with pages in common; lengths below zero and past the table are clamped."""
    c = make_cache(sdpa_lib, 9, 16, 2, 128, "e4m3", torch.bfloat16, 30)
    table = torch.tensor([[3, 5, 7, 1], [3, 5, 2, 0], [3, 5, 7, 8]], dtype=torch.int32)
    q = torch.randn(3 * rows, 8, 128, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    lens = torch.tensor([50, -7, 1 << 30], dtype=torch.int32).cuda()
    out, lse = sdpa_lib.sdpa_paged_forward(q, c, table.cuda(), lens, is_causal=True, return_lse=True)
    k, v = ref.values(c.k, c.k_scale), ref.values(c.v, c.v_scale)
    want = ref.attend(q, k, v, table, [50, 0, 64], [rows] * 3, None, True)
    tol, _ = ref.attend_bounds(want, 64, 128, torch.bfloat16, torch.float16)
    check(out, want[0], tol, "out")
    assert torch.isinf(lse[rows:2 * rows]).all() and (out[rows:2 * rows] == 0).all()


@gpu
@pytest.mark.parametrize("rows_max", [1, 60])
def test_bad_offsets_stay_inside(sdpa_lib, rows_max):
    """Offsets out of order and out of range: rows of one sequence only are right, nothing else is
    touched."""
    c = make_cache(sdpa_lib, 9, 16, 1, 64, "e4m3", torch.float16, 31)
    buf = torch.full((10, 2, 64), 5.0, dtype=torch.float16, device="cuda")
    q = torch.randn(6, 2, 64, generator=torch.Generator().manual_seed(3)).half().cuda()
    table = tables(3, 2, 9, 1)
    cu = torch.tensor([-4, 4, 2, 99], dtype=torch.int32).cuda()   # rows 0-3, none, 2-5
    lens = torch.tensor([20, 20, 30], dtype=torch.int32).cuda()
    sdpa_lib.sdpa_paged_forward(q, c, table.cuda(), lens, cu, rows_max, buf[2:8])
    assert sdpa_lib.sdpa_last_device_status()[0] == 0
    k, v = ref.values(c.k, c.k_scale), ref.values(c.v, c.v_scale)
    for b, r in ((0, slice(0, 2)), (2, slice(4, 6))):
        want = ref.attend(q[r], k, v, table[b:b + 1], [int(lens[b])], [2])
        tol, _ = ref.attend_bounds(want, 30, 64, torch.float16, torch.float16)
        check(buf[2:8][r], want[0], tol, "out")
    assert (buf[:2] == 5).all() and (buf[8:] == 5).all()
    before = [x.clone() for x in (c.k.view(torch.uint8), c.v.view(torch.uint8))]
    kn = torch.randn(6, 1, 64, generator=torch.Generator().manual_seed(3)).half().cuda()
    sdpa_lib.sdpa_cache_append(c, kn, kn, table[:, :1].contiguous().cuda(), torch.tensor([4, 0, 4], dtype=torch.int32).cuda(), cu)
    torch.cuda.synchronize()
    touched = [int(table[0, 0]), int(table[2, 0])]
    rest = [p for p in range(9) if p not in touched]
    for x, y in zip(before, (c.k.view(torch.uint8), c.v.view(torch.uint8))):
        assert torch.equal(x[rest], y[rest]) and torch.equal(x[touched, 4:], y[touched, 4:])


@gpu
def test_waits_run_out(sdpa_lib):
    """The many-row kernel's waits are bounded: with its products withheld it returns, says so, and
    the next call is right."""
    c = make_cache(sdpa_lib, 20, 16, 1, 128, "e4m3", torch.bfloat16, 8)
    q = torch.randn(50, 2, 128, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    t = tables(1, 9, 20, 3)
    lens = torch.tensor([140], dtype=torch.int32).cuda()
    assert sdpa_lib.sdpa_last_device_status()[0] == 0
    sdpa_lib.sdpa_debug_set_wait_limit_ns(20_000_000)
    sdpa_lib.sdpa_debug_withhold_q_load(True)
    try:
        sdpa_lib.sdpa_paged_forward(q, c, t.cuda(), lens)
        rc, bits = sdpa_lib.sdpa_last_device_status()
    finally:
        sdpa_lib.sdpa_debug_withhold_q_load(False)
        sdpa_lib.sdpa_debug_set_wait_limit_ns(0)
    assert rc == 8 and bits & 1
    run_attend(sdpa_lib, c, q, t, [140], [50], True)
    assert sdpa_lib.sdpa_last_device_status()[0] == 0


@gpu
@pytest.mark.parametrize("rows", [50, 300])
def test_waits_run_out_over_a_used_workspace(sdpa_lib, monkeypatch, rows):
    """A workspace may hold anything: what it says of units to join is not followed when a call
    gives up."""
    c = make_cache(sdpa_lib, 20, 16, 1, 128, "e4m3", torch.bfloat16, 8)
    q = torch.randn(rows, 2, 128, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    t = tables(1, 19, 20, 3)
    lens = torch.tensor([300], dtype=torch.int32).cuda()
    plain = torch.empty

    def used(*a, **kw):
        x = plain(*a, **kw)
        return x.fill_(0x7f) if x.dtype == torch.uint8 else x

    monkeypatch.setattr(torch, "empty", used)
    sdpa_lib.sdpa_debug_set_wait_limit_ns(20_000_000)
    sdpa_lib.sdpa_debug_withhold_q_load(True)
    try:
        sdpa_lib.sdpa_paged_forward(q, c, t.cuda(), lens)
        rc, bits = sdpa_lib.sdpa_last_device_status()
    finally:
        sdpa_lib.sdpa_debug_withhold_q_load(False)
        sdpa_lib.sdpa_debug_set_wait_limit_ns(0)
    assert rc == 8 and bits & 1
    run_attend(sdpa_lib, c, q, t, [300], [rows], True)
    assert sdpa_lib.sdpa_last_device_status()[0] == 0


@gpu
@pytest.mark.parametrize("batch", [129, 300])
def test_attend_large_batches(sdpa_lib, batch):
    g = torch.Generator().manual_seed(batch)
    lens = [int(x) for x in torch.randint(0, 70, (batch,), generator=g)]
    c = make_cache(sdpa_lib, batch * 5 + 1, 16, 1, 64, "e4m3", torch.float16, 4)
    q = torch.randn(batch, 2, 64, generator=g).half().cuda()
    run_attend(sdpa_lib, c, q, tables(batch, 5, batch * 5 + 1, 4), lens, [1] * batch, True, use_cu=False)


@gpu
@pytest.mark.parametrize("rows", [1, 50])
@pytest.mark.parametrize("cache", ["e4m3", "16"])
def test_pages_beyond_the_length_may_hold_anything(sdpa_lib, cache, rows):
    """NaN and infinities behind a sequence's end, in its last page and in pages past it, bad
    page entries past it, and a bad entry inside (its keys are removed)."""
    P, lens = 16, [37, 52]
    dtype = torch.bfloat16
    c = make_cache(sdpa_lib, 9, P, 2, 128, cache, dtype, 6)
    table = tables(2, 4, 9, 11)
    clean = c.k.clone(), c.v.clone()
    for b, n in enumerate(lens):
        for t, x in ((c.k, math.nan), (c.v, math.nan), (c.v, math.inf)):
            junk = torch.full((P, 2, 128), x).to(t.dtype).cuda()
            for pg in range(n // P, 4):
                keep = max(0, n - pg * P)
                if pg * P + P > n:
                    t[int(table[b, pg]), keep:].view(torch.uint8).copy_(junk[keep:].contiguous().view(torch.uint8))
    q = torch.randn(2 * rows, 8, 128, generator=torch.Generator().manual_seed(9)).to(dtype).cuda()
    # the 64-bit form must not meet the junk through 0 * NaN: it indexes keys, so it does not
    run_attend(sdpa_lib, c, q, table, lens, [rows, rows], True)
    table[0, 3], table[1, 1] = -1, 9
    run_attend(sdpa_lib, c, q, table, lens, [rows, rows], False)
    c.k.copy_(clean[0]), c.v.copy_(clean[1])


@gpu
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.7])
@pytest.mark.parametrize("cache", ["e4m3", "16"])
def test_scales_of_the_scores(sdpa_lib, cache, scale):
    c = make_cache(sdpa_lib, 20, 32, 2, 64, cache, torch.bfloat16, 8, spread=0.5)
    q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    run_attend(sdpa_lib, c, q, tables(3, 6, 20, 2), [150, 1, 65], [1, 1, 1], True, scale=scale)


@gpu
@pytest.mark.parametrize("rows", [1, 20])
def test_uneven_page_scales(sdpa_lib, rows):
    """Pages whose value scales lie far apart: the weight of a key carries its page's scale."""
    c = make_cache(sdpa_lib, 12, 16, 1, 128, "e4m3", torch.bfloat16, 10, spread=0.3)
    e = torch.randint(-20, 12, (12, 1), generator=torch.Generator().manual_seed(1))
    c.v_scale.copy_(torch.exp2(e.float()))
    q = torch.randn(2 * rows, 4, 128, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    run_attend(sdpa_lib, c, q, tables(2, 5, 12, 2), [77, 80], [rows, rows], True)


@gpu
def test_scales_out_of_range_are_taken_as_the_nearest(sdpa_lib):
    c = make_cache(sdpa_lib, 6, 16, 1, 64, "e4m3", torch.float16, 12)
    q = torch.randn(1, 2, 64, generator=torch.Generator().manual_seed(2)).half().cuda()
    c.v_scale.copy_(torch.tensor([[0.0], [math.nan], [-1.0], [0.01], [0.02], [0.0]]))
    c.k_scale.copy_(torch.tensor([[0.0], [0.01], [0.01], [0.01], [math.nan], [0.0]]))
    table = torch.arange(5, dtype=torch.int32)[None]
    out, lse = sdpa_lib.sdpa_paged_forward(q, c, table.cuda(), torch.tensor([80], dtype=torch.int32).cuda(), return_lse=True)
    least = 2.0 ** -50
    sv = torch.tensor([[least], [least], [least], [0.01], [0.02], [least]])
    sk = torch.tensor([[least], [0.01], [0.01], [0.01], [least], [least]])
    want = ref.attend(q, ref.values(c.k, sk), ref.values(c.v, sv), table, [80], [1])
    tol, lse_tol = ref.attend_bounds(want, 80, 64, torch.float16, torch.float16)
    check(out, want[0], tol, "out")
    check(lse, want[1], lse_tol, "lse")


@gpu
@pytest.mark.parametrize("size", [1e-30, 1e30])
def test_small_and_large_queries(sdpa_lib, size):
    """bf16 queries far outside fp16's range over an 8-bit cache."""
    c = make_cache(sdpa_lib, 8, 16, 1, 128, "e4m3", torch.bfloat16, 14)
    q = (torch.randn(2, 3, 128, generator=torch.Generator().manual_seed(4)) * size).bfloat16().cuda()
    run_attend(sdpa_lib, c, q, tables(2, 4, 8, 1), [50, 64], [1, 1], True, scale=0.1 / size)


@gpu
@pytest.mark.parametrize("rows", [1, 64])
def test_strided_views_and_rows_behind_the_last_sequence(sdpa_lib, rows):
    """q cut from rows of queries, keys and values; out and lse into wider buffers; rows beyond
    cu_seqlens[-1] stay as they were."""
    H, D, total = 8, 128, 2 * rows + 3
    c = make_cache(sdpa_lib, 20, 16, 2, D, "16", torch.bfloat16, 20)
    qkv = torch.randn(total, H + 4, D, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    q = qkv[:, :H]
    out = torch.full((total, H, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((total, 2 * H), 7.0, device="cuda")
    table, lens = tables(2, 9, 20, 5), [140, 75]
    cu = torch.tensor([0, rows, 2 * rows], dtype=torch.int32, device="cuda")
    sdpa_lib.sdpa_paged_forward(q, c, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), cu, rows,
                                out[..., :D], is_causal=True, lse=lse[:, ::2])
    want = ref.attend(q[:2 * rows], ref.values(c.k), ref.values(c.v), table, lens, [rows, rows], None, True)
    tol, lse_tol = ref.attend_bounds(want, 140, D, torch.bfloat16, torch.bfloat16)
    check(out[:2 * rows, :, :D], want[0], tol, "out")
    check(lse[:2 * rows, ::2], want[1], lse_tol, "lse")
    assert (out[2 * rows:] == 7).all() and (out[..., D:] == 7).all()
    assert (lse[2 * rows:] == 7).all() and (lse[:, 1::2] == 7).all()


@gpu
def test_offsets_past_32_bits(sdpa_lib):
    """A cache of more than 2^32 elements: pages at its far end."""
    P, D, hkv, n_pages = 64, 128, 8, 66000
    k = torch.empty(n_pages, P, hkv, D, dtype=E4M3, device="cuda")
    v = torch.empty_like(k)
    sk, sv = torch.ones(n_pages, hkv, device="cuda"), torch.ones(n_pages, hkv, device="cuda")
    g = torch.Generator().manual_seed(1)
    far = [n_pages - 1, 65537, 3]
    for t in (k, v):
        for p in far:
            t[p] = torch.randn(P, hkv, D, generator=g).to(E4M3).cuda()
    c = sdpa_lib.SdpaPagedCache(k, v, sk, sv)
    q = torch.randn(2, 16, D, generator=g).bfloat16().cuda()
    table = torch.tensor([[far[0], far[1]], [far[2], far[0]]], dtype=torch.int32)
    out = sdpa_lib.sdpa_paged_forward(q, c, table.cuda(), torch.tensor([128, 100], dtype=torch.int32).cuda())
    kk, vv = (torch.stack([t[p].float().cpu().double() for p in far]) for t in (k, v))
    want = ref.attend(q, kk, vv, torch.tensor([[0, 1], [2, 0]]), [128, 100], [1, 1])
    tol, _ = ref.attend_bounds(want, 128, D, torch.bfloat16, torch.float16)
    check(out, want[0], tol, "out")
    # and appended to
    kn, vn = (torch.randn(2, hkv, D, generator=g).bfloat16().cuda() for _ in range(2))
    sdpa_lib.sdpa_cache_append(c, kn, vn, table.cuda(), torch.tensor([65, 65], dtype=torch.int32).cuda())
    for b, p in enumerate((far[1], far[0])):
        for t, s, x in ((k, sk, kn), (v, sv, vn)):
            got = t[p, 0].float() * s[p][:, None]
            assert ((got - x[b].float()).abs() <= 2.0 ** -4 * x[b].float().abs() + s[p][:, None] * 2.0 ** -10).all()


APPEND = [  # D, cache, dtype, page, kv heads, H, rot, interleaved, counts, lengths with the new tokens
    (128, "e4m3", torch.bfloat16, 16, 2, 8, 128, False, [1, 1, 1, 0], [1, 16, 17, 40]),
    (128, "e4m3", torch.bfloat16, 64, 8, 32, 128, False, [130, 1, 64], [130, 63, 100]),
    (128, "e4m3", torch.float16, 32, 3, 6, 64, True, [5, 33, 70], [37, 33, 95]),
    (64, "e4m3", torch.bfloat16, 16, 5, 10, 64, True, [17, 2], [50, 2]),
    (64, "e4m3", torch.float16, 128, 1, 64, 8, False, [200, 1, 3], [300, 7, 128]),
    (128, "16", torch.bfloat16, 16, 2, 16, 128, False, [1, 40, 0, 3], [9, 47, 3, 16]),
    (64, "16", torch.float16, 32, 16, 16, 32, True, [33, 1], [65, 1]),
    (64, "16", torch.bfloat16, 16, 1, 7, 0, False, [3, 20], [3, 50]),
    (128, "e4m3", torch.bfloat16, 16, 2, 0, 0, False, [3, 20], [20, 50]),
]


@gpu
@pytest.mark.parametrize("kind", ["tokens", "heads", "padded"])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"D{c[0]}-{c[1]}-{str(c[2])[6:]}-P{c[3]}-{c[4]}-{c[5]}-rot{c[6]}-{c[8]}")
def test_append(sdpa_lib, case, kind):
    D, cache, dtype, P, hkv, H, rot, inter, counts, lens = case
    g = torch.Generator().manual_seed(D + P + hkv)
    mp = -(-max(lens) // P)
    n_pages = len(lens) * mp + 2
    c = make_cache(sdpa_lib, n_pages, P, hkv, D, cache, dtype, 2 * D + P, kind)
    if cache == "e4m3":      # some pages' scales are too small for what comes, some are large enough
        for s in (c.k_scale, c.v_scale):
            s.copy_(torch.exp2(torch.randint(-12, -4, s.shape, generator=g).float()))
    total = sum(counts)
    k, v = (torch.randn(total, hkv, D, generator=g).to(dtype).cuda() for _ in range(2))
    q = torch.randn(total, H, D, generator=g).to(dtype).cuda() if H else None
    cos = sin = None
    if rot:
        a = torch.rand(max(lens) + 1, rot // 2, generator=g) * 6.3
        cos, sin = a.cos().cuda(), a.sin().cuda()
    table = tables(len(lens), mp, n_pages, 1)
    before = [t.clone() for t in (c.k, c.v)]
    ck, cv = ref.values(c.k, c.k_scale), ref.values(c.v, c.v_scale)
    ks, vs = (None, None) if cache == "16" else (c.k_scale.cpu().double(), c.v_scale.cpu().double())
    old_ks, old_vs = (None, None) if ks is None else (ks.clone(), vs.clone())
    written, grown = ref.append(ck, cv, ks, vs, k, v, table, lens, counts, cos, sin, inter)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    qo = sdpa_lib.sdpa_cache_append(c, k, v, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), cu,
                                    cos=cos, sin=sin, interleaved=inter, q=q)
    mask = torch.zeros(n_pages, P, dtype=torch.bool)
    for p, r in written:
        mask[p, r] = True
    # the rotation: three roundings to 32 bits of terms no larger than |x1| + |x2|
    turn = 2.0 ** -22 * 8
    for name, got, want, s, old, was in (("k", c.k, ck, c.k_scale, old_ks, before[0]), ("v", c.v, cv, c.v_scale, old_vs, before[1])):
        want_s = ks if name == "k" else vs
        x = ref.values(got, s)
        if cache == "16":
            tol = ref.half_step(dtype) * want.abs() * (1 + 2.0 ** -10) + turn
            check(x[mask], want[mask], tol[mask], name)
            assert torch.equal(got.cpu()[~mask], was.cpu()[~mask])
            continue
        assert torch.equal(s.cpu().double(), want_s), name
        step = (ref.half_step(E4M3) * want.abs() * (1 + 2.0 ** -10) + want_s[:, None, :, None] * 2.0 ** -10 + turn)
        check(x[mask], want[mask], step[mask], name)
        kept = torch.ones(n_pages, hkv, dtype=torch.bool)
        for nm, p, h in grown:
            if nm == name:
                kept[p, h] = False
        # codes under a scale that did not grow are untouched; others are rounded once more
        same = (~mask)[:, :, None, None] & kept[:, None, :, None]
        fresh = torch.zeros(n_pages, hkv, dtype=torch.bool)
        for p, r in written:
            if r == 0:
                fresh[p] = True
        assert torch.equal(got.cpu().float()[same.expand_as(x)], was.cpu().float()[same.expand_as(x)])
        grew = (~mask)[:, :, None, None] & (~kept & ~fresh)[:, None, :, None]
        first = {p: min(r for pp, r in written if pp == p) for p, _ in written}
        rows = torch.zeros(n_pages, P, dtype=torch.bool)
        for p, r0 in first.items():
            rows[p, :r0] = True
        grew = (grew & rows[:, :, None, None]).expand_as(x)
        check(x[grew], want[grew], step[grew], name + " earlier rows")
    if q is not None:
        want = q.cpu().double()
        t = 0
        for b, n in enumerate(counts):
            for i in range(n):
                if rot:
                    pos = lens[b] - n + i
                    want[t] = ref.rotate(want[t], cos[pos].cpu().double(), sin[pos].cpu().double(), inter)
                t += 1
        check(qo, want, ref.half_step(dtype) * want.abs() * (1 + 2.0 ** -10) + turn, "q")


@gpu
def test_append_in_place_from_one_buffer(sdpa_lib):
    """q, k and v cut from one buffer of rows, q rotated in place; the result equals separate tensors'."""
    H, hkv, D, total = 8, 2, 128, 37
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn(total, H + 2 * hkv, D, generator=g).bfloat16().cuda()
    a = torch.rand(64, D // 2, generator=g) * 6
    cos, sin = a.cos().cuda(), a.sin().cuda()
    table, lens = tables(1, 4, 5, 1).cuda(), torch.tensor([40], dtype=torch.int32, device="cuda")
    caches = [make_cache(sdpa_lib, 5, 16, hkv, D, "e4m3", torch.bfloat16, 4) for _ in range(2)]
    q, k, v = qkv[:, :H], qkv[:, H:H + hkv], qkv[:, H + hkv:]
    apart = sdpa_lib.sdpa_cache_append(caches[0], k.clone(), v.clone(), table, lens, cos=cos, sin=sin, q=q.clone())
    rest = qkv[:, H:].clone()
    got = sdpa_lib.sdpa_cache_append(caches[1], k, v, table, lens, cos=cos, sin=sin, q=q, q_out=q)
    assert got is q and torch.equal(q, apart) and torch.equal(qkv[:, H:], rest)
    for name in ("k", "v"):
        assert torch.equal(getattr(caches[0], name).view(torch.uint8), getattr(caches[1], name).view(torch.uint8))
        assert torch.equal(getattr(caches[0], name + "_scale"), getattr(caches[1], name + "_scale"))


@gpu
def test_append_leaves_out_what_has_no_place(sdpa_lib):
    """Negative positions, positions past the tables, bad page entries, tokens behind the last
    sequence: nothing is written for them, queries of tokens without a position included."""
    P, D = 16, 64
    c = make_cache(sdpa_lib, 8, P, 1, D, "16", torch.float16, 4)
    table = torch.tensor([[0, 1], [2, 99], [3, 4], [5, -3]], dtype=torch.int32)
    counts, lens = [5, 4, 6, 3], [3, 18, 34, 20]   # 2 tokens negative; bad page; 2 past the table; bad page
    total = sum(counts) + 2
    g = torch.Generator().manual_seed(1)
    k, v, q = (torch.randn(total, 1, D, generator=g).half().cuda() for _ in range(3))
    a = torch.rand(31, D // 2, generator=g)        # position 31 is past the angles
    cos, sin = a.cos().cuda(), a.sin().cuda()
    ck, cv, was = ref.values(c.k), ref.values(c.v), c.k.clone()
    written, _ = ref.append(ck, cv, None, None, k, v, table, lens, counts, cos, sin)
    q_out = torch.full_like(q, 9.0)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    sdpa_lib.sdpa_cache_append(c, k, v, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), cu,
                               cos=cos, sin=sin, q=q, q_out=q_out)
    mask = torch.zeros(8, P, dtype=torch.bool)
    for p, r in written:
        mask[p, r] = True
    check(ref.values(c.k)[mask], ck[mask], (2.0 ** -11 * ck.abs() + 2.0 ** -19)[mask], "k")
    assert torch.equal(c.k.cpu()[~mask], was.cpu()[~mask])
    untouched = [0, 1, 9 + 3, 9 + 4, 9 + 5, 18, 19]
    for t in range(total):
        assert bool((q_out[t] == 9).all()) == (t in untouched), t


@gpu
def test_append_infinities_and_nan(sdpa_lib):
    """They do not make the scale; infinities become +-448 codes, NaN stays NaN."""
    c = make_cache(sdpa_lib, 2, 16, 1, 64, "e4m3", torch.bfloat16, 4)
    x = torch.ones(3, 1, 64)
    x[0, 0, 0], x[1, 0, 1], x[2, 0, 2] = math.inf, -math.inf, math.nan
    x = x.bfloat16().cuda()
    sdpa_lib.sdpa_cache_append(c, x, x, torch.tensor([[1]], dtype=torch.int32).cuda(), torch.tensor([3], dtype=torch.int32).cuda())
    for t, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
        assert s[1, 0].item() == 2.0 ** -8
        got = t[1, :3, 0].float().cpu()
        assert got[0, 0] == 448 and got[1, 1] == -448 and math.isnan(got[2, 2])
        got[0, 0] = got[1, 1] = got[2, 2] = 256
        assert (got == 256).all()
    z = torch.zeros(1, 1, 64).bfloat16().cuda()
    sdpa_lib.sdpa_cache_append(c, z, z, torch.tensor([[0]], dtype=torch.int32).cuda(), torch.tensor([1], dtype=torch.int32).cuda())
    assert c.k_scale[0, 0].item() == 2.0 ** -50 and (c.k[0, 0].float() == 0).all()


@gpu
@pytest.mark.parametrize("cache", ["e4m3", "16"])
def test_decoding_loop(sdpa_lib, cache):
    """Prompts appended and attended to in uneven chunks, then single tokens, captured as one graph
    and replayed: every step against 64-bit attention over the values that the cache holds."""
    B, H, hkv, D, P, steps = 3, 8, 2, 128, 16, 6
    g = torch.Generator().manual_seed(5)
    dtype = torch.bfloat16
    mp = 8
    c = make_cache(sdpa_lib, B * mp + 1, P, hkv, D, cache, dtype, 2)
    table = tables(B, mp, B * mp + 1, 2)
    a = torch.arange(mp * P)[:, None] * torch.exp2(-torch.arange(D // 2) / 8.0)
    cos, sin = a.cos().cuda(), a.sin().cuda()
    counts = [41, 16, 7]
    kv_lens = torch.tensor(counts, dtype=torch.int32, device="cuda")
    tab = table.cuda()

    def check_step(q, out, counts, lens):
        want = ref.attend(q, ref.values(c.k, c.k_scale), ref.values(c.v, c.v_scale), table, lens, counts, None, True)
        weight = dtype if cache == "16" else torch.float16
        tol, _ = ref.attend_bounds(want, max(lens), D, dtype, weight)
        check(out, want[0], tol, "out")

    total = sum(counts)
    q, k, v = (torch.randn(total, n, D, generator=g).to(dtype).cuda() for n in (H, hkv, hkv))
    cu = torch.tensor([0, 41, 57, 64], dtype=torch.int32, device="cuda")
    qr = sdpa_lib.sdpa_cache_append(c, k, v, tab, kv_lens, cu, cos=cos, sin=sin, q=q)
    out = sdpa_lib.sdpa_paged_forward(qr, c, tab, kv_lens, cu, 41, is_causal=True)
    check_step(qr, out, counts, counts)

    q, k, v = (torch.randn(B, n, D, generator=g).to(dtype).cuda() for n in (H, hkv, hkv))
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    kv_lens += 1
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        qr = sdpa_lib.sdpa_cache_append(c, k, v, tab, kv_lens, cos=cos, sin=sin, q=q)
        sdpa_lib.sdpa_paged_forward(qr, c, tab, kv_lens, is_causal=True)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        qr = sdpa_lib.sdpa_cache_append(c, k, v, tab, kv_lens, cos=cos, sin=sin, q=q)
        out = sdpa_lib.sdpa_paged_forward(qr, c, tab, kv_lens, is_causal=True)
        kv_lens += 1
    lens = [n + 1 for n in counts]
    for _ in range(steps):
        for t, n in ((q, H), (k, hkv), (v, hkv)):
            t.copy_(torch.randn(B, n, D, generator=g).to(dtype))
        graph.replay()
        torch.cuda.synchronize()
        check_step(qr, out, [1] * B, lens)
        lens = [n + 1 for n in lens]


@gpu
def test_two_streams_at_once(sdpa_lib):
    """Calls on two streams at the same time do not share anything."""
    c = make_cache(sdpa_lib, 130, 64, 2, 128, "e4m3", torch.bfloat16, 2)
    table = tables(2, 64, 130, 2).cuda()
    lens = torch.tensor([4000, 4096], dtype=torch.int32, device="cuda")
    q = [torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(i)).bfloat16().cuda() for i in range(2)]
    want = [sdpa_lib.sdpa_paged_forward(x, c, table, lens) for x in q]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(sdpa_lib.sdpa_paged_forward(q[i], c, table, lens, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for x in got[i]:
            assert torch.equal(x, want[i])


@gpu
@pytest.mark.parametrize("size", [1e-30, 1e30])
@pytest.mark.parametrize("rows", [12, 40, 100])
def test_small_and_large_queries_of_many_rows(sdpa_lib, size, rows):
    """The tensor-core form splits a query row into 8-bit terms under a power of two of its own.
    (Elements below 2^-9 of the row's largest are off by up to 2^-17 of it: four of them by 2^-17 * 4
    * 4 against a key of 4 each change a score by 5e-5, inside (D + 16) 2^-24 sum |q| |k| = 7e-5.)"""
    c = make_cache(sdpa_lib, 16, 16, 1, 128, "e4m3", torch.bfloat16, 14)
    q = (torch.randn(2 * rows, 3, 128, generator=torch.Generator().manual_seed(4)) * size).bfloat16().cuda()
    run_attend(sdpa_lib, c, q, tables(2, 8, 16, 1), [110, 128], [rows] * 2, True, scale=0.1 / size)


@gpu
@pytest.mark.parametrize("scale", [0.0, 1e-42, -0.3])
@pytest.mark.parametrize("cache", ["e4m3", "16"])
@pytest.mark.parametrize("rows", [12, 100])
def test_scales_of_the_scores_of_many_rows(sdpa_lib, cache, scale, rows):
    c = make_cache(sdpa_lib, 20, 32, 2, 64, cache, torch.float16, 8, spread=0.5)
    q = torch.randn(2 * rows, 6, 64, generator=torch.Generator().manual_seed(2)).half().cuda()
    run_attend(sdpa_lib, c, q, tables(2, 6, 20, 2), [150, rows - 3], [rows] * 2, True, scale=scale)


@gpu
@pytest.mark.parametrize("where", [3, 129, 256, 299])
@pytest.mark.parametrize("cache", ["e4m3", "16"])
@pytest.mark.parametrize("rows", [1, 12, 100])
def test_nan_inside_the_length(sdpa_lib, cache, rows, where):
    """A NaN that the rows see reaches them: in a value one column of its head, in a key the rows
    of its head; and nothing else."""
    P, D, lens = 16, 128, [300, 290]
    c = make_cache(sdpa_lib, 40, P, 2, D, cache, torch.bfloat16, 6)
    table = tables(2, 19, 40, 11)
    q = torch.randn(2 * rows, 8, D, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    for t, head in ((c.v, 1), (c.k, 0)):
        page, row = int(table[0, where // P]), where % P
        x = t[page, row, head].float()
        x[70] = math.nan
        t[page, row, head].copy_(x.to(t.dtype))
    cu = torch.tensor([0, rows, 2 * rows], dtype=torch.int32, device="cuda")
    out, lse = sdpa_lib.sdpa_paged_forward(q, c, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), cu, rows,
                                           return_lse=True)
    want = ref.attend(q, ref.values(c.k, c.k_scale), ref.values(c.v, c.v_scale), table, lens, [rows] * 2)
    nan = torch.zeros(2 * rows, 8, D, dtype=torch.bool)
    nan[:rows, 4:, 70] = True
    nan[:rows, :4] = True
    assert torch.equal(torch.isnan(out.cpu()), nan) and torch.equal(torch.isnan(want[0]), nan)
    assert torch.equal(torch.isnan(lse.cpu()), nan[..., 0])
    tol, _ = ref.attend_bounds(want, 300, D, torch.bfloat16, torch.bfloat16 if cache == "16" else torch.float16)
    check(out.cpu()[~nan], want[0][~nan], tol[~nan], "out")


@gpu
@pytest.mark.parametrize("cache", ["e4m3", "16"])
@pytest.mark.parametrize("rows", [6, 80])
def test_captured_many_rows(sdpa_lib, cache, rows):
    """The tensor-core form captured once and replayed with other lengths, tables and queries, an
    append before it."""
    B, H, hkv, D, P, mp = 2, 8, 2, 64, 32, 12
    g = torch.Generator().manual_seed(rows)
    c = make_cache(sdpa_lib, B * mp, P, hkv, D, cache, torch.float16, 4)
    q, k, v = (torch.randn(B * rows, n, D, generator=g).half().cuda() for n in (H, hkv, hkv))
    tab, lens = tables(B, mp, B * mp, 1).cuda(), torch.tensor([rows, 200], dtype=torch.int32, device="cuda")
    sdpa_lib.sdpa_cache_append(c, k, v, tab, lens)
    sdpa_lib.sdpa_paged_forward(q, c, tab, lens, is_causal=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sdpa_lib.sdpa_cache_append(c, k, v, tab, lens)
        out, lse = sdpa_lib.sdpa_paged_forward(q, c, tab, lens, is_causal=True, return_lse=True)
    for seed, n in ((2, [rows, 384]), (3, [331, rows + 1])):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        tab.copy_(tables(B, mp, B * mp, seed))
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g).half())
        graph.replay()
        torch.cuda.synchronize()
        eager = sdpa_lib.sdpa_paged_forward(q, c, tab, lens, is_causal=True, return_lse=True)
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])
        run_attend(sdpa_lib, c, q, tab.cpu(), n, [rows] * B, True, use_cu=False)


@gpu
def test_calls_on_another_stream(sdpa_lib):
    """stream= of both calls, with the work before them still running on it."""
    c = make_cache(sdpa_lib, 24, 32, 2, 128, "e4m3", torch.bfloat16, 4)
    d = sdpa_lib.SdpaPagedCache(c.k.clone(), c.v.clone(), c.k_scale.clone(), c.v_scale.clone())
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(50, n, 128, generator=g).bfloat16().cuda() for n in (8, 2, 2))
    tab, lens = tables(1, 20, 24, 1).cuda(), torch.tensor([600], dtype=torch.int32, device="cuda")
    a = (torch.arange(640)[:, None] * torch.exp2(-torch.arange(64) / 8.0))
    cos, sin = a.cos().cuda(), a.sin().cuda()
    qr = sdpa_lib.sdpa_cache_append(c, k, v, tab, lens, cos=cos, sin=sin, q=q)
    want = sdpa_lib.sdpa_paged_forward(qr, c, tab, lens, is_causal=True)
    late = [torch.zeros_like(x) for x in (q, k, v)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        busy = torch.randn(4096, 4096, device="cuda")
        for _ in range(10):
            busy = busy @ busy * 1e-2
        for x, y in zip(late, (q, k, v)):
            x.copy_(y)
    qr2 = sdpa_lib.sdpa_cache_append(d, late[1], late[2], tab, lens, cos=cos, sin=sin, q=late[0], stream=s)
    got = sdpa_lib.sdpa_paged_forward(qr2, d, tab, lens, is_causal=True, stream=s)
    s.synchronize()
    assert torch.equal(qr, qr2) and torch.equal(want, got) and torch.equal(c.k_scale, d.k_scale)
    assert torch.equal(c.k.view(torch.uint8), d.k.view(torch.uint8)) and torch.equal(c.v.view(torch.uint8), d.v.view(torch.uint8))


@gpu
@pytest.mark.parametrize("cache", ["e4m3", "16"])
@pytest.mark.parametrize("rows", [1, 7, 900])
def test_one_page_of_1024(sdpa_lib, cache, rows):
    """The largest pages, a cache of one page, appended to from its first row and attended to."""
    c = make_cache(sdpa_lib, 1, 1024, 1, 64, cache, torch.bfloat16, 4)
    g = torch.Generator().manual_seed(rows)
    table = torch.zeros(1, 1, dtype=torch.int32)
    n = 1024 - rows
    for count, length in ((n, n), (rows, 1024)):
        k, v = (torch.randn(count, 1, 64, generator=g).bfloat16().cuda() for _ in range(2))
        sdpa_lib.sdpa_cache_append(c, k, v, table.cuda(), torch.tensor([length], dtype=torch.int32, device="cuda"))
        x = ref.values(c.v, c.v_scale)[0, length - count:length]
        w = v.cpu().double()
        if cache == "16":
            assert torch.equal(x, w)
        else:   # one rounding: half a step, or half of the least subnormal 2^-9 under the page's scale
            check(x, w, ref.half_step(E4M3) * w.abs() + c.v_scale.item() * 2.0 ** -10, "v")
    q = torch.randn(rows, 4, 64, generator=g).bfloat16().cuda()
    run_attend(sdpa_lib, c, q, table, [1024], [rows], True, use_cu=False)


@gpu
@pytest.mark.parametrize("rot", [0, 64])
def test_scale_grows_token_by_token(sdpa_lib, rot):
    """Tokens that grow, one call each: codes and scales as the same steps give in plain tensors,
    bit for bit (values and ratios are such that each step is one rounding)."""
    c = make_cache(sdpa_lib, 3, 16, 2, 64, "e4m3", torch.bfloat16, 4)
    g = torch.Generator().manual_seed(9)
    codes, scale = torch.zeros(16, 2, 64, dtype=E4M3), None
    table = torch.tensor([[2]], dtype=torch.int32, device="cuda")
    cos, sin = (torch.ones(16, 32, device="cuda"), torch.zeros(16, 32, device="cuda")) if rot else (None, None)
    for i in range(16):
        x = (torch.randn(1, 2, 64, generator=g) * 2.0 ** (1.5 * i - 20 if i % 5 else -20)).bfloat16()
        sdpa_lib.sdpa_cache_append(c, x.cuda(), x.cuda(), table, torch.tensor([i + 1], dtype=torch.int32, device="cuda"),
                                   cos=cos, sin=sin)
        need = torch.tensor([ref.scale_for(float(x[0, h].float().abs().max())) for h in range(2)])
        new = need if i == 0 else torch.maximum(need, scale)
        if i:
            codes[:i] = (codes[:i].float() * (scale / new)[:, None]).to(E4M3)
        scale = new
        codes[i] = (x[0].float() / scale[:, None]).to(E4M3)
        for t, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
            assert torch.equal(s[2].cpu(), scale), i
            assert torch.equal(t[2, :i + 1].cpu().float(), codes[:i + 1].float()), i


@gpu
def test_append_beyond_the_tables(sdpa_lib):
    """Lengths past the page table and past the angles: tokens that have a place are written, the
    others are left out, and so are their queries."""
    for cache in ("e4m3", "16"):
        for n_pos, last in ((100, 32), (20, 20)):
            c = make_cache(sdpa_lib, 6, 16, 1, 64, cache, torch.bfloat16, 4)
            k, v, q = (torch.randn(40, n, 64, generator=torch.Generator().manual_seed(n_pos)).bfloat16().cuda() for n in (1, 1, 3))
            table = torch.tensor([[4, 1]], dtype=torch.int32, device="cuda")
            was = [t.clone().view(torch.uint8) for t in (c.k, c.v)]
            out = torch.full_like(q, 7.0)
            one, zero = torch.ones(n_pos, 32, device="cuda"), torch.zeros(n_pos, 32, device="cuda")
            # 40 tokens at positions 5 .. 44
            sdpa_lib.sdpa_cache_append(c, k, v, table, torch.tensor([45], dtype=torch.int32, device="cuda"), cos=one, sin=zero,
                                       q=q, q_out=out)
            kept = last - 5
            assert torch.equal(out[:kept], q[:kept]) and (out[kept:] == 7).all()
            for t, w, x in ((c.k, was[0], k), (c.v, was[1], v)):
                s = None if cache == "16" else (c.k_scale if t is c.k else c.v_scale)
                got = ref.values(t, s)[[4, 1]].reshape(32, 64)[5:last]
                want = x[:kept, 0].cpu().double()
                if cache == "16":
                    assert torch.equal(got, want)
                    assert torch.equal(t.view(torch.uint8)[4, :5], w[4, :5])
                else:
                    # one rounding: half a step, or half of the least subnormal 2^-9 under the pages' scales
                    check(got, want, ref.half_step(E4M3) * want.abs() + s[[4, 1]].max().item() * 2.0 ** -10, "codes")
                rest = torch.tensor([0, 2, 3, 5], device="cuda")
                assert torch.equal(t.view(torch.uint8)[rest], w[rest])
                if last == 20:
                    assert torch.equal(t.view(torch.uint8)[1, 4:], w[1, 4:])


@gpu
@pytest.mark.parametrize("rows", [1, 12, 100])
@pytest.mark.parametrize("shift,width", [(8, 152), (16, 152), (16, 160), (0, 128)])
def test_rows_of_out_on_any_16_bytes(sdpa_lib, rows, shift, width):
    """Output rows that begin on 16-byte boundaries and not on 32-byte ones, and on both."""
    c = make_cache(sdpa_lib, 16, 32, 2, 128, "16", torch.bfloat16, 4)
    q = torch.randn(rows, 6, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    wide = torch.full((rows * 6 * width + 64,), 9.0, dtype=torch.bfloat16, device="cuda")
    out = wide[shift:shift + rows * 6 * width].view(rows, 6, width)[..., :128]
    run_attend(sdpa_lib, c, q, tables(1, 10, 16, 1), [300], [rows], True, use_cu=False, out=out)
    untouched = torch.ones_like(wide, dtype=torch.bool)
    untouched[shift:shift + rows * 6 * width].view(rows, 6, width)[..., :128] = False
    assert (wide[untouched] == 9).all()
