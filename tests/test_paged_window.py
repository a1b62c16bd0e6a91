"""Attention over pages with a sliding window and first tokens that stay visible: against a plain 64-bit form, over
pages that are gone behind the window, and beside the forward without a window."""
import math

import numpy as np
import pytest
import torch

import scaled_dot_product_forward_gb300 as sdpa
from tests import paged_ref as ref
from tests.test_paged import check, make_cache, tables

gpu = pytest.mark.gpu


def attend(q, k, v, table, lens, counts, window, sinks, scale=None):
    """As paged_ref.attend, row by row, for the keys that a row sees."""
    q = q.cpu().double()
    total, H, D = q.shape
    P, hkv = k.shape[1], k.shape[2]
    G, sc = H // hkv, (1.0 / math.sqrt(D) if scale is None else scale)
    out, spread, top = (torch.zeros(total, H, D, dtype=torch.float64) for _ in range(3))
    lse, reach = torch.full((total, H), -math.inf, dtype=torch.float64), torch.zeros(total, H, dtype=torch.float64)
    row = 0
    for b, n in enumerate(counts):
        length = min(max(int(lens[b]), 0), table.shape[1] * P)
        for i in range(n):
            pos = length - n + i
            keys = [j for j in range(pos + 1) if j > pos - window or j < sinks]
            keys = [(int(table[b, j // P]), j % P) for j in keys]
            keys = [(p, r) for p, r in keys if 0 <= p < k.shape[0]]
            if keys:
                pages, rows = torch.tensor([x[0] for x in keys]), torch.tensor([x[1] for x in keys])
                kk, vv = k[pages, rows], v[pages, rows]                     # [keys, hkv, D]
                qq = q[row].view(hkv, G, D)
                s = sc * torch.einsum("khd,hgd->hgk", kk, qq)
                m = s.amax(-1, keepdim=True)
                e = torch.exp(s - m)
                lse[row] = (m[..., 0] + torch.log(e.sum(-1))).view(H)
                p = e / e.sum(-1, keepdim=True)
                out[row] = torch.einsum("hgk,khd->hgd", p, vv).reshape(H, D)
                spread[row] = torch.einsum("hgk,khd->hgd", p, vv.abs()).reshape(H, D)
                reach[row] = abs(sc) * torch.einsum("khd,hgd->hgk", kk.abs(), qq.abs()).amax(-1).view(H)
                top[row] = vv.abs().amax(0)[:, None].expand(hkv, G, D).reshape(H, D)
            row += 1
    return out, lse, spread, reach, top


def call(lib, cache, q, table, lens, counts, window, sinks, **kw):
    cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    return lib.sdpa_paged_forward(q, cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), cu,
                                  max(counts), is_causal=True, window=window, sinks=sinks, return_lse=True, **kw)


def run(lib, cache, q, table, lens, counts, window, sinks, seen_table=None, **kw):
    """seen_table: the table as the plain form reads it (the call's may have lost entries that no row sees)."""
    out, lse = call(lib, cache, q, table, lens, counts, window, sinks, **kw)
    k, v = ref.values(cache.k, cache.k_scale), ref.values(cache.v, cache.v_scale)
    want = attend(q, k, v, table if seen_table is None else seen_table, lens, counts, window, sinks, kw.get("scale"))
    weight = torch.bfloat16 if cache.k.dtype == torch.bfloat16 else torch.float16
    tol, lse_tol = ref.attend_bounds(want, max(1, max(lens)), q.shape[2], q.dtype, weight)
    check(out, want[0], tol, "out")
    empty = torch.isinf(want[1])
    assert torch.equal(torch.isinf(lse.cpu()), empty)
    assert torch.all(out.cpu()[empty] == 0)
    if not empty.all():
        check(lse.cpu()[~empty], want[1][~empty], lse_tol[~empty], "lse")
    assert lib.sdpa_last_device_status()[0] == 0
    return out, lse


def gone(table, lens, counts, window, sinks, P, what):
    """The table without the entries that no row of a sequence sees (and those behind its end)."""
    t = table.clone()
    for b, (n, L) in enumerate(zip(counts, lens)):
        lo = max(0, L - n + 1 - window) if n else L
        t[b, -(-sinks // P):lo // P] = what
    return t


CASES = [  # D, cache, dtype, page, kv heads, G, memory order, counts, lengths, window, sinks
    (128, "e4m3", torch.bfloat16, 16, 4, 4, "tokens", [1, 1, 1, 1, 1], [1, 0, 17, 333, 1200], 100, 4),
    (128, "e4m3", torch.float16, 64, 1, 16, "heads", [1, 1, 1], [63, 640, 900], 65, 1),
    (128, "16", torch.bfloat16, 32, 2, 8, "tokens", [2, 1, 2], [100, 5, 700], 33, 0),
    (128, "16", torch.float16, 16, 3, 1, "padded", [1, 7, 16], [530, 7, 9], 1, 0),
    (64, "e4m3", torch.bfloat16, 128, 2, 7, "heads", [1, 3, 2], [800, 3, 500], 130, 129),
    (64, "e4m3", torch.float16, 16, 4, 1, "padded", [1, 1], [1000, 31], 16, 16),
    (64, "16", torch.bfloat16, 64, 1, 3, "heads", [5, 2], [729, 64], 1, 3),
    (64, "16", torch.float16, 32, 2, 16, "tokens", [1, 1, 1], [700, 33, 2], 500, 300),
    # 17 to 64 rows a head
    (128, "e4m3", torch.bfloat16, 32, 1, 5, "tokens", [10, 1, 9], [990, 300, 9], 128, 4),
    (128, "16", torch.float16, 16, 2, 8, "heads", [7, 8, 1], [900, 8, 513], 77, 17),
    (64, "e4m3", torch.float16, 16, 1, 64, "tokens", [1, 1], [1290, 200], 300, 0),
    (64, "16", torch.bfloat16, 64, 2, 4, "padded", [16, 3], [777, 500], 1, 1),
    # more
    (128, "e4m3", torch.bfloat16, 64, 2, 8, "tokens", [33, 70, 1], [33, 760, 550], 100, 4),
    (128, "e4m3", torch.float16, 16, 1, 16, "heads", [40, 9], [1500, 700], 200, 130),
    (128, "16", torch.bfloat16, 16, 1, 8, "heads", [130, 3], [900, 629], 64, 1),
    (64, "16", torch.float16, 128, 1, 4, "tokens", [177, 5], [900, 64], 256, 0),
    (64, "e4m3", torch.bfloat16, 32, 2, 4, "tokens", [300, 1, 20], [300, 900, 20], 1, 0),
    (64, "e4m3", torch.float16, 1024, 1, 8, "tokens", [60, 61], [1800, 100], 129, 5),
    (128, "16", torch.bfloat16, 256, 2, 3, "padded", [100, 90], [70, 1000], 300, 600),
]


@gpu
@pytest.mark.parametrize("lost", ["kept", "gone", "junk"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"D{c[0]}-{c[1]}-{str(c[2])[6:]}-P{c[3]}-{c[4]}x{c[5]}-{c[6]}-{c[7]}-w{c[9]}-s{c[10]}")
def test_window(sdpa_lib, case, lost):
    """All pages there; entries behind the window gone (none, out of range); or pages there that hold NaN."""
    D, cache, dtype, P, hkv, G, kind, counts, lens, window, sinks = case
    seed = D + P + hkv * 10 + G
    mp = -(-max(lens) // P) + 1
    n_pages = len(lens) * mp + 2
    c = make_cache(sdpa_lib, n_pages, P, hkv, D, cache, dtype, seed, kind)
    q = torch.randn(sum(counts), hkv * G, D, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()
    t = tables(len(lens), mp, n_pages, seed)
    used = t
    if lost == "gone":
        used = gone(t, lens, counts, window, sinks, P, -1 if seed % 2 else n_pages + 7)
    elif lost == "junk":
        bad = int(set(range(n_pages)).difference(t.flatten().tolist()).pop())
        for x in (c.k, c.v):
            if cache == "e4m3":
                x[bad] = torch.full_like(x[bad].float(), math.nan).to(x.dtype)
            else:
                x[bad] = math.nan
        used = gone(t, lens, counts, window, sinks, P, bad)
    run(sdpa_lib, c, q, used, lens, counts, window, sinks, seen_table=t)


@gpu
@pytest.mark.parametrize("cache", ["e4m3", "16"])
@pytest.mark.parametrize("rows", [1, 3, 40])
def test_many_ctas_a_sequence(sdpa_lib, cache, rows):
    """A long window of one sequence, cut between all CTAs and joined; any bound on the rows gives the results, and
    a call gives them again bit for bit."""
    lens, P = [9001], 64
    c = make_cache(sdpa_lib, 142, P, 1, 128, cache, torch.bfloat16, 7)
    q = torch.randn(rows, 4, 128, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    t = tables(1, 141, 142, 3)
    a = run(sdpa_lib, c, q, t, lens, [rows], 5000, 70)
    b = call(sdpa_lib, c, q, t, lens, [rows], 5000, 70)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    cu = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    want = attend(q, ref.values(c.k, c.k_scale), ref.values(c.v, c.v_scale), t, lens, [rows], 5000, 70)
    tol, _ = ref.attend_bounds(want, 9001, 128, q.dtype, torch.bfloat16 if cache == "16" else torch.float16)
    for bound in (1, 5000):
        got = sdpa_lib.sdpa_paged_forward(q, c, t.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), cu, bound,
                                          is_causal=True, window=5000, sinks=70)
        check(got, want[0], tol, f"bound {bound}")


@gpu
@pytest.mark.parametrize("cache", ["e4m3", "16"])
@pytest.mark.parametrize("D,counts", [(128, [1, 1, 1]), (64, [9, 2, 5]), (128, [200, 1, 77])])
def test_a_window_over_everything(sdpa_lib, cache, D, counts):
    """A window of all that the tables hold gives the causal results bit for bit, one of all that the sequences hold
    the same keys; so do sinks that reach as far as the sequences."""
    lens, P = [700, 1, 300], 32
    c = make_cache(sdpa_lib, 70, P, 2, D, cache, torch.float16, 5)
    q = torch.randn(sum(counts), 8, D, generator=torch.Generator().manual_seed(3)).half().cuda()
    t = tables(3, 23, 70, 3)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    want = sdpa_lib.sdpa_paged_forward(q, c, t.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), cu, max(counts),
                                       is_causal=True, return_lse=True)
    for window, sinks in ((23 * P, 0), (1 << 62, 1 << 70), (700, 0), (1, 700), (1, 1 << 62), (23 * P - 1, 9)):
        got = call(sdpa_lib, c, q, t, lens, counts, window, sinks)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (window, sinks)


@gpu
def test_captured_and_on_a_side_stream(sdpa_lib):
    """A captured call follows the lengths on the device; a call on another stream gives the same."""
    lens, P = [900, 40], 16
    c = make_cache(sdpa_lib, 130, P, 2, 64, "e4m3", torch.bfloat16, 5)
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    t, dev_lens = tables(2, 60, 130, 3).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    kw = dict(is_causal=True, window=50, sinks=3)
    first = sdpa_lib.sdpa_paged_forward(q, c, t, dev_lens, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = sdpa_lib.sdpa_paged_forward(q, c, t, dev_lens, stream=side, **kw)
    side.synchronize()
    assert torch.equal(first, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sdpa_lib.sdpa_paged_forward(q, c, t, dev_lens, **kw)
    for new in ([900, 40], [901, 41], [300, 960], [1, 0]):
        dev_lens.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        assert torch.equal(out, sdpa_lib.sdpa_paged_forward(q, c, t, dev_lens, **kw)), new


def test_refusals():
    from tests.test_paged_refusals import ARG, cache, status
    c = cache()
    q, t, lens = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 3, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    f = sdpa.sdpa_paged_forward
    for kw in (dict(window=0, is_causal=True), dict(window=-3, is_causal=True), dict(window=5, is_causal=False), dict(window=5),
               dict(window=5, sinks=-1, is_causal=True), dict(sinks=3, is_causal=True), dict(sinks=-1)):
        assert status(f, q, c, t, lens, **kw) == ARG, kw
    # the C entry
    lib = sdpa.load_library()
    assert lib.sdpa_paged_forward_window(*[None] * 3, 0, None, 1, 1, None, None, None, None, 1, 1, None, None, 1, 1, 0, 0, 1.0,
                                         None, 0, None) == ARG
    assert lib.sdpa_paged_forward_window(*[None] * 3, 0, None, 1, 1, None, None, None, None, 1, 1, None, None, 1, 1, 5, -1, 1.0,
                                         None, 0, None) == ARG
    assert lib.sdpa_paged_forward_window(*[None] * 3, 0, None, 1, 1, None, None, None, None, 1, 1, None, None, 1, 1, 5, 0, 1.0,
                                         None, 0, None) == 1
