"""Pages of a cache as a whole: taking, forking and releasing them, copying and compacting them, against plain forms; and
a small model's serving loop that uses them with the append, its norms and the windowed attention."""
import math

import pytest
import torch

import scaled_dot_product_forward_gb300 as sdpa
from tests import paged_ref as ref
from tests.test_paged import make_cache, tables

E4M3 = torch.float8_e4m3fn
gpu = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Accounts:
    """The accounts as lists."""

    def __init__(self, refs, table, P):
        self.refs, self.table, self.P = refs, table, P

    def is_page(self, p):
        return 0 <= p < len(self.refs)

    def free(self):
        return iter([p for p, n in enumerate(self.refs) if n <= 0])

    def limit(self, n, table=None):
        return min(max(n, 0), len((table or self.table)[0]) * self.P)

    def take(self, lo, hi):
        free, missing = self.free(), 0
        for r, row in enumerate(self.table):
            for e in range(-(-self.limit(lo[r]) // self.P), -(-self.limit(hi[r]) // self.P)):
                row[e] = next(free, -1)
                missing += row[e] < 0
                if row[e] >= 0:
                    self.refs[row[e]] = 1
        return missing

    def fork(self, lens, src, dst, new=None):
        out = self.table if new is None else new
        ok = [0 <= s < len(self.table) and 0 <= d < len(out) and not (new is None and s == d) for s, d in zip(src, dst)]
        source = [list(r) for r in self.table]
        for s, d, good in zip(src, dst, ok):
            if not good:
                continue
            full = self.limit(lens[s]) // self.P
            row = [p if e < full and self.is_page(p) else -1 for e, p in enumerate(source[s])]
            for p in out[d]:
                if self.is_page(p):
                    self.refs[p] -= 1
            for p in row:
                if p >= 0:
                    self.refs[p] += 1
            out[d][:] = row
        free, copies, missing = self.free(), [], 0
        for s, d, good in zip(src, dst, ok):
            copies.append((-1, -1, 0))
            if not good:
                continue
            full, begun = divmod(self.limit(lens[s]), self.P)
            if begun and self.is_page(source[s][full]):
                p = next(free, -1)
                missing += p < 0
                if p >= 0:
                    self.refs[p] = 1
                    copies[-1] = (source[s][full], p, begun)
                    out[d][full] = p
        return copies, missing

    def release(self, lo, hi, rows):
        n = len(self.table) if rows is None else len(rows)
        for i in range(n):
            r = i if rows is None else rows[i]
            if not 0 <= r < len(self.table):
                continue
            row = self.table[r]
            for e in range(-(-max(lo[i] if lo else 0, 0) // self.P), min(len(row), max(hi[i], 0) // self.P) if hi else len(row)):
                if self.is_page(row[e]):
                    self.refs[row[e]] -= 1
                row[e] = -1


def state(n_pages, rows, columns, P, seed, held=0.3, room=0):
    """refs and a table with some entries shared, some gone, in agreement; columns are a part of a wider buffer."""
    g = torch.Generator().manual_seed(seed)
    table = torch.full((rows, columns), -1, dtype=torch.int32)
    refs = (torch.rand(n_pages, generator=g) < held).int()
    if room:   # free pages at the end only
        refs[:n_pages - room] = 1
    pick = torch.rand(rows, columns, generator=g) < 0.6
    table[pick] = torch.randint(0, n_pages, (int(pick.sum()),), generator=g, dtype=torch.int32)
    refs.index_add_(0, table[table >= 0].long(), torch.ones(int((table >= 0).sum()), dtype=torch.int32))
    wide = torch.full((rows, columns + 3), -7, dtype=torch.int32, device="cuda")
    wide[:, 1:1 + columns] = table.cuda()
    return refs.cuda(), wide[:, 1:1 + columns], wide, Accounts(refs.tolist(), table.tolist(), P), g


def agree(refs, table, wide, want):
    assert refs.tolist() == want.refs
    assert table.tolist() == want.table
    assert torch.all(wide[:, 0] == -7) and torch.all(wide[:, -2:] == -7)


SIZES = [  # pages, rows, columns, page size, free pages at the end (0: everywhere)
    (1, 1, 1, 16, 0),
    (5, 3, 2, 64, 0),
    (17, 4, 7, 16, 0),
    (1000, 33, 12, 128, 0),
    (4099, 1500, 3, 32, 0),
    (131072, 40, 50, 16, 100),
    (131073, 7, 1300, 16, 0),
    (300001, 20, 9, 1024, 50),
    (20000, 32768, 1, 16, 0),
]


@gpu
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_take(sdpa_lib, size):
    n_pages, rows, columns, P, room = size
    refs, table, wide, want, g = state(n_pages, rows, columns, P, sum(size), room=room)
    most = columns * P
    for k in range(3):
        lo = torch.randint(-5, most + 5, (rows,), generator=g)
        hi = lo + torch.randint(-P, (3 * P if k else most) + 1, (rows,), generator=g)
        if k == 2:   # a row of any length, past the table
            lo[0], hi[0] = -(1 << 31), (1 << 31) - 1
        missing = sdpa_lib.sdpa_pages_take(refs, table, i32(lo.tolist()), i32(hi.tolist()), P)
        assert missing.item() == want.take(lo.tolist(), hi.tolist())
        agree(refs, table, wide, want)


@gpu
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_fork(sdpa_lib, size, apart):
    n_pages, rows, columns, P, room = size
    refs, table, wide, want, g = state(n_pages, rows, columns, P, sum(size) + 1, room=room)
    most = columns * P
    new = new_want = None
    if apart:
        _, new, new_wide, other, _ = state(n_pages, rows + 2, columns, P, sum(size) + 2)
        new_want = other.table
        for row in new_want:
            for p in row:
                if p >= 0:
                    want.refs[p] += 1
        refs.copy_(i32(want.refs))
    for k in range(3):
        perm = torch.randperm(rows, generator=g).tolist()
        lens = [int(x) for x in torch.randint(-3, most + 9, (rows,), generator=g)]
        if k == 1:
            lens = [x // P * P for x in lens]
        if apart:
            dst = torch.randperm(rows + 2, generator=g)[:max(1, rows - 1)].tolist()
            src = torch.randint(0, rows, (len(dst),), generator=g).tolist()
        else:
            dst, pool = perm[:max(1, rows // 2)], perm[rows // 2:]
            src = [pool[int(x)] for x in torch.randint(0, len(pool), (len(dst),), generator=g)]
        if k == 2:   # pairs that name no row, and a row to itself
            src[0] = -1 if rows % 2 else rows
            if len(dst) > 2:
                dst[1] = 1 << 30
                if not apart:
                    src[2] = dst[2]
        got = sdpa_lib.sdpa_pages_fork(refs, table, i32(lens), i32(src), i32(dst), P, new)
        copies, missing = want.fork(lens, src, dst, new_want)
        assert list(zip(got.src.tolist(), got.dst.tolist(), got.rows.tolist())) == copies
        assert got.missing.item() == missing
        agree(refs, table, wide, want)
        if apart:
            assert new.tolist() == new_want
            assert torch.all(new_wide[:, 0] == -7) and torch.all(new_wide[:, -2:] == -7)


@gpu
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_release(sdpa_lib, size):
    n_pages, rows, columns, P, room = size
    refs, table, wide, want, g = state(n_pages, rows, columns, P, sum(size) + 3, room=room)
    most = columns * P
    for k in range(3):
        n = rows if k < 2 else rows + 5
        lo = torch.randint(-5, most + 5, (n,), generator=g).tolist()
        hi = [x + int(y) for x, y in zip(lo, torch.randint(-P, most, (n,), generator=g))]
        # rows named twice, and some that are none
        which = torch.randint(-1, rows + 1, (n,), generator=g).tolist() if k == 2 else None
        a, b = (lo, None) if k == 1 else (lo, hi)
        sdpa_lib.sdpa_pages_release(refs, table, i32(a), i32(b) if b else None, P, i32(which) if which else None)
        want.release(a, b, which)
        agree(refs, table, wide, want)
    sdpa_lib.sdpa_pages_release(refs, table, None, None, P)
    want.release(None, None, None)
    agree(refs, table, wide, want)
    assert torch.all(table == -1)


CACHES = [  # D, cache, dtype, page, kv heads, memory order
    (128, "e4m3", torch.bfloat16, 16, 8, "tokens"),
    (128, "e4m3", torch.float16, 64, 3, "heads"),
    (128, "16", torch.bfloat16, 32, 5, "padded"),
    (64, "e4m3", torch.bfloat16, 128, 20, "tokens"),
    (64, "16", torch.float16, 256, 1, "heads"),
    (64, "16", torch.bfloat16, 16, 33, "tokens"),
    (64, "e4m3", torch.float16, 1024, 2, "padded"),
    (128, "16", torch.float16, 1024, 1, "tokens"),
]


def bits(c):
    """The cache as whole numbers (NaN codes keep theirs), and its scales."""
    kind = torch.uint8 if c.k.dtype == E4M3 else torch.int16
    return [c.k.view(kind).cpu().clone(), c.v.view(kind).cpu().clone()], [None if s is None else s.cpu().clone() for s in (c.k_scale, c.v_scale)]


def cache_of(sdpa_lib, case, n_pages, seed):
    D, kind, dtype, P, hkv, order = case
    c = make_cache(sdpa_lib, n_pages, P, hkv, D, kind, dtype, seed, order)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for x in (c.k, c.v):   # any bits at all, NaN and infinities among them
        view = x.view(torch.uint8 if kind == "e4m3" else torch.int16)
        few = torch.randint(0, 256 if kind == "e4m3" else 1 << 15, view.shape, generator=g, device="cuda").to(view.dtype)
        view[: n_pages // 2] = few[: n_pages // 2]
    return c


@gpu
@pytest.mark.parametrize("partly", [False, True])
@pytest.mark.parametrize("case", CACHES, ids=lambda c: f"D{c[0]}-{c[1]}-{str(c[2])[6:]}-P{c[3]}-{c[4]}-{c[5]}")
def test_copy(sdpa_lib, case, partly):
    P, n_pages = case[3], 23
    c = cache_of(sdpa_lib, case, n_pages, 3)
    (k, v), scales = bits(c)
    g = torch.Generator().manual_seed(4)
    perm = torch.randperm(n_pages, generator=g).tolist()
    src, dst = perm[:9] + [-1, perm[0], n_pages, perm[2], perm[22]], perm[9:18] + [perm[18], -4, perm[19], n_pages + 5, perm[22]]
    rows = torch.randint(0, P + 1, (len(src),), generator=g).tolist()
    rows[0], rows[1], rows[2] = P, 0, P + 100
    rows[3] = -3
    sdpa_lib.sdpa_cache_copy_pages(c, i32(src), i32(dst), i32(rows) if partly else None)
    for a, b, n in zip(src, dst, rows):
        n = min(max(n, 0), P) if partly else P
        if not (0 <= a < n_pages and 0 <= b < n_pages) or n == 0:
            continue
        for x in (k, v):
            x[b, :n] = x[a, :n]
        for s in scales:
            if s is not None:
                s[b] = s[a]
    got, got_scales = bits(c)
    assert torch.equal(got[0], k) and torch.equal(got[1], v)
    for a, b in zip(got_scales, scales):
        assert a is None or torch.equal(a, b)


@gpu
def test_copy_many(sdpa_lib):
    """More pages than blocks at a time; keys and values side by side in one pool."""
    pool = torch.randint(0, 1 << 15, (6000, 2, 16, 4, 64), generator=torch.Generator().manual_seed(3)).to(torch.int16).cuda().view(torch.float16)
    c = sdpa_lib.SdpaPagedCache(pool[:, 0], pool[:, 1])
    before = pool.view(torch.int16).clone()
    perm = torch.randperm(6000, generator=torch.Generator().manual_seed(4)).cuda()
    src, dst = perm[:3000].to(torch.int32), perm[3000:].to(torch.int32)
    sdpa_lib.sdpa_cache_copy_pages(c, src, dst)
    before[perm[3000:]] = before[perm[:3000]]
    assert torch.equal(pool.view(torch.int16), before)


def e4m3_value(codes):
    return codes.view(E4M3).float()


@gpu
@pytest.mark.parametrize("case", CACHES, ids=lambda c: f"D{c[0]}-{c[1]}-{str(c[2])[6:]}-P{c[3]}-{c[4]}-{c[5]}")
def test_compact(sdpa_lib, case):
    D, kind, dtype, P, hkv, _ = case
    B, old, new = 4, 3, 2
    n_pages = B * (old + new) + 1
    c = cache_of(sdpa_lib, case, n_pages, 6)      # (scales: powers of two)
    (k, v), scales = bits(c)
    perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(4)).to(torch.int32)
    table, new_table = perm[:B * old].view(B, old).clone(), perm[B * old:B * (old + new)].view(B, new).clone()
    g = torch.Generator().manual_seed(5)
    width = 2 * P + 3                               # more than the new pages hold
    kept = torch.randint(0, old * P, (B, width), generator=g).to(torch.int32)    # in any order, some twice
    kept[0] = torch.randperm(old * P, generator=g)[:width].sort().values.to(torch.int32)
    counts = [width, P + 1, 0, 1]
    kept[1, 0], kept[1, 1], kept[1, 2] = -1, old * P, -(1 << 31)     # no positions
    table[1, 1] = -1                                 # no page
    new_table[0, 1] = n_pages + 3
    expect_k, expect_v = k.clone(), v.clone()
    expect_s = [None if s is None else s.clone() for s in scales]
    for b, n in enumerate(counts):
        for e in range(new):
            page = int(new_table[b, e])
            if not 0 <= page < n_pages:
                continue
            tokens = []
            for i in range(e * P, min(n, (e + 1) * P)):
                pos = int(kept[b, i])
                if 0 <= pos < old * P and 0 <= int(table[b, pos // P]) < n_pages:
                    tokens.append((i % P, int(table[b, pos // P]), pos % P))
            if not tokens:
                continue
            at, pages, rows = (torch.tensor(x) for x in zip(*tokens))
            for x, out, s, out_s in ((k, expect_k, scales[0], expect_s[0]), (v, expect_v, scales[1], expect_s[1])):
                moved = x[pages, rows]
                if s is not None:
                    now = s[pages].amax(0)
                    out_s[page] = now
                    ratio = (s[pages] / now)[:, :, None]
                    # (exact products: one rounding)
                    moved = torch.where(ratio == 1, moved, (e4m3_value(moved) * ratio).to(E4M3).view(torch.uint8))
                out[page, at] = moved
    wide = torch.zeros(B, width + 5, dtype=torch.int32)
    wide[:, :width] = kept
    sdpa_lib.sdpa_cache_compact(c, table.cuda(), wide.cuda()[:, :width], new_table.cuda(), i32(counts))
    got, got_s = bits(c)
    for a, b in zip(got, (expect_k, expect_v)):
        if kind == "e4m3":   # (a scaled NaN has one code)
            nan = torch.isnan(e4m3_value(b))
            assert torch.equal(torch.isnan(e4m3_value(a)), nan)
            assert torch.equal(a[~nan], b[~nan])
        else:
            assert torch.equal(a, b)
    for a, b in zip(got_s, expect_s):
        assert a is None or torch.equal(a, b)
    # no lengths: all of kept's rows; two captured calls give the same
    sdpa_lib.sdpa_cache_compact(c, table.cuda(), kept.cuda(), new_table.cuda())
    first = bits(c)
    graph = torch.cuda.CUDAGraph()
    args = table.cuda(), kept.cuda(), new_table.cuda()
    with torch.cuda.graph(graph):
        sdpa_lib.sdpa_cache_compact(c, *args)
    graph.replay()
    again = bits(c)
    assert all(torch.equal(a, b) for a, b in zip(first[0], again[0]))


@gpu
def test_compact_other_scales(sdpa_lib):
    """Scales that are no powers of two, and ones out of range."""
    c = make_cache(sdpa_lib, 9, 32, 3, 64, "e4m3", torch.bfloat16, 5)
    c.k_scale[2, 1], c.k_scale[3, 1], c.v_scale[1, 0], c.v_scale[0, 2] = math.nan, 0.0, 1e30, -4.0
    s = [x.cpu().nan_to_num(0.0).clamp(2.0 ** -50, 2.0 ** 50).double() for x in (c.k_scale, c.v_scale)]
    before = [x.float().cpu().double() for x in (c.k, c.v)]
    table, new_table = i32([[0, 1, 2, 3]]), i32([[5, 7]])
    pos = torch.randperm(128, generator=torch.Generator().manual_seed(3))[:60]
    sdpa_lib.sdpa_cache_compact(c, table, pos[None].to(torch.int32).cuda(), new_table)
    for x, old, scale, now in ((c.k, before[0], s[0], c.k_scale), (c.v, before[1], s[1], c.v_scale)):
        x = x.float().cpu().double()
        for i, p in enumerate(pos.tolist()):
            page = (5, 7)[i // 32]
            best = scale[[q // 32 for q in pos.tolist()[i // 32 * 32:i // 32 * 32 + 32]]].amax(0)
            assert torch.equal(now[page].cpu().double(), best)
            want = old[p // 32, p % 32] * scale[p // 32][:, None]
            # a quotient and a product in fp32 (2^-23 together), a rounding to e4m3, half its least step
            tol = want.abs() * (2.0 ** -4 + 2.0 ** -22) + best[:, None] * 2.0 ** -10
            assert torch.all((x[page, i % 32] * best[:, None] - want).abs() <= tol)


@gpu
def test_captured_and_on_a_side_stream(sdpa_lib):
    """A captured step of the accounts goes on from where the last one left them; a side stream's gives the same."""
    def fresh():
        refs, table, wide, want, _ = state(500, 12, 8, 16, 77)
        return refs, table, want
    lens, to = [20, 16, 0, 128, 33, 5, 77, 90, 1, 2, 3, 4], [60, 17, 40, 128, 34, 5, 100, 128, 30, 2, 3, 90]
    src, dst = [0, 1, 3, 4], [8, 9, 10, 11]

    def step(refs, table, **kw):
        sdpa_lib.sdpa_pages_release(refs, table, d_to, None, 16, **kw)
        copies = sdpa_lib.sdpa_pages_fork(refs, table, d_lens, d_src, d_dst, 16, **kw)
        return copies, sdpa_lib.sdpa_pages_take(refs, table, d_lens, d_to, 16, **kw)

    d_lens, d_to, d_src, d_dst = i32(lens), i32(to), i32(src), i32(dst)
    refs, table, want = fresh()
    step(refs, table)            # (loads the kernels)
    refs, table, want = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        copies, missing = step(refs, table)
    other_refs, other_table, _ = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        graph.replay()
        want.release(to, None, None)
        expect, _ = want.fork(lens, src, dst)
        assert missing.item() == want.take(lens, to)
        assert list(zip(copies.src.tolist(), copies.dst.tolist(), copies.rows.tolist())) == expect
        assert refs.tolist() == want.refs and table.tolist() == want.table
        step(other_refs, other_table, stream=side)
        side.synchronize()
        assert torch.equal(refs, other_refs) and torch.equal(table, other_table)


@gpu
@pytest.mark.parametrize("kind", ["e4m3", "16"])
def test_serving_loop(sdpa_lib, kind):
    """Prompts, answers token by token in one captured step, forks of a sequence, pages given back behind the window,
    and at the end tokens dropped: beside a cache where every sequence keeps all its pages for itself."""
    D, H, hkv, P, window, sinks, B, columns, dtype = 64, 8, 2, 16, 40, 4, 4, 16, torch.bfloat16
    g = torch.Generator().manual_seed(11)
    n_pages = 70
    small = make_cache(sdpa_lib, n_pages, P, hkv, D, kind, dtype, 2)
    large = make_cache(sdpa_lib, B * columns, P, hkv, D, kind, dtype, 2)
    large_table = torch.arange(B * columns, dtype=torch.int32, device="cuda").view(B, columns)
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[5] = refs[0] = 1       # somebody else's
    table = torch.full((B, columns), -1, dtype=torch.int32, device="cuda")
    angle = torch.arange(columns * P, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) * 2 / D)
    cos, sin = angle.cos().float().cuda(), angle.sin().float().cuda()
    w = (1 + 0.2 * torch.randn(D, generator=g)).cuda()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    before, behind, first = torch.zeros_like(lens), torch.zeros_like(lens), torch.full_like(lens, sinks)

    def both(q, k, v, cu, most):
        outs = []
        for c, t in ((small, table), (large, large_table)):
            rq = sdpa_lib.sdpa_cache_append(c, k, v, t, lens, cu, cos=cos, sin=sin, q=q, q_norm=w, k_norm=w)
            outs.append(sdpa_lib.sdpa_paged_forward(rq, c, t, lens, cu, most, is_causal=True, window=window, sinks=sinks))
        return outs

    def tokens(n):
        return [torch.randn(n, h, D, generator=g).to(dtype).cuda() for h in (H, hkv, hkv)]

    def check_accounts():
        held = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        held[5] = held[0] = 1
        used = table[table >= 0].long()
        held.index_add_(0, used, torch.ones(used.numel(), dtype=torch.int32, device="cuda"))
        assert torch.equal(held, refs)

    # two prompts
    lens.copy_(i32([90, 21, 0, 0]))
    assert sdpa_lib.sdpa_pages_take(refs, table, before, lens, P).item() == 0
    a, b = both(*tokens(111), i32([0, 90, 111, 111, 111]), 90)
    assert torch.equal(a, b)
    # rows 2 and 3 go on as row 0 does
    for layer in (small,):
        copies = sdpa_lib.sdpa_pages_fork(refs, table, lens, i32([0, 0]), i32([2, 3]), P)
        sdpa_lib.sdpa_cache_copy_pages(layer, copies.src, copies.dst, copies.rows)
    assert copies.missing.item() == 0
    for x in (large.k, large.v):
        y = x.view(torch.uint8 if kind == "e4m3" else torch.int16).view(B, columns, P, hkv, D)
        y[2:] = y[:1].clone()
    if kind == "e4m3":
        for s in (large.k_scale, large.v_scale):
            s.view(B, columns, hkv)[2:] = s.view(B, columns, hkv)[:1].clone()
    lens[2:] = lens[0]
    check_accounts()
    # a captured step, replayed
    q, k, v = tokens(B)

    def step():
        behind.copy_(lens).add_(1 - window)
        sdpa_lib.sdpa_pages_release(refs, table, first, behind, P)
        before.copy_(lens)
        lens.add_(1)
        missing = sdpa_lib.sdpa_pages_take(refs, table, before, lens, P)
        return missing, both(q, k, v, None, None)

    saved = [x.clone() for x in (refs, table, lens)]
    step()      # (loads the kernels)
    for x, y in zip((refs, table, lens), saved):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        missing, outs = step()
    for i in range(100):
        for x, y in zip((q, k, v), tokens(B)):
            x.copy_(y)
        graph.replay()
        assert missing.item() == 0
        assert torch.equal(*outs), i
        check_accounts()
    assert lens.tolist() == [190, 121, 190, 190]
    assert int((table >= 0).sum()) < int((lens / P).ceil().sum())
    # of row 1 every other token of the window and the sinks stay, in new pages of row 3
    assert sdpa_lib.sdpa_pages_release(refs, table, None, None, P, i32([3])) is None
    length = int(lens[1])
    keep = list(range(sinks)) + list(range(length - window, length, 2))
    to = torch.zeros_like(lens)
    to[3] = len(keep)
    assert sdpa_lib.sdpa_pages_take(refs, table, torch.zeros_like(lens), to, P).item() == 0
    check_accounts()
    sdpa_lib.sdpa_cache_compact(small, table[1:2], i32([keep]), table[3:4])
    q = tokens(1)[0]
    got = sdpa_lib.sdpa_paged_forward(q, small, table[3:4], to[3:4])
    kk, vv = ref.values(large.k, large.k_scale), ref.values(large.v, large.v_scale)
    pages = torch.tensor([[columns + p // P, p % P] for p in keep])
    kk, vv = kk[pages[:, 0], pages[:, 1]][None].clone(), vv[pages[:, 0], pages[:, 1]][None].clone()
    one = torch.zeros(1, 1, dtype=torch.int64)
    # (as one page of all the kept tokens)
    want = ref.attend(q, kk, vv, one, [len(keep)], [1])
    tol, _ = ref.attend_bounds(want, len(keep), D, dtype, torch.bfloat16 if kind == "16" else torch.float16)
    if kind == "e4m3":
        # codes that moved to a larger scale may have been rounded below the least normal: half a step of 2^-9 of that scale each
        tol = tol + 2.0 ** -10 * float(small.v_scale.max()) + 2.0 ** -10 * float(small.k_scale.max()) * \
            (q.double().abs().sum(-1).cpu()[..., None] / math.sqrt(D)) * 2 * vv.abs().max()
    assert torch.all((got.double().cpu() - want[0]).abs() <= tol)


def test_refusals():
    from tests.test_paged_refusals import cache, status
    NULL, SHAPE, DTYPE, LAYOUT, ARG = 1, 3, 4, 5, 6
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)   # noqa: E731
    refs, t, n = z(10), z(4, 3), z(4)
    f = sdpa.sdpa_pages_take
    assert status(f, refs.long(), t, n, n, 16) == DTYPE
    assert status(f, refs, t.float(), n, n, 16) == DTYPE
    assert status(f, refs, t, n.long(), n, 16) == DTYPE
    assert status(f, refs[None], t, n, n, 16) == SHAPE
    assert status(f, refs, t[0], n, n, 16) == SHAPE
    assert status(f, refs, t, n[:3], n, 16) == SHAPE
    assert status(f, refs, t, n, z(4, 1), 16) == SHAPE
    assert status(f, z(20)[::2], t, n, n, 16) == LAYOUT
    assert status(f, refs, z(3, 4).t(), n, n, 16) == LAYOUT
    assert status(f, refs, t, n, z(8)[::2], 16) == LAYOUT
    assert status(f, refs, t, n, n, 16) == ARG        # host tensors never reach a kernel
    f = sdpa.sdpa_pages_fork
    assert status(f, refs, t, n.long(), n, n, 16) == DTYPE
    assert status(f, refs, t, n, n.long(), n, 16) == DTYPE
    assert status(f, refs, t, n, n, n, 16, t.long()) == DTYPE
    assert status(f, refs, t, n[:2], n, n, 16) == SHAPE
    assert status(f, refs, t, n, n[:2], n, 16) == SHAPE
    assert status(f, refs, t, n, t, n, 16) == SHAPE
    assert status(f, refs, t, n, n, n, 16, z(4, 5)) == SHAPE
    assert status(f, refs, t, n, n, n, 16, z(3, 5).t()[:, :3]) == LAYOUT
    assert status(f, refs, t, n, n, n, 16) == ARG
    f = sdpa.sdpa_pages_release
    assert status(f, refs, t, n.float(), n, 16) == DTYPE
    assert status(f, refs, t, n, n, 16, n.long()) == DTYPE
    assert status(f, refs, t, n, n, 16, n[:3]) == SHAPE
    assert status(f, refs, t, n[:3], n, 16) == SHAPE
    assert status(f, refs, t, n, n, 16, t) == SHAPE
    assert status(f, refs, t, n, n, 16) == ARG
    assert status(f, refs, t, None, None, 16) == ARG
    c = cache()
    f = sdpa.sdpa_cache_copy_pages
    assert status(f, c, n.long(), n) == DTYPE
    assert status(f, c, n, n, n.float()) == DTYPE
    assert status(f, c, n, n[:3]) == SHAPE
    assert status(f, c, t, t) == SHAPE
    assert status(f, c, z(8)[::2], n) == LAYOUT
    assert status(f, c, n, n) == ARG
    f = sdpa.sdpa_cache_compact
    assert status(f, c, t.long(), t, t) == DTYPE
    assert status(f, c, t, t.long(), t) == DTYPE
    assert status(f, c, t, t, t, n.long()) == DTYPE
    assert status(f, c, t, t[:2], t) == SHAPE
    assert status(f, c, t, t, t[:2]) == SHAPE
    assert status(f, c, t, t, t, n[:2]) == SHAPE
    assert status(f, c, t, n, t) == SHAPE
    assert status(f, c, z(3, 4).t(), t, t) == LAYOUT
    assert status(f, c, t, t, t) == ARG
    # nothing to do is a wrong shape
    for g, args in ((sdpa.sdpa_pages_take, (z(0), t, n, n, 16)), (sdpa.sdpa_pages_take, (refs, z(0, 3), z(0), z(0), 16)),
                    (sdpa.sdpa_pages_take, (refs, z(4, 0), n, n, 16)), (sdpa.sdpa_pages_fork, (refs, t, n, z(0), z(0), 16)),
                    (sdpa.sdpa_pages_release, (refs, t, None, None, 16, z(0))), (sdpa.sdpa_cache_copy_pages, (c, z(0), z(0))),
                    (f, (c, t, z(4, 0), t)), (f, (c, z(0, 3), z(0, 3), z(0, 3)))):
        assert status(g, *args) == SHAPE


def test_refusals_of_the_c_entries():
    """Addresses that are never read: everything is refused before any CUDA call."""
    import ctypes
    NULL, SHAPE, DTYPE, LAYOUT, ARG = 1, 3, 4, 5, 6
    lib = sdpa.load_library()
    M = 1 << 20
    base = 1 << 32

    def caller(f, names, **defaults):
        def call(**kw):
            d = dict(defaults, **kw)
            return f(*[d[n] for n in names.split()], None)
        return call

    take = caller(lib.sdpa_pages_take, "refs n_pages table st rows cols P lo hi missing", refs=base, n_pages=100, table=base + M, st=8,
                  rows=4, cols=8, P=16, lo=base + 2 * M, hi=base + 3 * M, missing=base + 4 * M)
    fork = caller(lib.sdpa_pages_fork, "refs n_pages table st rows new nst nrows cols P lens src dst n a b c missing", refs=base, n_pages=100,
                  table=base + M, st=8, rows=4, new=base + M, nst=8, nrows=4, cols=8, P=16, lens=base + 2 * M, src=base + 3 * M,
                  dst=base + 4 * M, n=3, a=base + 5 * M, b=base + 6 * M, c=base + 7 * M, missing=base + 8 * M)
    release = caller(lib.sdpa_pages_release, "refs n_pages table st rows cols P which lo hi n", refs=base, n_pages=100, table=base + M, st=8,
                     rows=4, cols=8, P=16, which=base + 2 * M, lo=base + 3 * M, hi=base + 4 * M, n=3)
    for f in (take, fork, release):
        for kw in (dict(refs=None), dict(table=None)):
            assert f(**kw) == NULL, kw
        for kw in (dict(n_pages=0), dict(n_pages=(1 << 30) + 1), dict(rows=0), dict(cols=0), dict(P=24), dict(P=8), dict(cols=1 << 28, st=1 << 28)):
            assert f(**kw) == SHAPE, kw
        for kw in (dict(refs=base + 8), dict(table=base + M + 2), dict(st=7), dict(st=0)):
            assert f(**kw) == LAYOUT, kw
        for kw in (dict(refs=base + M), dict(refs=base + M + 112)):
            assert f(**kw) == ARG, kw
    for kw in (dict(lo=None), dict(hi=None), dict(missing=None)):
        assert take(**kw) == NULL
    assert take(rows=32769) == SHAPE and take(rows=32768, cols=1 << 17, st=1 << 17) == SHAPE
    assert take(lo=base + 1) == LAYOUT and take(missing=base + 2) == LAYOUT
    for kw in (dict(lo=base + 396), dict(hi=base + M + 124), dict(missing=base), dict(missing=base + M), dict(missing=base + 2 * M)):
        assert take(**kw) == ARG, kw
    for name in ("new", "lens", "src", "dst", "a", "b", "c", "missing"):
        assert fork(**{name: None}) == NULL
    assert fork(n=0) == SHAPE and fork(n=32769) == SHAPE and fork(new=base + 9 * M, nrows=0) == SHAPE
    assert fork(new=base + 9 * M, nst=4) == LAYOUT and fork(src=base + 3 * M + 1) == LAYOUT
    for kw in (dict(nrows=5), dict(nst=9), dict(new=base + M + 64), dict(a=base + 6 * M + 8), dict(c=base + 3 * M), dict(missing=base + 5 * M),
               dict(new=base + 9 * M, a=base + 9 * M), dict(new=base + 2 * M)):
        assert fork(**kw) == ARG, kw
    assert release(n=0) == SHAPE and release(which=None, n=5) == SHAPE and release(n=1 << 31) == SHAPE
    assert release(lo=base + 2) == LAYOUT
    for kw in (dict(which=base), dict(lo=base + M), dict(hi=base + M + 60)):
        assert release(**kw) == ARG, kw

    s = sdpa._PagedCacheStruct(base, base + 64 * M, None, None, 10, 16, 2, 64, (2048, 128, 64), (2048, 128, 64), 0)
    at = ctypes.addressof(s)
    copy = caller(lib.sdpa_cache_copy_pages, "cache src dst rows n", cache=at, src=base + 128 * M, dst=base + 129 * M, rows=base + 130 * M, n=5)
    compact = caller(lib.sdpa_cache_compact, "cache table st cols kept kst most lens new nst ncols n", cache=at, table=base + 128 * M, st=4,
                     cols=4, kept=base + 129 * M, kst=9, most=9, lens=base + 130 * M, new=base + 131 * M, nst=2, ncols=2, n=3)
    for f in (copy, compact):
        assert f(cache=None) == NULL
        for field, value, want in (("k", None, NULL), ("elem", 7, DTYPE), ("elem", 2, NULL), ("head_dim", 32, SHAPE), ("page_size", 8, SHAPE),
                                   ("n_pages", 0, SHAPE), ("k", base + 8, LAYOUT), ("v", base, ARG), ("v", base + 512, ARG)):
            keep = getattr(s, field)
            setattr(s, field, value)
            assert f() == want, (field, value)
            setattr(s, field, keep)
    for kw in (dict(src=None), dict(dst=None)):
        assert copy(**kw) == NULL
    assert copy(n=0) == SHAPE and copy(n=1 << 31) == SHAPE and copy(rows=base + 128 * M + 1) == LAYOUT
    for kw in (dict(src=base), dict(dst=base + 64 * M + 40), dict(rows=base + 1000)):
        assert copy(**kw) == ARG, kw
    for kw in (dict(table=None), dict(kept=None), dict(new=None)):
        assert compact(**kw) == NULL
    for kw in (dict(n=0), dict(cols=0), dict(most=0), dict(ncols=0), dict(cols=1 << 28, st=1 << 28), dict(ncols=1 << 28, nst=1 << 28), dict(n=1 << 31)):
        assert compact(**kw) == SHAPE, kw
    for kw in (dict(st=3), dict(kst=8), dict(nst=1), dict(lens=base + 2), dict(kept=base + 129 * M + 2)):
        assert compact(**kw) == LAYOUT, kw
    for kw in (dict(table=base), dict(kept=base + 64), dict(lens=base + 64 * M), dict(new=base + 32 * 1024)):
        assert compact(**kw) == ARG, kw


@gpu
def test_far_pages(sdpa_lib):
    """Pages that begin behind 2^31 elements and 2^32 bytes: copied, compacted, read in a window."""
    D, hkv, P, n_pages = 128, 8, 1024, 2200
    k, v = (torch.empty(n_pages, P, hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c = sdpa_lib.SdpaPagedCache(k, v)
    g = torch.Generator(device="cuda").manual_seed(3)
    for x in (k, v):
        x[5].normal_(generator=g)
        x[2150].normal_(generator=g)
    sdpa_lib.sdpa_cache_copy_pages(c, i32([5, 2150]), i32([2199, 9]))
    for x in (k, v):
        assert torch.equal(x[2199], x[5]) and torch.equal(x[9], x[2150])
    pos = torch.randperm(2 * P, generator=torch.Generator().manual_seed(3))[:700]
    sdpa_lib.sdpa_cache_compact(c, i32([[2199, 2150]]), pos[None].to(torch.int32).cuda(), i32([[2180]]))
    for x in (k, v):
        want = torch.cat([x[5], x[9]])[pos.cuda()]
        assert torch.equal(x[2180, :700], want)
    q = torch.randn(3, 16, D, generator=g, device="cuda").bfloat16()
    lens = i32([1500])
    near, far = i32([[5, 9]]), i32([[2199, 2150]])
    for rows in (1, 3):
        a, b = (sdpa_lib.sdpa_paged_forward(q[:rows], c, t, lens, is_causal=True, window=700, sinks=5) for t in (near, far))
        assert torch.equal(a, b)
    wide = torch.randn(90, 16, D, generator=g, device="cuda").bfloat16()
    a, b = (sdpa_lib.sdpa_paged_forward(wide, c, t, lens, is_causal=True, window=700, sinks=5) for t in (near, far))
    assert torch.equal(a, b)
