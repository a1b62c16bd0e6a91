"""The forms that only large calls of the paged operators take: forks in two launches, append units of several heads; and
calls that two streams have at work together."""
import numpy as np
import pytest
import torch

from tests import test_pages as pages
from tests.test_norm_rotate import angles, weights
from tests.test_paged import make_cache, tables

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


FORKS = [  # pages, rows, columns, page size, free pages at the end (0: everywhere); pairs: half the rows, or a row less apart
    (150000, 192, 515, 16, 0),
    (60001, 192, 515, 64, 30),       # too few pages for the begun ones
    (30011, 40, 1300, 16, 0),        # two slabs a row, the last one partial
    (30011, 40, 1300, 32, 7),
    (9001, 3, 40001, 16, 1),         # one pair, forty slabs
    (30000, 32, 1024, 128, 0),       # 16 pairs: 16384 entries, one launch
    (30000, 32, 1025, 128, 0),       # 16400 entries, two
    (30000, 34, 1025, 128, 3),
]


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("size", FORKS, ids=str)
def test_fork_of_many_entries(sdpa_lib, size, apart):
    pages.test_fork(sdpa_lib, size, apart)


@pytest.mark.parametrize("apart", [False, True])
def test_captured_fork_of_many_entries(sdpa_lib, apart):
    """Both launches in one graph, replayed on accounts that go on from the last replay's."""
    rows, columns, P = 40, 1300, 16
    refs, table, wide, want, g = pages.state(20000, rows, columns, P, 5)
    new = new_want = None
    if apart:
        _, new, _, other, _ = pages.state(20000, rows, columns, P, 6)
        new_want = other.table
        for row in new_want:
            for p in row:
                if p >= 0:
                    want.refs[p] += 1
        refs.copy_(i32(want.refs))
    lens, src, dst = torch.zeros(rows, dtype=torch.int32, device="cuda"), i32([0] * 20), i32([0] * 20)

    def draw():
        perm = torch.randperm(rows, generator=g).tolist()
        n = [int(x) for x in torch.randint(0, columns * P, (rows,), generator=g)]
        a, b = [perm[20 + int(x)] for x in torch.randint(0, 20, (20,), generator=g)], perm[:20]
        for to, x in ((lens, n), (src, a), (dst, b)):
            to.copy_(i32(x))
        return n, a, b

    saved = [x.clone() for x in (refs, wide)] + ([new.clone()] if apart else [])
    draw()
    sdpa_lib.sdpa_pages_fork(refs, table, lens, src, dst, P, new)        # (loads the kernels)
    for x, y in zip((refs, wide, new), saved):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sdpa_lib.sdpa_pages_fork(refs, table, lens, src, dst, P, new)
    for _ in range(4):
        n, a, b = draw()
        graph.replay()
        copies, missing = want.fork(n, a, b, new_want)
        assert list(zip(got.src.tolist(), got.dst.tolist(), got.rows.tolist())) == copies and got.missing.item() == missing
        pages.agree(refs, table, wide, want)
        assert not apart or new.tolist() == new_want


# (units of a slot's heads, on 152 SMs: ((total / P + 2 sequences) 2 heads) warps / 8 have to be 1216 and more for
# two heads a unit, 2432 for four)
APPENDS = [  # D, dtype, page, kv heads, tokens a sequence; warps and heads a unit
    (128, torch.bfloat16, 16, 8, 1500),     # 2, 4
    (128, torch.float16, 16, 6, 1700),      # 2, 2
    (128, torch.float16, 32, 8, 1500),      # 4, 4
    (128, torch.bfloat16, 32, 10, 1000),    # 4, 2
    (128, torch.bfloat16, 64, 8, 1260),     # 8, 4
    (128, torch.bfloat16, 128, 8, 1260),    # 8, 2
    (128, torch.float16, 256, 32, 1260),    # 8, 4; a page's rows in several batches
    (64, torch.bfloat16, 32, 8, 2900),      # 2, 4
    (64, torch.float16, 64, 16, 1260),      # 4, 4
    (64, torch.bfloat16, 128, 20, 600),     # 8, 2
]


@pytest.mark.parametrize("norms", [False, True])
@pytest.mark.parametrize("case", APPENDS, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_append_of_several_heads_a_unit(sdpa_lib, case, norms):
    """Long e4m3 appends into begun pages, in all heads at once and each head in a cache of its own (whose units have one
    head): bit for bit the same.  Heads' magnitudes differ, so that some scales rise and others stay.  The values, which
    are neither normalised nor rotated, also against the definition."""
    D, dtype, P, hkv, per = case
    B, H = 8, 2 * hkv
    g = torch.Generator().manual_seed(sum(case[2:]) + D)
    before = [5, 0, P - 1, P, 3 * P // 2, 2 * P + 1, 1, P + P // 2]
    fresh = [per, per + 3, 0, per - 1, 2 * per, 1, per, per + P]
    max_pages = max(a + b for a, b in zip(before, fresh)) // P + 1
    n_pages = B * max_pages
    table = tables(B, max_pages, n_pages, 3).cuda()
    cos, sin = (x.cuda() for x in angles(max_pages * P, 64))
    w = weights(D, 3).cuda() if norms else None
    kw = dict(cos=cos, sin=sin, k_norm=w, q_norm=w, interleaved=norms)
    up = torch.exp2(torch.randint(-6, 7, (hkv, 1), generator=g).float())

    def rows(counts, heads, f):
        x = torch.randn(sum(counts), heads, D, generator=g) * f
        x[:, :, ::7] *= torch.exp2(torch.randint(-3, 4, (sum(counts), heads, 1), generator=g).float())
        return x.to(dtype).cuda()

    def lists(counts, base):
        return i32([a + b for a, b in zip(counts, base)]), i32(np.concatenate([[0], np.cumsum(counts)]).tolist())

    first = [rows(before, h, f) for h, f in ((H, 1.0), (hkv, 1.0), (hkv, 1.0))]
    # (with norms a key's size is its weight's: the rows of some sequences are as large as they come without)
    second = [rows(fresh, h, f) for h, f in ((H, 1.0), (hkv, up), (hkv, up.flip(0)))]
    whole = make_cache(sdpa_lib, n_pages, P, hkv, D, "e4m3", dtype, 4)
    single = [sdpa_lib.SdpaPagedCache(whole.k[:, :, h:h + 1].clone(), whole.v[:, :, h:h + 1].clone(),
                                      whole.k_scale[:, h:h + 1].clone(), whole.v_scale[:, h:h + 1].clone()) for h in range(hkv)]
    zero = [0] * B
    for (q, k, v), counts, base in ((first, before, zero), (second, fresh, before)):
        lens, cu = lists(counts, base)
        held = whole.v.clone(), whole.v_scale.clone()
        got = sdpa_lib.sdpa_cache_append(whole, k, v, table, lens, cu, q=q, **kw)
        for h, c in enumerate(single):
            part = slice(2 * h, 2 * h + 2)
            alone = sdpa_lib.sdpa_cache_append(c, k[:, h:h + 1], v[:, h:h + 1], table, lens, cu, q=q[:, part], **kw)
            assert torch.equal(alone, got[:, part])
            for x, y in ((c.k, whole.k), (c.v, whole.v)):
                assert torch.equal(x.view(torch.uint8)[:, :, 0], y.view(torch.uint8)[:, :, h]), h
            for x, y in ((c.k_scale, whole.k_scale), (c.v_scale, whole.v_scale)):
                assert torch.equal(x[:, 0], y[:, h]), h
        check_values(whole, v, table, counts, base, P, held)


def least_scale(most):
    """The least power of two s, in range, with most <= 448 s: found by that comparison, which is exact in 64 bits (a
    logarithm on the device need not be where most is 448 times a power of two)."""
    k = torch.full(most.shape, -50, dtype=torch.float64, device=most.device)
    for e in range(-50, 50):
        k += most.double() > 448 * 2.0 ** e
    return torch.ldexp(torch.ones_like(most), k.int())


def check_values(cache, v, table, counts, base, P, held):
    """The values' pages: scales, new codes and codes that were there, all exact (powers of two; one rounding)."""
    codes, scales = held
    want, want_s = codes.view(torch.uint8).clone(), scales.clone()
    token = 0
    for b, (n, start) in enumerate(zip(counts, base)):
        for e in range(start // P, -(-(start + n) // P) if n else 0):
            page, lo, hi = int(table[b, e]), max(start, e * P), min(start + n, (e + 1) * P)
            new = v[token + lo - start:token + hi - start].float()
            now = least_scale(new.abs().amax((0, 2)))
            row = lo - e * P
            if row:
                old = scales[page]
                now = torch.maximum(now, old)
                raised = (codes[page, :row].float() * (old / now)[:, None]).to(E4M3).view(torch.uint8)
                want[page, :row] = torch.where((now > old)[:, None], raised, want[page, :row])
            want[page, row:row + hi - lo] = (new / now[:, None]).to(E4M3).view(torch.uint8)
            want_s[page] = now
        token += n
    assert torch.equal(cache.v_scale, want_s)
    assert torch.equal(cache.v.view(torch.uint8), want)


def test_two_streams_at_work_together(sdpa_lib):
    """Two streams whose queues are full before either begins (behind a short sleep each): attention of few and of many
    rows, with workspaces of their own, norms, appends, moved pages and accounts; eager, then a captured graph each."""
    lib = sdpa_lib
    g = torch.Generator().manual_seed(7)
    n_pages, P, hkv, D, B, columns = 1200, 16, 2, 128, 4, 150
    c = make_cache(lib, n_pages, P, hkv, D, "e4m3", torch.bfloat16, 4)
    lens, cu = i32([2400, 1700, 1, 640]), i32([0, 190, 191, 192, 400])
    a, b, kept, kept_to = i32([1, 2, 3]), i32([11, 12, 13]), i32([list(range(1, 32, 2))]), i32([[20]])
    old = i32([[11, 12]])
    from_lens, to_lens, src, dst = i32([0] * B), i32([2000, 16, 5, 700]), i32([0, 3]), i32([1, 2])
    w, own = torch.rand(D, generator=g).cuda(), []
    for i in range(2):
        x = {"table": tables(B, columns, n_pages, i + 1).cuda(),
             "q": torch.randn(B, 8, D, generator=g).bfloat16().cuda(), "many": torch.randn(400, 8, D, generator=g).bfloat16().cuda(),
             "k": torch.randn(400, hkv, D, generator=g).bfloat16().cuda(), "mine": make_cache(lib, 1000, P, hkv, D, "e4m3", torch.bfloat16, 4 + i),
             "own_table": tables(B, columns, 700, 9 - i).cuda() + 100, "refs": torch.zeros(600, dtype=torch.int32, device="cuda"),
             "rows": torch.full((B, columns), -1, dtype=torch.int32, device="cuda")}
        own.append(x)

    def work(i):
        x, out = own[i], []
        out.append(lib.sdpa_paged_forward(x["q"], c, x["table"], lens, is_causal=True))
        out.append(lib.sdpa_paged_forward(x["many"], c, x["table"], lens, cu, 208, is_causal=True))
        out.append(lib.sdpa_paged_forward(x["q"], c, x["table"], lens, is_causal=True, window=300, sinks=4))
        out.append(lib.sdpa_paged_forward(x["many"], c, x["table"], lens, cu, 208, is_causal=True, window=100, sinks=20))
        out += [lib.sdpa_norm_rotate(x["many"], q_norm=w)[0],
                lib.sdpa_cache_append(x["mine"], x["k"], x["k"], x["own_table"], lens, cu, q=x["many"], q_norm=w, k_norm=w)]
        lib.sdpa_cache_copy_pages(x["mine"], a, b)
        lib.sdpa_cache_compact(x["mine"], old, kept, kept_to)
        out.append(lib.sdpa_pages_take(x["refs"], x["rows"], from_lens, to_lens, P))
        out += lib.sdpa_pages_fork(x["refs"], x["rows"], to_lens, src, dst, P)
        out += [x["refs"].clone(), x["rows"].clone()]
        lib.sdpa_pages_release(x["refs"], x["rows"], None, None, P)
        out += [x["refs"].clone(), x["mine"].k.view(torch.uint8).clone(), x["mine"].v_scale.clone()]
        return out

    for i in range(2):
        work(i)         # (the caches' pages are then as every later pass leaves them)
    torch.cuda.synchronize()
    want = []
    for i in range(2):
        want.append(work(i))
        torch.cuda.synchronize()
    assert want[0][-3].sum() == 0 and want[0][-5].sum() > 0
    streams, passes = [torch.cuda.Stream(), torch.cuda.Stream()], 6
    got = [[], []]
    for s in streams:
        with torch.cuda.stream(s):
            torch.cuda._sleep(40_000_000)       # (20 ms: the host is ahead of both)
    for _ in range(passes):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(work(i))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(work(i))
        graphs.append(graph)
    for s in streams:
        with torch.cuda.stream(s):
            torch.cuda._sleep(10_000_000)
    for _ in range(20):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for i in range(2):
        for x in [*got[i], outs[i]]:
            assert len(x) == len(want[i])
            for u, v in zip(x, want[i]):
                assert torch.equal(u, v)
