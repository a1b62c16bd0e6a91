"""The paged operators' two ways from Python to the library: the compiled module's, which calls on the current stream
take, and the one in Python, which looks at every argument and is taken for a stream that is named.  Both give the
same; what the first does not take is refused, by name, by the second."""
import pytest
import torch

from tests.test_paged import make_cache, tables

pytestmark = pytest.mark.gpu
NULL, SHAPE, DTYPE, LAYOUT, ARG = 1, 3, 4, 5, 6


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Calls:
    """The operators on one small state, each with a dict of keywords added."""

    def __init__(self, lib, kind="e4m3", dtype=torch.bfloat16):
        self.lib, self.kind, self.dtype = lib, kind, dtype
        g = torch.Generator().manual_seed(3)
        self.q, self.k, self.v = (torch.randn(7, h, 64, generator=g).to(dtype).cuda() for h in (8, 2, 2))
        self.table, self.lens, self.cu = tables(3, 5, 20, 3).cuda(), i32([40, 70, 33]), i32([0, 3, 4, 7])
        a = torch.arange(80, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
        self.cos, self.sin = a.cos().float().cuda(), a.sin().float().cuda()
        self.w = torch.nn.Parameter((1 + 0.2 * torch.randn(64, generator=g)).cuda())

    def cache(self):
        return make_cache(self.lib, 20, 16, 2, 64, self.kind, self.dtype, 4)

    @staticmethod
    def held(c):
        return [x.view(torch.uint8) for x in (c.k, c.v)] + [x for x in (c.k_scale, c.v_scale) if x is not None]

    def append(self, **kw):
        c = self.cache()
        out = self.lib.sdpa_cache_append(c, self.k, self.v, self.table, self.lens, self.cu, cos=self.cos, sin=self.sin, q=self.q, **kw)
        return [out] + self.held(c)

    def forward(self, **kw):
        out = self.lib.sdpa_paged_forward(self.q, self.cache(), self.table, self.lens, self.cu, 3, **kw)
        return list(out) if isinstance(out, tuple) else [out]

    def rotate(self, **kw):
        return [x for x in self.lib.sdpa_norm_rotate(self.q, self.k, i32([0, 5, 9, 79, 3, 3, 1]), cos=self.cos, sin=self.sin, **kw)]

    def pages(self, **kw):
        refs = torch.zeros(30, dtype=torch.int32, device="cuda")
        t = torch.full((4, 6), -1, dtype=torch.int32, device="cuda")
        a = self.lib.sdpa_pages_take(refs, t, i32([0] * 4), i32([40, 0, 90, 1]), 16, **kw)
        b = self.lib.sdpa_pages_fork(refs, t, i32([40, 0, 90, 1]), i32([0, 2]), i32([1, 3]), 16, **kw)
        self.lib.sdpa_pages_release(refs, t, i32([17, 0]), None, 16, i32([2, 0]), **kw)
        new = torch.full((2, 6), -1, dtype=torch.int32, device="cuda")
        d = self.lib.sdpa_pages_fork(refs, t, i32([40, 0, 90, 1]), i32([1]), i32([1]), 16, new, **kw)
        self.lib.sdpa_pages_release(refs, t, None, i32([64] * 4), 16, **kw)
        return [refs, t, a, *b, *d, new]

    def move(self, **kw):
        c = self.cache()
        self.lib.sdpa_cache_copy_pages(c, i32([1, 2]), i32([5, 6]), **kw)
        self.lib.sdpa_cache_copy_pages(c, i32([3, 4]), i32([7, 8]), i32([5, 16]), **kw)
        self.lib.sdpa_cache_compact(c, i32([[1, 2]]), i32([[3, 31, 17, 0]]), i32([[10]]), i32([3]), **kw)
        self.lib.sdpa_cache_compact(c, i32([[1, 2]]), i32([[3, 31, 17, 0]]), i32([[11]]), **kw)
        return self.held(c)


def same(a, b):
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert x.dtype == y.dtype and x.shape == y.shape and torch.equal(x, y)


@pytest.mark.parametrize("kind,dtype", [("e4m3", torch.bfloat16), ("16", torch.float16)])
def test_both_ways_give_the_same(sdpa_lib, kind, dtype):
    calls = Calls(sdpa_lib, kind, dtype)
    runs = [("append", {}), ("append", dict(interleaved=True)), ("append", dict(q_norm=calls.w, k_norm=calls.w, eps=1e-5)),
            ("append", dict(k_norm=calls.w)), ("forward", {}), ("forward", dict(is_causal=True, return_lse=True)),
            ("forward", dict(is_causal=True, window=20, sinks=3, scale=0.3)), ("rotate", {}),
            ("rotate", dict(q_norm=calls.w, k_norm=calls.w, eps=1e-3, interleaved=True)), ("pages", {}), ("move", {})]
    side = torch.cuda.Stream()
    for name, kw in runs:
        f = getattr(calls, name)
        want = f(stream=torch.cuda.current_stream(), **kw)
        same(f(**kw), want)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):   # (current there)
            got = f(**kw)
        side.synchronize()
        same(got, want)


def test_results_are_the_given_tensors(sdpa_lib):
    calls = Calls(sdpa_lib)
    out, lse = torch.empty_like(calls.q), torch.empty(7, 8, device="cuda")
    got = sdpa_lib.sdpa_paged_forward(calls.q, calls.cache(), calls.table, calls.lens, calls.cu, 3, out, lse=lse)
    assert got[0] is out and got[1] is lse
    same(list(got), calls.forward(return_lse=True))
    q = calls.q.clone()
    assert sdpa_lib.sdpa_cache_append(calls.cache(), calls.k, calls.v, calls.table, calls.lens, calls.cu, q=q, q_out=q) is q
    assert sdpa_lib.sdpa_cache_append(calls.cache(), calls.k, calls.v, calls.table, calls.lens, calls.cu) is None
    q, k = calls.q.clone(), calls.k.clone()
    a, b = sdpa_lib.sdpa_norm_rotate(q, k, q_norm=calls.w, q_out=q, k_out=k)
    assert a is q and b is k
    a, b = sdpa_lib.sdpa_norm_rotate(calls.q, q_norm=calls.w)
    assert b is None and torch.equal(a, q)
    # an eps that is a whole number, a bound that is numpy's
    sdpa_lib.sdpa_norm_rotate(calls.q, q_norm=calls.w, eps=1)
    import numpy as np
    same([sdpa_lib.sdpa_paged_forward(calls.q, calls.cache(), calls.table, calls.lens, calls.cu, np.int64(3))], calls.forward())


def test_refusals_on_the_device(sdpa_lib):
    lib, calls = sdpa_lib, Calls(sdpa_lib)
    c, q, k, t, lens, cu = calls.cache(), calls.q, calls.k, calls.table, calls.lens, calls.cu
    wide = torch.zeros(7, 8, 128, dtype=torch.bfloat16, device="cuda")
    n, refs, rows = i32([0, 0, 0]), torch.zeros(9, dtype=torch.int32, device="cuda"), torch.zeros(3, 5, dtype=torch.int32, device="cuda")
    for status, f, args, kw in (
            (DTYPE, lib.sdpa_cache_append, (c, k.float(), k.float(), t, lens, cu), {}),
            (SHAPE, lib.sdpa_cache_append, (c, k, k[:, :1], t, lens, cu), {}),
            (ARG, lib.sdpa_cache_append, (c, k, k.cpu(), t, lens, cu), {}),
            (ARG, lib.sdpa_cache_append, (c, k, calls.v, t, lens, cu), dict(k_norm=calls.w.detach(), eps=0.0)),
            (LAYOUT, lib.sdpa_cache_append, (c, k.transpose(1, 2).contiguous().transpose(1, 2), calls.v, t, lens, cu), {}),
            (LAYOUT, lib.sdpa_cache_append, (c, wide[:, :2, 1:65], calls.v, t, lens, cu), {}),
            (DTYPE, lib.sdpa_paged_forward, (q.half().float(), c, t, lens, cu, 3), {}),
            (SHAPE, lib.sdpa_paged_forward, (q[:, :7], c, t, lens, cu, 3), {}),
            (NULL, lib.sdpa_paged_forward, (q, c, t, lens, cu), {}),
            (ARG, lib.sdpa_paged_forward, (q, c, t, lens, cu, 3, q), {}),
            (ARG, lib.sdpa_paged_forward, (q, c, t, lens, cu, 3), dict(window=0, is_causal=True)),
            (ARG, lib.sdpa_paged_forward, (q, c, t, lens, cu, 3), dict(window=5)),
            (ARG, lib.sdpa_paged_forward, (q, c, t, lens, cu, 3), dict(sinks=2)),
            (ARG, lib.sdpa_paged_forward, (q, c, t, lens, cu, 3), dict(scale=float("inf"))),
            (ARG, lib.sdpa_norm_rotate, (q, k), dict(q_out=k.expand(7, 2, 64).repeat(1, 4, 1), k_out=q[:, :2])),
            (SHAPE, lib.sdpa_norm_rotate, (q[:, :, :32],), {}),
            (SHAPE, lib.sdpa_pages_take, (refs, rows, n, n, 24), {}),
            (ARG, lib.sdpa_pages_take, (refs, rows, rows[0, :3], n, 16), {}),
            (SHAPE, lib.sdpa_pages_fork, (refs, rows, n, n[:0], n[:0], 16), {}),
            (ARG, lib.sdpa_pages_fork, (refs, rows, n, n, n, 16, rows[:2]), {}),
            (SHAPE, lib.sdpa_pages_release, (refs, rows, n[:2], None, 16), {}),
            (LAYOUT, lib.sdpa_pages_release, (refs, rows, i32([0] * 6)[::2], None, 16), {}),
            (SHAPE, lib.sdpa_cache_copy_pages, (c, n, n[:2]), {}),
            (ARG, lib.sdpa_cache_copy_pages, (c, n, n.cpu()), {}),
            (SHAPE, lib.sdpa_cache_compact, (c, t, t[:2], t), {}),
            (DTYPE, lib.sdpa_cache_compact, (c, t, t.long(), t), {})):
        with pytest.raises(lib.SdpaError) as e:
            f(*args, **kw)
        assert e.value.status == status, (f.__name__, status, e.value.status)


def test_two_streams_at_once(sdpa_lib):
    """Calls that run beside each other share nothing: attention (a workspace each), norms, moves of other pages."""
    lib = sdpa_lib
    g = torch.Generator().manual_seed(7)
    n_pages, P = 400, 16
    c = make_cache(lib, n_pages, P, 2, 128, "e4m3", torch.bfloat16, 4)
    lens = i32([1500, 700, 1, 40])
    tabs = [tables(4, 94, n_pages, s).cuda() for s in (1, 2)]
    qs = [torch.randn(4, 8, 128, generator=g).bfloat16().cuda() for _ in range(2)]
    many = [torch.randn(200, 8, 128, generator=g).bfloat16().cuda() for _ in range(2)]
    cu = i32([0, 90, 91, 92, 200])
    moved = [make_cache(lib, 40, P, 2, 128, "e4m3", torch.bfloat16, 4) for _ in range(2)]
    w = torch.rand(128, generator=g).cuda()

    def work(i):
        lib.sdpa_cache_copy_pages(moved[i], i32([1, 2, 3]), i32([11, 12, 13]))
        lib.sdpa_cache_compact(moved[i], i32([[11, 12]]), i32([list(range(1, 32, 2))]), i32([[20]]))
        return [lib.sdpa_paged_forward(qs[i], c, tabs[i], lens, is_causal=True, window=300, sinks=4),
                lib.sdpa_paged_forward(many[i], c, tabs[i], lens, cu, 108, is_causal=True, window=100, sinks=20),
                lib.sdpa_norm_rotate(many[i], q_norm=w)[0], moved[i].k[20].view(torch.uint8).clone()]

    want = [work(0), work(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(work(i))
    torch.cuda.synchronize()
    for i in range(2):
        for x in got[i]:
            same(x, want[i])
