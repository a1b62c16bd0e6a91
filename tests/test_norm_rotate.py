"""Norms of query and key heads with the rotation in the same pass, on the way into a paged cache and in rows without
one: against a plain 64-bit form, and each beside the other."""
import math

import numpy as np
import pytest
import torch

import scaled_dot_product_forward_gb300 as sdpa
from tests import paged_ref as ref
from tests.test_paged import check, make_cache, tables

E4M3 = torch.float8_e4m3fn
gpu = pytest.mark.gpu
U = 2.0 ** -24   # half a step of fp32, relatively


def angles(n, rot, seed=1):
    a = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
    return (a + seed).cos().float(), (a + seed).sin().float()


def turned(x, weight, eps, pos, cos, sin, interleaved):
    """x [tokens, heads, D] normalised (weight not None) and rotated (cos not None) in 64 bits, with a bound on what
    fp32 arithmetic may lose of it before the last rounding.

    The norm: at most ten roundings on a sum of squares (positive terms: relative to the sum), half of which pass
    through the root, two ulp of the reciprocal root (4 U), and a product with the row's factor and the weight: 11 U
    of |y|.  The rotation: that of both products' factors, a rounding each, and one of the sum: 13 U of |a c| + |b s|."""
    y, lost = x.double(), torch.zeros(x.shape, dtype=torch.float64)
    if weight is not None:
        y = y / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + float(np.float32(eps))) * weight.double()
        lost = 11 * U * y.abs()
    if cos is None:
        return y, lost
    half = cos.shape[1]
    c, s = cos.double()[pos][:, None], sin.double()[pos][:, None]
    a = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    b = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    z = y.clone()
    z[..., a] = y[..., a] * c - y[..., b] * s
    z[..., b] = y[..., b] * c + y[..., a] * s
    lost = lost.clone()
    for this, other in ((a, b), (b, a)):
        lost[..., this] = 13 * U * ((y[..., this] * c).abs() + (y[..., other] * s).abs())
    return z, lost


def rounded(y, lost, dtype):
    """Bound with the one rounding to a 16-bit type (half its least subnormal step too)."""
    least = torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2
    return ref.half_step(dtype) * (y.abs() + lost) + lost + least + 1e-40


def rows(total, heads, D, dtype, seed, spread=1.0):
    x = torch.randn(total, heads, D, generator=torch.Generator().manual_seed(seed)) * spread
    x[..., :: D // 4] *= 8
    return x.to(dtype)


def weights(D, seed):
    return 1 + 0.3 * torch.randn(D, generator=torch.Generator().manual_seed(seed))


ROWS = [  # D, dtype, total, heads, kv heads, rot (0: none), interleaved, which norms
    (128, torch.bfloat16, 1, 1, 1, 128, False, "qk"),
    (128, torch.float16, 7, 32, 8, 128, True, "qk"),
    (128, torch.bfloat16, 300, 5, 3, 64, False, "k"),
    (128, torch.float16, 33, 64, 1, 24, True, "q"),
    (128, torch.bfloat16, 2500, 3, 0, 128, False, "q"),
    (64, torch.bfloat16, 1, 16, 16, 64, False, "qk"),
    (64, torch.float16, 1000, 9, 2, 32, True, "qk"),
    (64, torch.bfloat16, 129, 33, 17, 8, False, "qk"),
    (64, torch.float16, 5, 48, 4, 0, False, "qk"),
    (128, torch.bfloat16, 6, 24, 8, 0, False, "k"),
    (64, torch.bfloat16, 40, 4, 2, 64, True, ""),
]


@gpu
@pytest.mark.parametrize("place", ["new", "in place", "side by side"])
@pytest.mark.parametrize("case", ROWS, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_rows(sdpa_lib, case, place):
    D, dtype, total, H, Hkv, rot, interleaved, norms = case
    q, k = rows(total, H, D, dtype, 1), rows(total, max(Hkv, 1), D, dtype, 2, 0.01)
    if total > 4:
        q[3] = 0            # rows of zeros stay zeros
        k[2, 0] = 0
    qw, kw = weights(D, 3) if "q" in norms else None, weights(D, 4) if "k" in norms else None
    pos = torch.randint(0, 5000, (total,), generator=torch.Generator().manual_seed(6))
    cos, sin = angles(5000, rot) if rot else (None, None)
    if place == "side by side":
        both = torch.cat([q, k, torch.zeros(total, 2, D, dtype=dtype)], 1).cuda()
        dq, dk = both[:, :H], both[:, H:H + max(Hkv, 1)]
    else:
        dq, dk = q.cuda(), k.cuda()
    kw_args = dict(cos=cos.cuda() if rot else None, sin=sin.cuda() if rot else None, interleaved=interleaved,
                   q_norm=qw.cuda() if qw is not None else None, k_norm=kw.cuda() if kw is not None else None, eps=1e-5)
    if Hkv == 0:
        dk = None
        kw_args.pop("k_norm")
    if place != "new":
        kw_args.update(q_out=dq, k_out=dk)
    got_q, got_k = sdpa_lib.sdpa_norm_rotate(dq, dk, pos.to(torch.int32).cuda(), **kw_args)
    if place != "new":
        assert got_q is dq and got_k is dk
    for got, x, w in ((got_q, q, qw), (got_k, k, kw)):
        if got is None:
            continue
        y, lost = turned(x, w, 1e-5, pos, cos, sin, interleaved)
        check(got, y, rounded(y, lost, dtype), "rows")
    if place == "side by side":
        assert torch.all(both[:, H + max(Hkv, 1):] == 0)


@gpu
def test_rows_left_out_and_numbered(sdpa_lib):
    """Rows without a place in the tables keep what their outputs hold; no positions are the rows' numbers."""
    q, k = rows(40, 4, 64, torch.bfloat16, 1).cuda(), rows(40, 2, 64, torch.bfloat16, 2).cuda()
    cos, sin = (x.cuda() for x in angles(30, 64))
    w = weights(64, 3).cuda()
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    q0, k0 = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    kw = dict(cos=cos, sin=sin, q_norm=w, k_norm=w)
    a = sdpa_lib.sdpa_norm_rotate(q, k, pos - 5, q_out=q0, k_out=k0, **kw)
    left = torch.zeros(40, dtype=torch.bool, device="cuda")
    left[:5] = left[35:] = True
    for x in a:
        assert torch.all(x[left] == 7) and not torch.any((x[~left] == 7).flatten(1).all(1))
    b = sdpa_lib.sdpa_norm_rotate(q[5:35], k[5:35], **kw)
    assert torch.equal(a[0][5:35], b[0]) and torch.equal(a[1][5:35], b[1])


@gpu
@pytest.mark.parametrize("D", [64, 128])
def test_large_and_small_values(sdpa_lib, D):
    """bf16 rows whose squares overflow fp32 or vanish in it, beside ordinary ones in the same warp; infinities and NaN."""
    q = rows(6, 8, D, torch.bfloat16, 5)
    for i, f in enumerate((1e30, 3e37, 1e-25, 1.0, 2.0 ** 61, 2.0 ** 66)):
        q[i, ::2] = (q[i, ::2].double().clamp(-8, 8) * f).to(torch.bfloat16)
    w = weights(D, 3)
    for eps in (1e-6, 2.0 ** -100):
        got, _ = sdpa_lib.sdpa_norm_rotate(q.cuda(), q_norm=w.cuda(), eps=eps)
        y, lost = turned(q, w, eps, None, None, None, False)
        # (the factor of rows above 2^102 is below fp32's least normal: half a step of 2^-149)
        huge = q.double().abs().amax(-1, keepdim=True)
        check(got, y, rounded(y, lost + huge * 2.0 ** -149 * w.double().abs(), torch.bfloat16), f"eps {eps}")
    bad = rows(3, 2, D, torch.bfloat16, 6)
    bad[0, 0, 5], bad[1, 1, 9] = math.inf, math.nan
    got = sdpa_lib.sdpa_norm_rotate(bad.cuda(), q_norm=w.cuda())[0].cpu()
    assert torch.isnan(got[0, 0, 5]) and torch.all(got[0, 0, :5] == 0) and torch.all(got[0, 0, 6:] == 0)
    assert torch.isnan(got[1, 1]).all()
    assert torch.isfinite(got[2]).all() and torch.isfinite(got[0, 1]).all() and torch.isfinite(got[1, 0]).all()


APPEND = [  # D, cache, dtype, page, kv heads, G, memory order, rot, interleaved, norms, counts, lengths
    (128, "e4m3", torch.bfloat16, 16, 2, 4, "tokens", 128, False, "qk", [1, 1, 1], [1, 16, 17]),
    (128, "e4m3", torch.float16, 64, 1, 8, "heads", 64, True, "qk", [70, 0, 3], [100, 5, 3]),
    (128, "16", torch.bfloat16, 32, 3, 1, "tokens", 128, False, "qk", [33, 1, 5], [40, 31, 5]),
    (64, "e4m3", torch.bfloat16, 128, 2, 3, "padded", 32, False, "k", [200, 9], [210, 137]),
    (64, "16", torch.float16, 16, 4, 4, "heads", 64, True, "q", [1, 17, 2], [9, 17, 33]),
    (64, "e4m3", torch.float16, 16, 1, 1, "tokens", 0, False, "qk", [40, 2], [41, 18]),
    (128, "16", torch.bfloat16, 64, 2, 2, "padded", 0, False, "k", [3, 65], [3, 70]),
    (128, "e4m3", torch.bfloat16, 256, 1, 2, "tokens", 128, False, "qk", [300, 1], [301, 257]),
]


@gpu
@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"D{c[0]}-{c[1]}-{str(c[2])[6:]}-P{c[3]}-{c[4]}x{c[5]}-{c[6]}-rot{c[7]}-{c[9]}-{c[10]}")
def test_append(sdpa_lib, case):
    D, kind, dtype, P, hkv, G, order, rot, interleaved, norms, counts, lens = case
    mp = -(-max(lens) // P) + 1
    n_pages = len(lens) * mp + 2
    c = make_cache(sdpa_lib, n_pages, P, hkv, D, kind, dtype, 4, order)
    total = sum(counts)
    q, k, v = rows(total, hkv * G, D, dtype, 1), rows(total, hkv, D, dtype, 2, 3.0), rows(total, hkv, D, dtype, 3)
    qw, kw = weights(D, 3) if "q" in norms else None, weights(D, 4) if "k" in norms else None
    cos, sin = angles(max(lens), rot) if rot else (None, None)
    t = tables(len(lens), mp, n_pages, 3)
    before = [x.clone() for x in (c.k.float(), c.v.float())]
    scales = [None if s is None else s.clone().cpu().double() for s in (c.k_scale, c.v_scale)]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    got = sdpa_lib.sdpa_cache_append(
        c, k.cuda(), v.cuda(), t.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), cu, cos=cos.cuda() if rot else None,
        sin=sin.cuda() if rot else None, interleaved=interleaved, q=q.cuda(), q_norm=qw.cuda() if qw is not None else None,
        k_norm=kw.cuda() if kw is not None else None, eps=1e-6)
    pos = torch.cat([torch.arange(L - n, L) for n, L in zip(counts, lens)])
    y, lost = turned(q, qw, 1e-6, pos, cos, sin, interleaved)
    check(got, y, rounded(y, lost, dtype), "queries")
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(counts)])
    page, row = t[seq, pos // P].long(), pos % P
    for name, x, w, cache, scale, old, old_scale in (("k", k, kw, c.k, c.k_scale, before[0], scales[0]),
                                                     ("v", v, None, c.v, c.v_scale, before[1], scales[1])):
        y, lost = turned(x, w, 1e-6, pos, cos if name == "k" else None, sin if name == "k" else None, interleaved)
        held = cache.float().cpu().double()
        if scale is None:
            check(held[page, row], y, rounded(y, lost, dtype), name)
        else:
            now = scale.cpu().double()
            for p in page.unique().tolist():
                mine = page == p
                begin = int(row[mine].min())
                for h in range(hkv):
                    top = y[mine][:, h].abs().max().item()
                    off = lost[mine][:, h].max().item()
                    least = old_scale[p, h].item() if begin > 0 else 0.0
                    # (the largest value may be on either side of a border)
                    assert now[p, h].item() in {max(least, ref.scale_for(max(top + d, 0.0))) for d in (-off, 0.0, off)}, (name, p, h)
            s = now[page][:, :, None]
            tol = ref.half_step(E4M3) * (y.abs() + lost) + lost + s * 2.0 ** -10
            check(held[page, row] * s, y, tol, name)
        # rows that are nobody's are as they were (those of 8-bit pages under the scale of now)
        others = torch.ones(held.shape[:2], dtype=torch.bool)
        others[page, row] = False
        if scale is not None:
            others[page] = False
        assert torch.equal(held[others], old.cpu().double()[others])


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_both_ways_are_one(sdpa_lib, D, interleaved):
    """The rows that the append writes are those of sdpa_norm_rotate, bit for bit; without norms both give the plain
    append's; a norm of one of the two leaves the other."""
    lens, counts, P = [60, 5, 300], [37, 5, 260], 64
    total = sum(counts)
    q, k, v = (rows(total, h, D, torch.bfloat16, s).cuda() for h, s in ((12, 1), (3, 2), (3, 3)))
    cos, sin = (x.cuda() for x in angles(300, D))
    qw, kw = weights(D, 5).cuda(), weights(D, 6).cuda()
    t = tables(3, 5, 17, 3)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(L - n, L) for n, L in zip(counts, lens)]).to(torch.int32)
    seq = torch.cat([torch.full((n,), b) for b, n in enumerate(counts)])
    page, row = t[seq, pos // P].long(), (pos % P).long()

    def append(**kw):
        c = make_cache(sdpa_lib, 17, P, 3, D, "16", torch.bfloat16, 4)
        got = sdpa_lib.sdpa_cache_append(c, k, v, t.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), cu, cos=cos,
                                         sin=sin, interleaved=interleaved, q=q, **kw)
        return got, c.k[page, row]

    plain_q, plain_k = append()
    for norms in (dict(q_norm=qw, k_norm=kw), dict(q_norm=qw), dict(k_norm=kw), {}):
        a = append(**norms)
        b = sdpa_lib.sdpa_norm_rotate(q, k, pos.cuda(), cos=cos, sin=sin, interleaved=interleaved, **norms)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]), list(norms)
        if "q_norm" not in norms:
            assert torch.equal(a[0], plain_q)
        if "k_norm" not in norms:
            assert torch.equal(a[1], plain_k)


@gpu
def test_captured_and_on_a_side_stream(sdpa_lib):
    q, k = rows(50, 8, 128, torch.float16, 1).cuda(), rows(50, 2, 128, torch.float16, 2).cuda()
    cos, sin = (x.cuda() for x in angles(100, 128))
    w = weights(128, 3).cuda()
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    kw = dict(cos=cos, sin=sin, q_norm=w, k_norm=w)
    want = sdpa_lib.sdpa_norm_rotate(q, k, pos, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = sdpa_lib.sdpa_norm_rotate(q, k, pos, stream=side, **kw)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sdpa_lib.sdpa_norm_rotate(q, k, pos, **kw)
    graph.replay()
    for a in (other, out):
        assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])
    pos.add_(13)
    q.mul_(2)
    graph.replay()
    want = sdpa_lib.sdpa_norm_rotate(q, k, pos, **kw)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_refusals():
    from tests.test_paged_refusals import cache, status
    NULL, SHAPE, DTYPE, LAYOUT, ARG = 1, 3, 4, 5, 6
    f = sdpa.sdpa_norm_rotate
    q, k, w = torch.zeros(4, 6, 64).bfloat16(), torch.zeros(4, 2, 64).bfloat16(), torch.ones(64)
    cos, sin = torch.zeros(9, 32), torch.zeros(9, 32)
    assert status(f, q.float()) == DTYPE
    assert status(f, q, k.half()) == DTYPE
    assert status(f, q, k, q_out=q.half()) == DTYPE
    assert status(f, q, k, torch.zeros(4)) == DTYPE
    assert status(f, q, k, torch.zeros(4, dtype=torch.int64)) == DTYPE
    assert status(f, q, k, q_norm=w.half()) == DTYPE
    assert status(f, q, k, cos=cos.half(), sin=sin.half()) == DTYPE
    assert status(f, q, k_norm=w) == NULL
    assert status(f, q, k_out=k) == NULL
    assert status(f, q, k, cos=cos) == NULL
    assert status(f, q[0]) == SHAPE
    assert status(f, q, k[:3]) == SHAPE
    assert status(f, q, k[..., :32]) == SHAPE
    assert status(f, q, k, q_out=q[:, :3]) == SHAPE
    assert status(f, q, k, k_out=k[:, :1]) == SHAPE
    assert status(f, q, k, torch.zeros(3, dtype=torch.int32)) == SHAPE
    assert status(f, q, k, torch.zeros(4, 1, dtype=torch.int32)) == SHAPE
    assert status(f, q, k, q_norm=torch.ones(32)) == SHAPE
    assert status(f, q, k, q_norm=torch.ones(64, 1)) == SHAPE
    assert status(f, q, k, cos=cos, sin=sin[:3]) == SHAPE
    assert status(f, q, k, torch.zeros(8, dtype=torch.int32)[::2]) == LAYOUT
    assert status(f, q, k, q_norm=torch.ones(128)[::2]) == LAYOUT
    assert status(f, q, k, cos=torch.zeros(32, 9).t(), sin=torch.zeros(32, 9).t()) == LAYOUT
    # host tensors never reach a kernel
    assert status(f, q, k, q_norm=w, k_norm=w) == ARG
    c = cache()
    a, t, lens, kv = sdpa.sdpa_cache_append, torch.zeros(2, 3, dtype=torch.int32), torch.ones(2, dtype=torch.int32), k[:2]
    assert status(a, c, kv, kv.clone(), t, lens, q_norm=w) == NULL
    assert status(a, c, kv, kv.clone(), t, lens, k_norm=w.double()) == DTYPE
    assert status(a, c, kv, kv.clone(), t, lens, k_norm=w[:32]) == SHAPE
    assert status(a, c, kv, kv.clone(), t, lens, q=q[:2], q_norm=torch.ones(128)[::2]) == LAYOUT
    assert status(a, c, kv, kv.clone(), t, lens, k_norm=w) == ARG


def test_refusals_of_the_c_entry():
    """Addresses that are never read: everything is refused before any CUDA call."""
    import ctypes
    NULL, SHAPE, DTYPE, LAYOUT, ARG = 1, 3, 4, 5, 6
    lib = sdpa.load_library()
    st = lambda *x: ctypes.addressof(keep.setdefault(x, (ctypes.c_int64 * len(x))(*x)))   # noqa: E731
    keep = {}
    base = 1 << 32

    def f(**kw):
        d = dict(q=base, qo=base + (1 << 20), H=2, qs=st(128, 64), qos=st(128, 64), k=base + (2 << 20), ko=base + (3 << 20), Hk=1,
                 ks=st(64, 64), kos=st(64, 64), dt=0, total=4, D=64, pos=base + (4 << 20), cos=base + (5 << 20), sin=base + (6 << 20),
                 n_pos=9, rot=64, inter=0, qn=base + (7 << 20), kn=base + (8 << 20), eps=1e-6)
        d.update(kw)
        return lib.sdpa_norm_rotate(*[d[n] for n in ("q", "qo", "H", "qs", "qos", "k", "ko", "Hk", "ks", "kos", "dt", "total", "D", "pos",
                                                      "cos", "sin", "n_pos", "rot", "inter", "qn", "kn", "eps")], None)

    for kw in (dict(q=None), dict(qo=None), dict(qs=None), dict(k=None), dict(ko=None), dict(sin=None), dict(k=None, ko=None)):
        assert f(**kw) == NULL, kw
    assert f(dt=2) == DTYPE
    for kw in (dict(D=96), dict(total=0), dict(total=1 << 31), dict(H=0), dict(Hk=0), dict(H=1 << 27), dict(rot=12), dict(rot=72), dict(rot=0),
               dict(n_pos=0)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(q=base + 8), dict(ko=base + (3 << 20) + 2), dict(qs=st(100, 64)), dict(kos=st(0, 64)), dict(pos=base + 2),
               dict(cos=base + (5 << 20) + 4), dict(qn=base + 4), dict(kn=base + 8)):
        assert f(**kw) == LAYOUT, kw
    for kw in (dict(eps=0.0), dict(eps=-1e-6), dict(eps=math.nan), dict(eps=2.0), dict(eps=1e-31), dict(qo=base + 128), dict(ko=base),
               dict(qo=base + (2 << 20)), dict(ko=base + (1 << 20)), dict(qo=base + (4 << 20)), dict(ko=base + (5 << 20)),
               dict(qo=base + (8 << 20)), dict(qo=base, qos=st(256, 128))):
        assert f(**kw) == ARG, kw
