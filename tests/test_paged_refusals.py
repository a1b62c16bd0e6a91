"""What the paged cache's operators refuse: on the host, before any CUDA call
(so that these run without a GPU)."""
import ctypes

import pytest
import torch

import scaled_dot_product_forward_gb300 as sdpa

NULL, RANK, SHAPE, DTYPE, LAYOUT, ARG = 1, 2, 3, 4, 5, 6
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def lib():
    from scaled_dot_product_forward_gb300 import _build
    _build.build()
    return sdpa.load_library()


def cache(**kw):
    shape = kw.pop("shape", (4, 16, 2, 64))
    dtype = kw.pop("dtype", torch.bfloat16)
    k, v = torch.zeros(shape, dtype=dtype), torch.zeros(shape, dtype=dtype)
    return sdpa.SdpaPagedCache(kw.pop("k", k), kw.pop("v", v), **kw)


def status(f, *a, **kw):
    with pytest.raises(sdpa.SdpaError) as e:
        f(*a, **kw)
    return e.value.status


def test_cache_handles():
    z = torch.zeros
    ok = z(4, 16, 2, 64, dtype=torch.bfloat16)
    assert status(sdpa.SdpaPagedCache, ok.float(), ok.float()) == DTYPE
    assert status(sdpa.SdpaPagedCache, ok, ok.half()) == DTYPE
    assert status(sdpa.SdpaPagedCache, ok[0], ok[0]) == SHAPE
    assert status(sdpa.SdpaPagedCache, ok, ok[:3]) == SHAPE
    assert status(cache, shape=(4, 24, 2, 64)) == SHAPE
    assert status(cache, shape=(4, 16, 2, 96)) == SHAPE
    assert status(cache, shape=(0, 16, 2, 64)) == SHAPE
    assert status(cache, k=z(4, 16, 64, 2, dtype=torch.bfloat16).transpose(2, 3)) == LAYOUT
    assert status(cache, k_scale=z(4, 2), v_scale=z(4, 2)) == ARG
    assert status(cache, dtype=E4M3) == NULL
    assert status(cache, dtype=E4M3, k_scale=z(4, 2), v_scale=z(4, 2).double()) == DTYPE
    assert status(cache, dtype=E4M3, k_scale=z(4, 3), v_scale=z(4, 2)) == SHAPE
    assert status(cache, dtype=E4M3, k_scale=z(2, 4).t(), v_scale=z(4, 2)) == LAYOUT


def batch(n=2):
    return torch.zeros(n, 3, dtype=torch.int32), torch.ones(n, dtype=torch.int32)


def test_append_arguments():
    c = cache()
    t, lens = batch()
    k, v, q = (torch.zeros(2, n, 64, dtype=torch.bfloat16) for n in (2, 2, 4))
    f = sdpa.sdpa_cache_append
    assert status(f, c, k.half(), v.half(), t, lens) == DTYPE
    assert status(f, c, k, v.half(), t, lens) == DTYPE
    assert status(f, c, k, v, t.long(), lens) == DTYPE
    assert status(f, c, k, v, t, lens.long()) == DTYPE
    assert status(f, c, k, v, t[:1], lens) == SHAPE
    assert status(f, c, k, v, t, lens, torch.zeros(2, dtype=torch.int32)) == SHAPE
    assert status(f, c, k, v, t.t().contiguous().t(), lens) == LAYOUT
    assert status(f, c, k[:, :1], v[:, :1], t, lens) == SHAPE
    assert status(f, c, k, v[:1], t, lens) == SHAPE
    assert status(f, c, k, v, t, lens, cos=torch.zeros(9, 32)) == NULL
    assert status(f, c, k, v, t, lens, cos=torch.zeros(9, 32), sin=torch.zeros(8, 32)) == SHAPE
    assert status(f, c, k, v, t, lens, cos=torch.zeros(9, 32).half(), sin=torch.zeros(9, 32).half()) == DTYPE
    assert status(f, c, k, v, t, lens, cos=torch.zeros(32, 9).t(), sin=torch.zeros(32, 9).t()) == LAYOUT
    assert status(f, c, k, v, t, lens, q_out=q) == NULL
    assert status(f, c, k, v, t, lens, q=q[:1]) == SHAPE
    assert status(f, c, k, v, t, lens, q=q, q_out=q[:, :1]) == SHAPE
    # host tensors never reach a kernel
    assert status(f, c, k, v, t, lens) == ARG


def test_forward_arguments():
    c = cache()
    t, lens = batch()
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    f = sdpa.sdpa_paged_forward
    assert status(f, q.half(), c, t, lens) == DTYPE
    assert status(f, q.float(), c, t, lens) == DTYPE
    assert status(f, q[:, :3], c, t, lens) == SHAPE
    assert status(f, q[..., :32], c, t, lens) == SHAPE
    assert status(f, torch.zeros(3, 4, 64, dtype=torch.bfloat16), c, t, lens) == SHAPE
    assert status(f, q, c, t, lens, torch.zeros(3, dtype=torch.int32)) == NULL
    assert status(f, q, c, t, lens, out=q[:1]) == SHAPE
    assert status(f, q, c, t, lens, lse=torch.zeros(2, 3)) == SHAPE
    assert status(f, q, c, t, lens) == ARG


def test_forward_of_nothing():
    """Extents below one are a wrong shape, not a device without a workspace size."""
    c = cache()
    t, lens = batch()
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    cu = torch.zeros(3, dtype=torch.int32)
    f = sdpa.sdpa_paged_forward
    assert status(f, q[:0], c, t, lens) == SHAPE
    assert status(f, q[:, :0], c, t, lens) == SHAPE
    assert status(f, q, c, t, lens, cu, 0) == SHAPE
    assert status(f, q, c, t, lens, cu, -1) == SHAPE
    assert status(f, q, c, t[:, :0], lens) == SHAPE
    assert status(f, q, c, t[:0], lens[:0]) == SHAPE
    assert status(f, q, c, t[:0], lens[:0], cu[:1], 1) == SHAPE


class Raw:
    """The C entry points with made-up addresses far apart: every call here is refused before
    any of them is used."""

    def __init__(self, lib):
        self.lib = lib
        self.a = {n: (i + 1) << 40 for i, n in enumerate(
            ("k", "v", "ks", "vs", "kn", "vn", "q", "qo", "table", "lens", "cu", "cos", "sin", "out", "lse", "work"))}

    def struct(self, **kw):
        d = dict(k=self.a["k"], v=self.a["v"], k_scale=None, v_scale=None, n_pages=4, page_size=16, n_kv_heads=2,
                 head_dim=64, k_stride=(2048, 128, 64), v_stride=(2048, 128, 64), elem=0)
        d.update(kw)
        return sdpa._PagedCacheStruct(*[(ctypes.c_int64 * 3)(*x) if isinstance(x, tuple) else x for x in d.values()])

    @staticmethod
    def two(x):
        return (ctypes.c_int64 * 2)(*x) if x is not None else None

    def append(self, cache=None, **kw):
        a = self.a
        d = dict(k=a["kn"], v=a["vn"], dtype=0, total=6, k_stride=(128, 64), v_stride=(128, 64), table=a["table"], table_st=3,
                 max_pages=3, lens=a["lens"], cu=a["cu"], n_seqs=2, cos=a["cos"], sin=a["sin"], n_pos=48, rot=64, inter=0,
                 q=a["q"], qo=a["qo"], heads=4, q_stride=(256, 64), qo_stride=(256, 64))
        d.update(kw)
        return self.lib.sdpa_cache_append(
            ctypes.byref(cache or self.struct()), d["k"], d["v"], d["dtype"], d["total"], self.two(d["k_stride"]),
            self.two(d["v_stride"]), d["table"], d["table_st"], d["max_pages"], d["lens"], d["cu"], d["n_seqs"], d["cos"],
            d["sin"], d["n_pos"], d["rot"], d["inter"], d["q"], d["qo"], d["heads"], self.two(d["q_stride"]),
            self.two(d["qo_stride"]), None)

    def forward(self, cache=None, **kw):
        a = self.a
        d = dict(q=a["q"], out=a["out"], lse=a["lse"], dtype=0, total=6, heads=4, q_stride=(256, 64), o_stride=(256, 64),
                 lse_stride=(4, 1), table=a["table"], table_st=3, max_pages=3, lens=a["lens"], cu=a["cu"], n_seqs=2, max_q=4,
                 causal=1, scale=float("nan"), work=a["work"], size=0)
        d.update(kw)
        return self.lib.sdpa_paged_forward(
            d["q"], d["out"], d["lse"], d["dtype"], ctypes.byref(cache or self.struct()), d["total"], d["heads"],
            self.two(d["q_stride"]), self.two(d["o_stride"]), self.two(d["lse_stride"]), d["table"], d["table_st"],
            d["max_pages"], d["lens"], d["cu"], d["n_seqs"], d["max_q"], d["causal"], d["scale"], d["work"], d["size"], None)


CACHES = [  # (fields, status)
    (dict(k=None), NULL), (dict(elem=1), DTYPE), (dict(elem=2), NULL), (dict(head_dim=32), SHAPE), (dict(page_size=8), SHAPE),
    (dict(page_size=48), SHAPE), (dict(page_size=2048), SHAPE), (dict(n_pages=0), SHAPE), (dict(n_kv_heads=0), SHAPE),
    (dict(k=(1 << 40) + 8), LAYOUT), (dict(k_stride=(2048, 128, 60)), LAYOUT), (dict(v_stride=(2048, 0, 64)), LAYOUT),
    (dict(v_stride=(-2048, 128, 64)), LAYOUT), (dict(k_stride=(1 << 38, 128, 64)), LAYOUT),
    (dict(elem=2, k_scale=3 << 40, v_scale=4 << 40, k_stride=(2048, 128, 72)), LAYOUT),
    (dict(elem=2, k_scale=(3 << 40) + 2, v_scale=4 << 40), LAYOUT),
]


@pytest.mark.parametrize("fields,want", CACHES)
def test_caches(lib, fields, want):
    r = Raw(lib)
    c = r.struct(**fields)
    assert r.append(c) == want and r.forward(c) == want


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), NULL), (dict(lens=None), NULL), (dict(table=None), NULL), (dict(sin=None), NULL), (dict(qo=None), NULL),
    (dict(q_stride=None), NULL), (dict(dtype=1), DTYPE), (dict(dtype=5), DTYPE), (dict(total=0), SHAPE), (dict(n_seqs=0), SHAPE),
    (dict(cu=None, n_seqs=4), SHAPE), (dict(max_pages=0), SHAPE), (dict(max_pages=1 << 31), SHAPE), (dict(rot=4), SHAPE),
    (dict(rot=72), SHAPE), (dict(rot=12), SHAPE), (dict(n_pos=0), SHAPE), (dict(heads=0), SHAPE), (dict(total=1 << 31), SHAPE),
    (dict(k=(5 << 40) + 2), LAYOUT), (dict(k_stride=(100, 64)), LAYOUT), (dict(q_stride=(256, -64)), LAYOUT),
    (dict(table_st=2), LAYOUT), (dict(cos=(12 << 40) + 4), LAYOUT), (dict(lens=(10 << 40) + 1), LAYOUT),
    (dict(k=1 << 40), ARG), (dict(q=2 << 40), ARG), (dict(qo=5 << 40), ARG), (dict(qo=(7 << 40) + 16), ARG),
    (dict(qo=9 << 40), ARG), (dict(qo=7 << 40, qo_stride=(512, 64)), ARG),
])
def test_append_c_arguments(lib, kw, want):
    assert Raw(lib).append(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), NULL), (dict(out=None), NULL), (dict(work=None), NULL), (dict(lens=None), NULL), (dict(lse_stride=None), NULL),
    (dict(dtype=1), DTYPE), (dict(heads=3), SHAPE), (dict(heads=0), SHAPE), (dict(max_q=0), SHAPE), (dict(total=0), SHAPE),
    (dict(cu=None, n_seqs=4), SHAPE), (dict(total=1 << 31), SHAPE), (dict(max_pages=(1 << 27) - 1, table_st=1 << 27), SHAPE),
    (dict(q_stride=(256, 60)), LAYOUT), (dict(out=(14 << 40) + 8), LAYOUT), (dict(work=(16 << 40) + 4), LAYOUT),
    (dict(lse_stride=(0, 1)), LAYOUT), (dict(scale=float("inf")), ARG), (dict(out=7 << 40), ARG), (dict(out=1 << 40), ARG),
    (dict(lse=14 << 40), ARG), (dict(work=7 << 40, size=64), ARG), (dict(out=11 << 40), ARG),
])
def test_forward_c_arguments(lib, kw, want):
    assert Raw(lib).forward(**kw) == want


def test_workspace_sizes(lib):
    w = lib.sdpa_paged_workspace_bytes
    assert w(96, 8, 2, 1) == 0 and w(64, 7, 2, 1) == 0 and w(64, 8, 0, 1) == 0 and w(64, 8, 2, 0) == 0
    if not torch.cuda.is_available():
        assert w(64, 8, 2, 1) == 0
