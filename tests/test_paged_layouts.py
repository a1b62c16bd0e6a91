"""Operands of the paged cache's operators that share a buffer: taken where no
element is shared, refused where one is."""
import pytest
import torch

import scaled_dot_product_forward_gb300 as sdpa
from tests.test_paged import make_cache, run_attend, tables
from tests.test_paged_refusals import Raw

ARG = 6
NO_DEVICE = (7, 9)     # what a call without a GPU comes to once its arguments are taken
gpu = pytest.mark.gpu
# (made-up addresses: only where no kernel can be launched)
cpu = pytest.mark.skipif(torch.cuda.is_available(), reason="has a GPU")
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    from scaled_dot_product_forward_gb300 import _build
    _build.build()
    return sdpa.load_library()


B = 5 << 40            # a buffer of its own
# queries, keys and values (4 heads, 6 tokens, D 64) of one buffer, as (offset, token stride, head stride) in elements
SHARED = {
    "side by side": ((0, 768, 64), (256, 768, 64), (512, 768, 64)),
    "by head": ((0, 768, 192), (64, 768, 192), (128, 768, 192)),
    "heads first": ((0, 64, 384), (1536, 64, 384), (3072, 64, 384)),
    "heads first, by token": ((0, 192, 1152), (64, 192, 1152), (128, 192, 1152)),
}
# an output (tokens 6, heads 4) that meets queries at (0, 768, 192)
MEETS = [(0, 768, 64), (8, 768, 192), (56, 768, 192), (768, 768, 192), (1536 + 192, 768, 192), (720, 768, 192), (0, 192, 1152)]


def at(x):
    return B + 2 * x[0]


@cpu
@pytest.mark.parametrize("total", [6, 1])
@pytest.mark.parametrize("kind", SHARED)
def test_operands_of_one_buffer_are_taken(lib, kind, total):
    q, k, v = SHARED[kind]
    r = Raw(lib)
    c = r.struct(n_kv_heads=4, k_stride=(4096, 256, 64), v_stride=(4096, 256, 64))
    kw = dict(total=total, cu=r.a["cu"], n_seqs=1, k=at(k), v=at(v), k_stride=k[1:], v_stride=v[1:])
    assert r.append(c, q=at(q), qo=at(q), q_stride=q[1:], qo_stride=q[1:], **kw) in NO_DEVICE
    # queries elsewhere, the rotated ones into the buffer
    assert r.append(c, q=r.a["q"], qo=at(q), q_stride=(256, 64), qo_stride=q[1:], **kw) in NO_DEVICE
    assert r.append(c, q=r.a["q"], qo=at(k), q_stride=(256, 64), qo_stride=k[1:], **kw) == ARG
    kw = dict(total=total, n_seqs=1, size=1 << 40)
    assert r.forward(c, q=at(q), q_stride=q[1:], out=at(k), o_stride=k[1:], **kw) in NO_DEVICE
    assert r.forward(c, q=at(q), q_stride=q[1:], out=at(q), o_stride=q[1:], **kw) == ARG


@cpu
@pytest.mark.parametrize("out", MEETS)
def test_operands_that_share_elements_are_refused(lib, out):
    r = Raw(lib)
    kw = dict(q=B, q_stride=(768, 192), size=1 << 40)
    assert r.forward(out=at(out), o_stride=out[1:], **kw) == ARG
    assert r.append(q=B, q_stride=(768, 192), qo=at(out), qo_stride=out[1:]) == ARG


@cpu
@pytest.mark.parametrize("v", [0, 32, 2048, 2048 * 3, 2048 + 128])
def test_keys_pages_that_are_values_pages_are_not_appended_to(lib, v):
    """Both would be written; attention may read one tensor as both."""
    r = Raw(lib)
    c = r.struct(v=r.a["k"] + 2 * v)
    assert r.append(c) == ARG
    assert r.forward(c, size=1 << 40) in NO_DEVICE


@cpu
@pytest.mark.parametrize("v,strides", [(2048, (4096, 128, 64)), (128, (4096, 256, 64)), (64, (4096, 256, 128)), (8192, (2048, 128, 64)),
                                       (2048, (4096, 64, 1024)), (512, (4096, 64, 1024))])
def test_pages_of_one_pool_are_appended_to(lib, v, strides):
    """Keys' and values' pages, rows or heads in turn, or one after the other."""
    r = Raw(lib)
    c = r.struct(v=r.a["k"] + 2 * v, k_stride=strides, v_stride=strides)
    want = (ARG,) if (v, strides) == (512, (4096, 64, 1024)) else NO_DEVICE
    assert r.append(c) in want


@gpu
@pytest.mark.parametrize("rows", [1, 5, 40, 80])
@pytest.mark.parametrize("total_first", [True, False])
def test_queries_keys_and_values_by_head(sdpa_lib, rows, total_first):
    """[tokens, heads, 3, D] and [heads, tokens, 3, D] buffers: queries rotated in place beside the
    keys, keys and values appended, and the output written where the keys were; as with separate
    tensors, bit for bit."""
    H, D, P, n = 4, 128, 16, 2
    g = torch.Generator().manual_seed(rows)
    shape = (n * rows, H, 3, D) if total_first else (H, n * rows, 3, D)
    buf = torch.randn(shape, generator=g).bfloat16().cuda()
    q, k, v = ((buf if total_first else buf.transpose(0, 1))[:, :, i] for i in range(3))
    a = torch.rand(128, D // 2, generator=g) * 6
    cos, sin = a.cos().cuda(), a.sin().cuda()
    table = tables(n, 8, 17, 1)
    lens = torch.tensor([rows + 7, rows + 40], dtype=torch.int32, device="cuda")
    caches = [make_cache(sdpa_lib, 17, P, H, D, "e4m3", torch.bfloat16, 4) for _ in range(2)]
    apart = sdpa_lib.sdpa_cache_append(caches[0], k.clone(), v.clone(), table.cuda(), lens, cos=cos, sin=sin, q=q.clone())
    want = sdpa_lib.sdpa_paged_forward(apart, caches[0], table.cuda(), lens, is_causal=True)
    values = v.clone()
    got = sdpa_lib.sdpa_cache_append(caches[1], k, v, table.cuda(), lens, cos=cos, sin=sin, q=q, q_out=q)
    assert got is q and torch.equal(q, apart)
    for name in ("k", "v"):
        assert torch.equal(getattr(caches[0], name).view(torch.uint8), getattr(caches[1], name).view(torch.uint8))
    assert torch.equal(sdpa_lib.sdpa_paged_forward(q, caches[1], table.cuda(), lens, out=k, is_causal=True), want)
    assert torch.equal(k, want) and torch.equal(q, apart) and torch.equal(v, values)


@gpu
@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("dtype", [E4M3, torch.float16])
def test_one_tensor_as_keys_and_values(sdpa_lib, dtype, rows):
    """Attention reads it; it is not appended to."""
    k = torch.randn(10, 32, 1, 64, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    s = torch.full((10, 1), 0.5, device="cuda") if dtype is E4M3 else None
    c = sdpa_lib.SdpaPagedCache(k, k, s, s)
    q = torch.randn(rows, 4, 64, generator=torch.Generator().manual_seed(4)).half().cuda()
    run_attend(sdpa_lib, c, q, tables(1, 9, 10, 1), [270], [rows], True, use_cu=False)
    before = k.clone()
    with pytest.raises(sdpa.SdpaError) as e:
        sdpa_lib.sdpa_cache_append(c, q[:, :1], q[:, 1:2], tables(1, 9, 10, 1).cuda(),
                                   torch.tensor([270], dtype=torch.int32, device="cuda"))
    assert e.value.status == ARG
    torch.cuda.synchronize()
    assert torch.equal(k.view(torch.uint8), before.view(torch.uint8))
