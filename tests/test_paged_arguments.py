"""Arguments of the paged cache's binding at the edges of what it takes."""
import pytest
import torch

import scaled_dot_product_forward_gb300 as sdpa
from tests.test_paged import make_cache, tables
from tests.test_paged_refusals import cache, status

SHAPE, DTYPE, LAYOUT, ARG = 3, 4, 5, 6
gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    from scaled_dot_product_forward_gb300 import _build
    _build.build()
    return sdpa.load_library()


def one_column(n):
    """[n, 1] page tables, the second stride of each being another."""
    t = torch.zeros(n, dtype=torch.int32)
    return [t[:, None], t[None].t(), t.as_strided((n, 1), (1, 7)), torch.zeros(n, 4, dtype=torch.int32)[:, 1:2]]


def test_a_page_table_of_one_column(lib):
    """Its second stride means nothing.  (Host tensors come as far as the check of the device.)"""
    c, lens = cache(), torch.ones(3, dtype=torch.int32)
    q, k = (torch.zeros(3, n, 64, dtype=torch.bfloat16) for n in (4, 2))
    for t in one_column(3):
        assert status(sdpa.sdpa_cache_append, c, k, k.clone(), t, lens) == ARG
        assert status(sdpa.sdpa_paged_forward, q, c, t, lens) == ARG
    two = torch.zeros(2, 3, dtype=torch.int32).t()
    assert status(sdpa.sdpa_cache_append, c, k, k.clone(), two, lens) == LAYOUT
    assert status(sdpa.sdpa_paged_forward, q, c, two, lens) == LAYOUT


@gpu
def test_a_page_table_of_one_column_on_the_device(sdpa_lib):
    c = make_cache(sdpa_lib, 9, 32, 2, 64, "e4m3", torch.bfloat16, 3)
    q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    lens = torch.tensor([3, 32, 17], dtype=torch.int32, device="cuda")
    t = tables(3, 1, 9, 2).cuda()
    want = sdpa_lib.sdpa_paged_forward(q, c, t, lens)
    got = sdpa_lib.sdpa_paged_forward(q, c, t.view(1, 3).t(), lens)
    assert torch.equal(got, want)
    wide = torch.full((3, 5), -1, dtype=torch.int32, device="cuda")
    wide[:, 2] = t[:, 0]
    assert torch.equal(sdpa_lib.sdpa_paged_forward(q, c, wide.as_strided((3, 1), (5, 3), 2), lens), want)


def test_ranks(lib):
    """A wrong number of dimensions is a wrong shape, also where there is none."""
    c, lens, t = cache(), torch.ones(2, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32)
    k, v, q = (torch.zeros(2, n, 64, dtype=torch.bfloat16) for n in (2, 2, 4))
    angles = torch.zeros(9, 32)
    f = sdpa.sdpa_cache_append
    for x in (k[0, 0, 0], k[0, 0], k[0], k[None]):
        assert status(f, c, x, x, t, lens) == SHAPE
        assert status(f, c, k, x, t, lens) == SHAPE
        assert status(f, c, k, v, t, lens, q=x) == SHAPE
        assert status(f, c, k, v, t, lens, q=q, q_out=x) == SHAPE
        assert status(sdpa.sdpa_paged_forward, x, c, t, lens) == SHAPE
        assert status(sdpa.sdpa_paged_forward, q, c, t, lens, out=x) == SHAPE
    for x in (angles[0, 0], angles[0], angles[None]):
        assert status(f, c, k, v, t, lens, cos=x, sin=x) == SHAPE
        assert status(f, c, k, v, t, lens, cos=angles, sin=x) == SHAPE
        assert status(sdpa.sdpa_paged_forward, q, c, t, lens, lse=x) == SHAPE
    for x in (t[0], t[None], t[0, 0]):
        assert status(f, c, k, v, x, lens) == SHAPE
    for x in (lens[0], lens[None]):
        assert status(f, c, k, v, t, x) == SHAPE
        assert status(f, c, k, v, t, lens, x) == SHAPE


@gpu
@pytest.mark.parametrize("rows", [1, 30])
def test_any_bound_on_the_rows(sdpa_lib, rows):
    """max_seqlen_q is an upper bound: however large, it gives the results."""
    c = make_cache(sdpa_lib, 9, 32, 2, 64, "e4m3", torch.bfloat16, 3)
    q = torch.randn(2 * rows, 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    lens = torch.tensor([40, 96], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, rows, 2 * rows], dtype=torch.int32, device="cuda")
    t = tables(2, 3, 9, 2).cuda()
    want = sdpa_lib.sdpa_paged_forward(q, c, t, lens, cu, 2 * rows, is_causal=True)
    for most in (10 ** 6, 2 ** 31 - 1, 2 ** 31, 2 ** 40):
        assert torch.equal(sdpa_lib.sdpa_paged_forward(q, c, t, lens, cu, most, is_causal=True), want)
