"""A sequence that goes on after its tokens were compacted: its new tokens keep the positions that they have in the text,
which are no longer the places that they take in the cache."""
import pytest
import torch

from tests import paged_ref as ref
from tests.test_norm_rotate import angles, rounded, turned, weights
from tests.test_paged import check, make_cache

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("norms", [True, False])
@pytest.mark.parametrize("kind,D", [("16", 64), ("e4m3", 64), ("16", 128), ("e4m3", 128)])
def test_tokens_after_a_compaction(sdpa_lib, kind, D, norms):
    """New tokens are rotated by sdpa_norm_rotate with their positions and appended as they are.  Their cached keys are
    the formula's at those positions (16-bit: those that an append into the whole sequence writes, bit for bit), the kept
    keys stay, and the answers are attention over the kept and the new ones."""
    H, hkv, P, dtype, eps = 8, 2, 16, torch.bfloat16, 1e-5
    g = torch.Generator().manual_seed(5)
    length, steps, rot = 90, 21, D // 2
    keep = [0, 1, 2, 3] + list(range(47, length, 3))
    cos, sin = angles(length + steps, rot)
    w = weights(D, 3) if norms else None
    kw = dict(cos=cos.cuda(), sin=sin.cuda(), q_norm=w.cuda() if norms else None, k_norm=w.cuda() if norms else None, eps=eps)
    cache = make_cache(sdpa_lib, 20, P, hkv, D, kind, dtype, 4)
    whole, table = i32([[17, 3, 9, 4, 11, 0, 13]]), i32([[2, 19, 7, 8]])

    def tokens(n):
        return [torch.randn(n, h, D, generator=g).to(dtype) for h in (H, hkv, hkv)]

    q, k, v = tokens(length)
    sdpa_lib.sdpa_cache_append(cache, k.cuda(), v.cuda(), whole, i32([length]), q=q.cuda(), **kw)
    sdpa_lib.sdpa_cache_compact(cache, whole, i32([keep]), table)
    lens, n = i32([len(keep)]), len(keep)
    table_rows = table[0].tolist()
    for i in range(steps):
        pos = length + i
        q, k, v = tokens(1)
        held = ref.values(cache.k, cache.k_scale)
        rq, rk = sdpa_lib.sdpa_norm_rotate(q.cuda(), k.cuda(), i32([pos]), **kw)
        lens += 1
        n += 1
        sdpa_lib.sdpa_cache_append(cache, rk, v.cuda(), table, lens)
        out = sdpa_lib.sdpa_paged_forward(rq, cache, table, lens, is_causal=True)
        kk, vv = ref.values(cache.k, cache.k_scale), ref.values(cache.v, cache.v_scale)
        page, row = table_rows[(n - 1) // P], (n - 1) % P
        # the new key, by the formula at its position in the text
        y, lost = turned(k, w, eps, torch.tensor([pos]), cos, sin, False)
        tol = rounded(y, lost, dtype)
        if kind == "e4m3":      # and a rounding to the code: half a step, of the least normal's binade at least
            tol = tol + 2.0 ** -4 * (y.abs() + tol) + 2.0 ** -10 * cache.k_scale[page].cpu().double()[:, None]
        check(kk[page, row][None], y, tol, f"key {pos}")
        if kind == "16":
            sdpa_lib.sdpa_cache_append(cache, k.cuda(), v.cuda(), whole, i32([pos + 1]), q=q.cuda(), **kw)
            assert torch.equal(cache.k[int(whole[0, pos // P]), pos % P], cache.k[page, row])
            # the others are as they were
            old = [(table_rows[j // P], j % P) for j in range(n - 1)]
            assert all(torch.equal(kk[a], held[a]) for a in old)
        want = ref.attend(rq, kk, vv, table.cpu(), [n], [1], causal=True)
        tol, _ = ref.attend_bounds(want, n, D, dtype, torch.bfloat16 if kind == "16" else torch.float16)
        check(out, want[0], tol, f"answer {pos}")
