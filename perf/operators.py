"""The operators of a served model's key/value cache, as cases to be measured.

``append``: the keys and values of new tokens, rotated by their positions, go into a paged cache; the tokens'
queries are rotated in the same call.  ``attend``: the queries of 1 .. n new tokens of each sequence attend to
that sequence's pages.  The cache holds 16-bit values, or 8-bit ones (e4m3) with a power-of-two scale for each
page and head.  With ``own`` false both run in their plain form (elementary torch operations in 32 bits)."""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn
DEV = "cuda"
MIN_EXP, MAX_EXP = -50, 50   # range of the exponents of a page's scale


def listed():
    a = dict(op="attend", batch=1, q_len=1, kv_len=1000, ragged=False, heads=32, kv_heads=8, dim=128, page=16,
             cache="e4m3", dtype="bf16", causal=True, lse=False)
    w = dict(op="append", batch=64, new_len=1, kv_len=512, ragged=True, heads=32, kv_heads=8, dim=128, page=16,
             cache="e4m3", dtype="bf16", rot=128, interleaved=False)
    return [
        # one user's next token, a short conversation: latency
        dict(a, name="attend one sequence"),
        # a serving batch at ordinary, uneven lengths
        dict(a, name="attend batch of 64", batch=64, kv_len=4096, ragged=True, page=64),
        # a batch over very long contexts: two gigabytes of cache
        dict(a, name="attend long contexts", batch=8, kv_len=131072, page=64),
        # one query head a key/value head, small heads, 16-bit cache
        dict(a, name="attend 16-bit, 64-wide heads", batch=32, kv_len=2048, ragged=True, heads=16, kv_heads=16,
             dim=64, cache="16", dtype="fp16", lse=True),
        # several proposed tokens a sequence checked in one pass
        dict(a, name="attend five proposed tokens", batch=16, q_len=5, kv_len=16384, ragged=True, heads=64, page=32,
             lse=True),
        # all query heads on one key/value head
        dict(a, name="attend one shared head", batch=32, kv_len=8191, ragged=True, heads=64, kv_heads=1, page=128,
             dtype="fp16"),
        # a chunk of a long prompt behind what was read of it before
        dict(a, name="attend chunk of a prompt", q_len=2048, kv_len=16384, page=64),
        # prompts of many users at once, uneven, 16-bit cache
        dict(a, name="attend uneven prompts", batch=16, q_len=1024, kv_len=4096, ragged=True, cache="16"),
        # the cache's side of one decoding step
        dict(w, name="append one token each"),
        # a prompt's chunk for a few users
        dict(w, name="append prompts", batch=4, new_len=2048, kv_len=2500, ragged=True, page=64),
        # small heads, part of them rotated, neighbouring pairs, 16-bit cache
        dict(w, name="append 16-bit, part rotated", batch=24, new_len=333, kv_len=1000, heads=16, kv_heads=16,
             dim=64, cache="16", dtype="fp16", rot=32, interleaved=True, page=32),
        # many long prompts
        dict(w, name="append long prompts", batch=8, new_len=8192, kv_len=8192, ragged=False, page=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    heads = kv_heads * rng.choice([1, 2, 4, 8] if kv_heads > 4 else [1, 4, 7, 8, 16])
    c = dict(op=rng.choice(["attend", "attend", "append"]), ragged=rng.random() < 0.7, heads=heads, kv_heads=kv_heads, dim=dim,
             page=rng.choice([16, 32, 64, 128]), cache=rng.choice(["e4m3", "e4m3", "16"]), dtype=rng.choice(["bf16", "fp16"]))
    if c["op"] == "attend":
        c["q_len"] = rng.choice([1, 1, 1, rng.randint(2, 9), _log(rng, 10, 2048)])
        c["kv_len"] = max(c["q_len"], _log(rng, 1, 131072))
        c["batch"] = _log(rng, 1, 64)
        # the plain form's scores, the cache and the products stay below the listed cases' largest
        while c["batch"] > 1 and (c["batch"] * c["heads"] * c["q_len"] * c["kv_len"] > 1 << 30 or
                                  c["batch"] * c["kv_len"] * kv_heads * dim > 1 << 29):
            c["batch"] //= 2
        while c["heads"] * c["q_len"] * c["kv_len"] > 1 << 30:
            c["kv_len"] = max(1, c["kv_len"] // 2)
            c["q_len"] = min(c["q_len"], c["kv_len"])
        c["causal"], c["lse"] = rng.random() < 0.8, rng.random() < 0.5
    else:
        c["new_len"] = rng.choice([1, 1, rng.randint(2, 40), _log(rng, 41, 8192)])
        c["kv_len"] = c["new_len"] + rng.choice([0, rng.randint(1, 600)])
        c["batch"] = _log(rng, 1, 64)
        while c["batch"] > 1 and c["batch"] * c["new_len"] * (heads + 2 * kv_heads) * dim > 1 << 28:
            c["batch"] //= 2
        c["rot"] = rng.choice([dim, dim, dim // 2])
        c["interleaved"] = rng.random() < 0.3
    return c


def _lengths(case, seed):
    """New tokens of each sequence (the case's), and its cached tokens with the new ones (the seed's), on the host."""
    h, g = torch.Generator().manual_seed(17), torch.Generator().manual_seed(seed * 7919 + 17)
    B, n, kv = case["batch"], case.get("q_len", case.get("new_len")), case["kv_len"]
    if not case["ragged"]:
        return [n] * B, [kv] * B
    new = [int(x) for x in torch.randint((n + 1) // 2, n + 1, (B,), generator=h)]
    lens = [int(torch.randint(max(x, (kv + 3) // 4), kv + 1, (1,), generator=g)) for x in new]
    new[0], lens[-1] = n, max(kv, new[-1])
    lens[0] = max(lens[0], n)
    return new, lens


def _quantise(x):
    """x [pages, tokens, heads, D] as e4m3 with the least power-of-two scale a page and head under which it fits."""
    m, e = torch.frexp(x.abs().amax(dim=(1, 3)))
    e = torch.where(m > 0.875, e - 8, e - 9).masked_fill(m == 0, MIN_EXP).clamp(MIN_EXP, MAX_EXP)
    scale = torch.ldexp(torch.ones_like(m), e)
    return (x / scale[:, None, :, None]).clamp(-448, 448).to(E4M3), scale


def prepare(case, seed):
    new, lens = _lengths(case, seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    B, P, H, Hkv, D = case["batch"], case["page"], case["heads"], case["kv_heads"], case["dim"]
    dtype = TYPES[case["dtype"]]
    per_seq = -(-case["kv_len"] // P)
    n_pages = B * per_seq + 3
    s = dict(case=case, max_new=max(new), max_len=max(lens))
    perm = torch.randperm(n_pages, generator=g, device=DEV)[:B * per_seq]
    s["table"] = perm.view(B, per_seq).to(torch.int32).contiguous()   # pages as a serving program's pool hands them out
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    total = cu[-1]

    def normal(*shape, spread=1.0):
        return torch.randn(*shape, generator=g, device=DEV) * spread

    # keys carry a few channels far larger than the rest, values do not; the pool's pages are all in use
    loud = torch.ones(D, device=DEV)
    loud[:: D // 4] = 4.0
    for name, spread in (("k", loud), ("v", 0.5)):
        parts, scales = [], []
        for p0 in range(0, n_pages, max(1, (1 << 28) // (P * Hkv * D))):
            p1 = min(n_pages, p0 + max(1, (1 << 28) // (P * Hkv * D)))
            x = normal(p1 - p0, P, Hkv, D, spread=spread)
            if case["cache"] == "e4m3":
                x, scale = _quantise(x)
                scales.append(scale)
            else:
                x = x.to(dtype)
            parts.append(x)
        s["cache_" + name] = torch.cat(parts) if len(parts) > 1 else parts[0]
        s["scale_" + name] = torch.cat(scales) if scales else None
    s["q"] = normal(total, H, D).to(dtype)
    if case["op"] == "append":
        s["k"] = normal(total, Hkv, D, spread=loud).to(dtype)
        s["v"] = normal(total, Hkv, D, spread=0.5).to(dtype)
        half = case["rot"] // 2
        angle = torch.arange(per_seq * P, device=DEV, dtype=torch.float64)[:, None] * torch.pow(
            10000.0, -torch.arange(half, device=DEV, dtype=torch.float64) / half)
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    if own:
        import scaled_dot_product_forward_gb300 as sdpa
        s["sdpa"] = sdpa
        s["handle"] = sdpa.SdpaPagedCache(s["cache_k"], s["cache_v"], s["scale_k"], s["scale_v"])
    return s


def run(s):
    return _attend(s) if s["case"]["op"] == "attend" else _append(s)


def _token_places(s):
    """Sequence and index within its new tokens of each token, and each token's position."""
    cu, lens = s["cu"].long(), s["lens"].long()
    t = torch.arange(s["q"].shape[0], device=DEV)
    b = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[b]
    return b, i, lens[b] - (cu[b + 1] - cu[b]) + i


def _pages(s, name):
    """The sequences' pages as [B, tokens, Hkv, D] in 32 bits."""
    cache, scale, table = s["cache_" + name], s["scale_" + name], s["table"].long()
    if scale is None:
        x = cache[table].float()
    else:
        x = cache.view(torch.uint8)[table].view(E4M3).float() * scale[table][:, :, None, :, None]
    return x.flatten(1, 2)


def _attend(s):
    case = s["case"]
    if own:
        return s["sdpa"].sdpa_paged_forward(s["q"], s["handle"], s["table"], s["lens"], s["cu"], s["max_new"],
                                            is_causal=case["causal"], return_lse=case["lse"])
    B, H, Hkv, D = case["batch"], case["heads"], case["kv_heads"], case["dim"]
    n, G = s["max_new"], H // Hkv
    b, i, _ = _token_places(s)
    lens, count = s["lens"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    q = torch.zeros(B, n, H, D, device=DEV)
    q[b, i] = s["q"].float()
    q = q.view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    k = _pages(s, "k")
    j = torch.arange(k.shape[1], device=DEV)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)).view(B, Hkv, G, n, -1) * (1.0 / math.sqrt(D))
    del k
    seen = (j[None, :] < lens[:, None])[:, None, :]
    if case["causal"]:
        last = (lens - count)[:, None] + torch.arange(n, device=DEV)[None, :]
        seen = seen & (j[None, None, :] <= last[:, :, None])
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    scores.sub_(top).exp_()
    total = scores.sum(-1, keepdim=True)
    v = _pages(s, "v")
    v = torch.where((j[None, :] < lens[:, None])[:, :, None, None], v, torch.zeros_like(v))
    out = torch.matmul(scores.view(B, Hkv, G * n, -1), v.permute(0, 2, 1, 3)).view(B, Hkv, G, n, D)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    out = out.permute(0, 3, 1, 2, 4).reshape(B, n, H, D)[b, i].to(s["q"].dtype)
    if not case["lse"]:
        return out
    lse = (total.log() + top).permute(0, 3, 1, 2, 4).reshape(B, n, H)[b, i]
    return out, lse


def _rotate(x, cos, sin, interleaved):
    """x [tokens, heads, D] in 32 bits; cos, sin [tokens, pairs]: pair j of a head is turned by its angle."""
    c, s, half = cos[:, None, :], sin[:, None, :], cos.shape[1]
    y = x.clone()
    a = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    b = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def _append(s):
    case = s["case"]
    if own:
        q = s["sdpa"].sdpa_cache_append(s["handle"], s["k"], s["v"], s["table"], s["lens"], s["cu"], cos=s["cos"], sin=s["sin"],
                                        interleaved=case["interleaved"], q=s["q"])
        return _state(s, q)
    P = case["page"]
    b, i, pos = _token_places(s)
    page, row = s["table"].long()[b, pos // P], pos % P
    cos, sin = s["cos"][pos], s["sin"][pos]
    q = _rotate(s["q"].float(), cos, sin, case["interleaved"]).to(s["q"].dtype)
    k = _rotate(s["k"].float(), cos, sin, case["interleaved"])
    for name, x in (("k", k), ("v", s["v"].float())):
        cache, scale = s["cache_" + name], s["scale_" + name]
        if scale is None:
            cache[page, row] = x.to(cache.dtype)
            continue
        first = (row == 0) | (i == 0)     # the first new token of each page
        p, begin = page[first], row[first]
        most = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax")[p]
        m, e = torch.frexp(most)
        e = torch.where(m > 0.875, e - 8, e - 9).masked_fill(m == 0, MIN_EXP).clamp(MIN_EXP, MAX_EXP)
        need = torch.ldexp(torch.ones_like(m), e)
        old = torch.where((begin > 0)[:, None], scale[p], need)
        now = torch.maximum(old, need)
        scale[p] = now
        codes = cache.view(torch.uint8)
        held = codes[p].view(E4M3).float()
        kept = (torch.arange(P, device=DEV)[None, :] < begin[:, None])[:, :, None, None]
        held = torch.where(kept, held * (old / now)[:, None, :, None], held)
        codes[p] = held.to(E4M3).view(torch.uint8)
        codes[page, row] = (x / scale[page][:, :, None]).clamp(-448, 448).to(E4M3).view(torch.uint8)
    return _state(s, q)


def _state(s, q):
    return {"q": q, "k": s["cache_k"], "v": s["cache_v"], "k_scale": s["scale_k"], "v_scale": s["scale_v"]}


def exact(case, seed):
    s = prepare(case, seed)
    new, lens = _lengths(case, seed)
    P, H, Hkv, D = case["page"], case["heads"], case["kv_heads"], case["dim"]
    start = [sum(new[:b]) for b in range(len(new))]
    if case["op"] == "attend":
        out = torch.zeros(sum(new), H, D, dtype=torch.float64, device=DEV)
        lse = torch.full((sum(new), H), -math.inf, dtype=torch.float64, device=DEV)
        for b, (n, L) in enumerate(zip(new, lens)):
            pages = s["table"][b, :-(-L // P)].long()
            rows = slice(start[b], start[b] + n)
            for h in range(Hkv):
                kv = []
                for name in ("k", "v"):
                    x = s["cache_" + name][:, :, h].view(torch.uint8 if case["cache"] == "e4m3" else torch.int16)[pages]
                    x = x.view(s["cache_" + name].dtype).double()
                    if case["cache"] == "e4m3":
                        x = x * s["scale_" + name][pages, h].double()[:, None, None]
                    kv.append(x.flatten(0, 1)[:L])
                for g in range(h * (H // Hkv), (h + 1) * (H // Hkv)):
                    z = s["q"][rows, g].double() @ kv[0].T / math.sqrt(D)
                    if case["causal"]:
                        z = z.masked_fill(torch.ones_like(z, dtype=torch.bool).triu(L - n + 1), -math.inf)
                    lse[rows, g] = torch.logsumexp(z, -1)
                    out[rows, g] = torch.softmax(z, -1) @ kv[1]
        return (out, lse) if case["lse"] else out
    half = case["rot"] // 2
    at = torch.cat([torch.arange(L - n, L, device=DEV) for n, L in zip(new, lens)])
    turn = torch.complex(s["cos"].double(), s["sin"].double())[at][:, None]

    def turned(x):
        x = x.double()
        r, rest = x[..., :2 * half], x[..., 2 * half:]
        pairs = r.unflatten(-1, (half, 2)) if case["interleaved"] else r.unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        r = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([r, rest], -1)

    got = {"q": turned(s["q"]), "k_scale": None, "v_scale": None}
    for name, x in (("k", turned(s["k"])), ("v", s["v"].double())):
        held = s["cache_" + name].double()
        scale = None if s["scale_" + name] is None else s["scale_" + name].double()
        for b, (n, L) in enumerate(zip(new, lens)):
            done = L - n
            while done < L:
                page, row = int(s["table"][b, done // P]), done % P
                count = min(L - done, P - row)
                first = start[b] + done - (L - n)
                y = x[first:first + count]
                if scale is not None:
                    need = torch.exp2(torch.ceil(torch.log2(y.abs().amax(dim=(0, 2)) / 448)).clamp(MIN_EXP, MAX_EXP))
                    if row:
                        now = torch.maximum(need, scale[page])
                        held[page, :row] *= (scale[page] / now)[:, None]
                    else:
                        now = need
                    scale[page] = now
                    y = y / now[:, None]
                held[page, row:row + count] = y
                done += count
        got[name] = held
        got[name + "_scale"] = scale
    return got


def work(case):
    if not case["ragged"]:
        return _work(case, 0)
    each = [_work(case, seed) for seed in range(16)]     # lengths differ from seed to seed
    return {key: sum(w[key] for w in each) / len(each) for key in each[0]}


def _work(case, seed):
    new, lens = _lengths(case, seed)
    H, Hkv, D = case["heads"], case["kv_heads"], case["dim"]
    wide = 1 if case["cache"] == "e4m3" else 2
    P = case["page"]
    if case["op"] == "attend":
        pages = sum(-(-L // P) for L in lens)
        moved = 2 * sum(lens) * Hkv * D * wide + 4 * pages + 2 * 2 * sum(new) * H * D
        moved += 8 * pages * Hkv if wide == 1 else 0
        moved += 4 * sum(new) * H if case["lse"] else 0
        pairs = sum(n * L - (n * (n - 1) // 2 if case["causal"] else 0) for n, L in zip(new, lens))
        return {"bytes": moved, "flops": 4.0 * H * D * pairs}
    total = sum(new)
    pages = sum((L - 1) // P - (L - n) // P + 1 for n, L in zip(new, lens))
    places = len({p for n, L in zip(new, lens) for p in range(L - n, L)})
    moved = 2 * total * Hkv * D * (2 + wide) + 2 * 2 * total * H * D + 4 * case["rot"] * places + 4 * pages
    moved += 16 * pages * Hkv if wide == 1 else 0
    return {"bytes": moved, "flops": 6.0 * total * (H + Hkv) * case["rot"] / 2}
