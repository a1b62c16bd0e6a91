"""What a served model does with its paged key/value cache besides growing and reading all of it, as cases to be
measured.

``attend``: new tokens attend to a sliding window of their sequence and to its first few tokens.  ``norm``: query and
key heads are normalised and rotated in one pass, keys on their way into the cache, or both in rows of packed
documents.  ``fork``: sequences become copies of others, sharing their full pages and copying the begun one, and get
room for new tokens.  ``copy``: pages are copied.  ``compact``: the tokens of a sequence that are kept move together
into new pages.  With ``own`` false all run in their plain form (elementary torch operations in 32 bits)."""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn
DEV = "cuda"
EPS = 1e-6
MIN_EXP, MAX_EXP = -50, 50   # range of the exponents of a page's scale


def listed():
    a = dict(op="attend", batch=1, q_len=1, kv_len=5000, ragged=False, heads=32, kv_heads=8, dim=128, page=16,
             cache="e4m3", dtype="bf16", window=1024, sinks=4, released=False, lse=False)
    n = dict(op="norm", cached=True, batch=64, new_len=1, kv_len=512, ragged=True, heads=32, kv_heads=8, dim=128, page=16,
             cache="e4m3", dtype="bf16", rot=128, interleaved=False)
    f = dict(op="fork", groups=1, width=5, kv_len=1000, ragged=False, room=1, kv_heads=8, dim=128, page=16, spare=4096,
             cache="e4m3", dtype="bf16")
    c = dict(op="copy", pages=8, kv_heads=8, dim=128, page=16, cache="e4m3", dtype="bf16", partly=False)
    m = dict(op="compact", batch=32, kv_len=60, keep=0.4, kv_heads=8, dim=128, page=16, cache="e4m3", dtype="bf16")
    return [
        # one user's next token: latency
        dict(a, name="attend one sequence"),
        # a serving batch over long texts, whose pages behind the window have been given back
        dict(a, name="attend batch of 64", batch=64, kv_len=32768, ragged=True, window=4096, page=64, released=True),
        # a chunk of a long prompt behind what was read of it before
        dict(a, name="attend chunk of a prompt", q_len=4096, kv_len=16384, window=4096, page=64, released=True),
        # the cache's side of one decoding step
        dict(n, name="norm and append one token each"),
        # long prompts of a few users
        dict(n, name="norm and append prompts", batch=8, new_len=4096, kv_len=4096, ragged=False, page=64),
        # packed documents without a cache, small heads, neighbouring pairs, part of the head rotated
        dict(n, name="norm rows of documents", cached=False, batch=24, new_len=1000, kv_len=1000, heads=16, kv_heads=16, dim=64,
             dtype="fp16", rot=32, interleaved=True, cache="16"),
        # four samples of one prompt
        dict(f, name="fork samples of a prompt"),
        # one step of a beam search over many texts: of each text's four beams three become copies of the best
        dict(f, name="fork beams", groups=32, width=4, kv_len=8192, ragged=True, room=40, spare=16384),
        # begun pages of a few sequences
        dict(c, name="copy a few pages", partly=True),
        # a prefix of 131072 tokens to pages of its own
        dict(c, name="copy a long prefix", pages=2048, page=64),
        # the accepted ones of proposed tokens
        dict(m, name="compact accepted tokens"),
        # half of the tokens of long texts dropped
        dict(m, name="compact long texts", batch=8, kv_len=16384, keep=0.5, page=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    c = dict(op=rng.choice(["attend", "attend", "norm", "norm", "fork", "copy", "compact"]), kv_heads=kv_heads,
             dim=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64, 128]), cache=rng.choice(["e4m3", "e4m3", "16"]),
             dtype=rng.choice(["bf16", "fp16"]))
    wide = kv_heads * c["dim"]
    if c["op"] in ("attend", "norm"):
        c["heads"] = kv_heads * rng.choice([1, 2, 4, 8] if kv_heads > 4 else [1, 4, 7, 8, 16])
        c["ragged"], c["batch"] = rng.random() < 0.7, _log(rng, 1, 64)
    if c["op"] == "attend":
        c["q_len"] = rng.choice([1, 1, 1, rng.randint(2, 9), _log(rng, 10, 2048)])
        c["kv_len"] = max(c["q_len"], _log(rng, 1, 32768))
        c["window"] = _log(rng, 1, 4096)
        c["sinks"] = rng.choice([0, 1, 4, rng.randint(5, 300)])
        seen = c["q_len"] + min(c["kv_len"], c["window"] + c["sinks"])
        # the plain form's scores, the cache and the products stay below the listed cases' largest
        while c["batch"] > 1 and (c["batch"] * c["heads"] * c["q_len"] * seen > 1 << 29 or
                                  c["batch"] * c["kv_len"] * wide > 1 << 30):
            c["batch"] //= 2
        while c["heads"] * c["q_len"] * (c["q_len"] + seen) > 1 << 29:
            c["q_len"] = (c["q_len"] + 1) // 2
        c["released"], c["lse"] = rng.random() < 0.5, rng.random() < 0.5
    elif c["op"] == "norm":
        c["new_len"] = rng.choice([1, 1, rng.randint(2, 40), _log(rng, 41, 4096)])
        c["kv_len"] = c["new_len"] + rng.choice([0, rng.randint(1, 600)])
        while c["batch"] > 1 and c["batch"] * c["new_len"] * (c["heads"] + 2 * kv_heads) * c["dim"] > 1 << 27:
            c["batch"] //= 2
        c["cached"] = rng.random() < 0.7
        c["rot"] = rng.choice([c["dim"], c["dim"], c["dim"] // 2])
        c["interleaved"] = rng.random() < 0.3
    elif c["op"] == "fork":
        c["groups"], c["width"], c["kv_len"], c["room"] = _log(rng, 1, 32), rng.randint(2, 9), _log(rng, 1, 8192), rng.randint(1, 100)
        while c["groups"] > 1 and c["groups"] * c["kv_len"] * wide > 1 << 28:
            c["groups"] //= 2
        c["ragged"] = rng.random() < 0.7
        c["spare"] = c["groups"] * c["width"] * (100 // c["page"] + 3) + rng.randint(1, 4096)
        while c["spare"] * c["page"] * wide > 1 << 29:
            c["page"] //= 2
            c["spare"] = max(c["groups"] * c["width"] * (100 // c["page"] + 3), c["spare"] // 2)
            if c["page"] == 16:
                break
    elif c["op"] == "copy":
        c["pages"], c["partly"] = _log(rng, 1, 2048), rng.random() < 0.5
        while c["pages"] * c["page"] * wide > 1 << 27:
            c["pages"] //= 2
    else:
        c["batch"], c["kv_len"], c["keep"] = _log(rng, 1, 64), _log(rng, 1, 16384), rng.choice([0.1, 0.4, 0.5, 0.9])
        while c["batch"] > 1 and c["batch"] * c["kv_len"] * wide > 1 << 27:
            c["batch"] //= 2
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


def _fork_lengths(case, seed):
    g = torch.Generator().manual_seed(seed * 7919 + 17)
    kv = case["kv_len"]
    if not case["ragged"]:
        return [kv] * case["groups"]
    return [int(x) for x in torch.randint((kv + 1) // 2, kv + 1, (case["groups"],), generator=g)]


def _quantise(x):
    """x [pages, tokens, heads, D] as e4m3 with the least power-of-two scale a page and head under which it fits."""
    m, e = torch.frexp(x.abs().amax(dim=(1, 3)))
    e = torch.where(m > 0.875, e - 8, e - 9).masked_fill(m == 0, MIN_EXP).clamp(MIN_EXP, MAX_EXP)
    scale = torch.ldexp(torch.ones_like(m), e)
    return (x / scale[:, None, :, None]).clamp(-448, 448).to(E4M3), scale


def _pool(s, n_pages, g):
    """The cache's pages, all in use: keys carry a few channels far larger than the rest, values do not."""
    case = s["case"]
    P, Hkv, D = case["page"], case["kv_heads"], case["dim"]
    loud = torch.ones(D, device=DEV)
    loud[:: D // 4] = 4.0
    for name, spread in (("k", loud), ("v", 0.5)):
        parts, scales = [], []
        step = max(1, (1 << 28) // (P * Hkv * D))
        for p0 in range(0, n_pages, step):
            n = min(step, n_pages - p0)
            # (pages differ in size from each other, so that their scales do)
            x = torch.randn(n, P, Hkv, D, generator=g, device=DEV) * spread
            x = x * torch.exp2(torch.randint(-1, 2, (n, 1, Hkv, 1), generator=g, device=DEV).float())
            if case["cache"] == "e4m3":
                x, scale = _quantise(x)
                scales.append(scale)
            else:
                x = x.to(TYPES[case["dtype"]])
            parts.append(x)
        s["cache_" + name] = torch.cat(parts) if len(parts) > 1 else parts[0]
        s["scale_" + name] = torch.cat(scales) if scales else None


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    s = dict(case=case)
    g = torch.Generator(device=DEV).manual_seed(seed)
    {"attend": _prepare_batch, "norm": _prepare_batch, "fork": _prepare_fork, "copy": _prepare_copy,
     "compact": _prepare_compact}[case["op"]](s, seed, g)
    if own:
        import scaled_dot_product_forward_gb300 as sdpa
        s["sdpa"] = sdpa
        if "cache_k" in s:
            s["handle"] = sdpa.SdpaPagedCache(s["cache_k"], s["cache_v"], s["scale_k"], s["scale_v"])
    return s


def _prepare_batch(s, seed, g):
    case = s["case"]
    new, lens = _lengths(case, seed)
    B, P, H, Hkv, D = case["batch"], case["page"], case["heads"], case["kv_heads"], case["dim"]
    dtype = TYPES[case["dtype"]]
    per_seq = -(-case["kv_len"] // P)
    s.update(max_new=max(new), max_len=max(lens), lens=_i32(lens))
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu"], total = _i32(cu), cu[-1]

    def normal(*shape, spread=1.0):
        return torch.randn(*shape, generator=g, device=DEV) * spread

    if case["op"] == "attend" or case["cached"]:
        # pages as a serving program's pool hands them out; those that no new token sees have been given back
        held = torch.ones(B, per_seq, dtype=torch.bool)
        if case.get("released"):
            for b, (n, L) in enumerate(zip(new, lens)):
                held[b, -(-case["sinks"] // P):max(0, L - n + 1 - case["window"]) // P] = False
                held[b, -(-L // P):] = False
        held = held.to(DEV)
        n_pages = int(held.sum()) + 3
        table = torch.full((B, per_seq), -1, dtype=torch.int32, device=DEV)
        table[held] = torch.randperm(n_pages, generator=g, device=DEV)[:n_pages - 3].to(torch.int32)
        s["table"] = table
        _pool(s, n_pages, g)
    s["q"] = normal(total, H, D).to(dtype)
    if case["op"] == "attend":
        return
    loud = torch.ones(D, device=DEV)
    loud[:: D // 4] = 4.0
    s["k"] = normal(total, Hkv, D, spread=loud).to(dtype)
    s["v"] = normal(total, Hkv, D, spread=0.5).to(dtype)
    s["q_norm"], s["k_norm"] = 1 + normal(D, spread=0.2), 1 + normal(D, spread=0.2)
    b, i, pos = _token_places(s)
    s["positions"] = pos.to(torch.int32)
    half = case["rot"] // 2
    angle = torch.arange(per_seq * P, device=DEV, dtype=torch.float64)[:, None] * torch.pow(
        10000.0, -torch.arange(half, device=DEV, dtype=torch.float64) / half)
    s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()


def _prepare_fork(s, seed, g):
    case = s["case"]
    P, n = case["page"], case["groups"]
    lens = _fork_lengths(case, seed)
    per_seq = -(-(case["kv_len"] + case["room"]) // P)
    used = sum(-(-L // P) for L in lens)
    n_pages = n * -(-case["kv_len"] // P) + case["spare"]
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    # row g * width of the table is a text's best beam, the others are to become copies of it
    table = torch.full((n * case["width"], per_seq), -1, dtype=torch.int32, device=DEV)
    refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    refs[perm[used:used + case["spare"] // 4].long()] = 1      # other programs' pages
    at = 0
    for i, L in enumerate(lens):
        m = -(-L // P)
        table[i * case["width"], :m] = perm[at:at + m]
        at += m
    refs[perm[:used].long()] = 1
    each = torch.tensor(lens).repeat_interleave(case["width"])
    best = torch.arange(n).repeat_interleave(case["width"] - 1) * case["width"]
    other = torch.tensor([i * case["width"] + j for i in range(n) for j in range(1, case["width"])])
    to = each.clone()
    to[other] += case["room"]
    s.update(table=table, refs=refs, lens=each.to(torch.int32).to(DEV), to_lens=to.to(torch.int32).to(DEV),
             src=best.to(torch.int32).to(DEV), dst=other.to(torch.int32).to(DEV))
    _pool(s, n_pages, g)


def _prepare_copy(s, seed, g):
    case = s["case"]
    n = case["pages"]
    perm = torch.randperm(2 * n + 3, generator=g, device=DEV).to(torch.int32)
    s["src"], s["dst"] = perm[:n].contiguous(), perm[n:2 * n].contiguous()
    s["rows"] = torch.randint(1, case["page"] + 1, (n,), generator=g, device=DEV, dtype=torch.int32) if case["partly"] else None
    _pool(s, 2 * n + 3, g)


def _kept_counts(case, seed):
    """Kept tokens of each sequence, on the host."""
    h = torch.Generator().manual_seed(seed * 7919 + 29)
    return [max(1, round(case["kv_len"] * case["keep"] * (0.8 + 0.2 * float(x)))) for x in torch.rand(case["batch"], generator=h)]


def _prepare_compact(s, seed, g):
    case = s["case"]
    B, P, L = case["batch"], case["page"], case["kv_len"]
    counts, most = _kept_counts(case, seed), max(1, round(L * case["keep"]))
    old, new = -(-L // P), -(-most // P)
    n_pages = B * (old + new) + 3
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    s["table"] = perm[:B * old].view(B, old).contiguous()
    s["new_table"] = perm[B * old:B * (old + new)].view(B, new).contiguous()
    kept = torch.zeros(B, most, dtype=torch.int32, device=DEV)
    for b, n in enumerate(counts):
        kept[b, :n] = torch.randperm(L, generator=g, device=DEV)[:n].sort().values.to(torch.int32)
    s["kept"], s["kept_lens"] = kept, _i32(counts)
    _pool(s, n_pages, g)


def run(s):
    return {"attend": _attend, "norm": _norm, "fork": _fork, "copy": _copy, "compact": _compact}[s["case"]["op"]](s)


def _token_places(s):
    """Sequence and index within its new tokens of each token, and each token's position."""
    cu, lens = s["cu"].long(), s["lens"].long()
    t = torch.arange(s["q"].shape[0], device=DEV)
    b = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[b]
    return b, i, lens[b] - (cu[b + 1] - cu[b]) + i


def _attend(s):
    case = s["case"]
    if own:
        return s["sdpa"].sdpa_paged_forward(s["q"], s["handle"], s["table"], s["lens"], s["cu"], s["max_new"], is_causal=True,
                                            window=case["window"], sinks=case["sinks"], return_lse=case["lse"])
    B, H, Hkv, D, P = case["batch"], case["heads"], case["kv_heads"], case["dim"], case["page"]
    W, S, n, G = case["window"], case["sinks"], s["max_new"], H // Hkv
    b, i, _ = _token_places(s)
    lens, count = s["lens"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    q = torch.zeros(B, n, H, D, device=DEV)
    q[b, i] = s["q"].float()
    q = q.view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    # the first tokens, and those from the first new token's window on
    first = (lens - count + 1 - W).clamp(min=0).clamp(min=min(S, s["max_len"]))
    span = min(W + n - 1, s["max_len"])
    j = torch.cat([torch.arange(min(S, s["max_len"]), device=DEV).expand(B, -1),
                   first[:, None] + torch.arange(span, device=DEV)], 1)
    inside = j < lens[:, None]
    page = s["table"].long().gather(1, (j // P).clamp(max=s["table"].shape[1] - 1))
    inside &= page >= 0
    page, row = page.clamp(min=0), j % P

    def gathered(name):
        cache, scale = s["cache_" + name], s["scale_" + name]
        if scale is None:
            x = cache[page, row].float()
        else:
            x = cache.view(torch.uint8)[page, row].view(E4M3).float() * scale[page][..., None]
        return torch.where(inside[:, :, None, None], x, torch.zeros_like(x))

    scores = torch.matmul(q, gathered("k").permute(0, 2, 3, 1)).view(B, Hkv, G, n, -1) * (1.0 / math.sqrt(D))
    last = (lens - count)[:, None] + torch.arange(n, device=DEV)[None, :]
    at = j[:, None, :]
    seen = inside[:, None, :] & (at <= last[:, :, None]) & ((at > last[:, :, None] - W) | (at < S))
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    scores.sub_(top).exp_()
    total = scores.sum(-1, keepdim=True)
    out = torch.matmul(scores.view(B, Hkv, G * n, -1), gathered("v").permute(0, 2, 1, 3)).view(B, Hkv, G, n, D)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    out = out.permute(0, 3, 1, 2, 4).reshape(B, n, H, D)[b, i].to(s["q"].dtype)
    if not case["lse"]:
        return out
    lse = (total.log() + top).permute(0, 3, 1, 2, 4).reshape(B, n, H)[b, i]
    return out, lse


def _turned(x, weight, cos, sin, interleaved):
    """x [tokens, heads, D] normalised, and pair j of each head turned by its angle (cos, sin [tokens, pairs])."""
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    c, s, half = cos[:, None, :], sin[:, None, :], cos.shape[1]
    y = x.clone()
    a = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    b = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def _norm(s):
    case = s["case"]
    if own and not case["cached"]:
        return s["sdpa"].sdpa_norm_rotate(s["q"], s["k"], s["positions"], cos=s["cos"], sin=s["sin"], interleaved=case["interleaved"],
                                          q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
    if own:
        q = s["sdpa"].sdpa_cache_append(s["handle"], s["k"], s["v"], s["table"], s["lens"], s["cu"], cos=s["cos"], sin=s["sin"],
                                        interleaved=case["interleaved"], q=s["q"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
        return dict(_state(s), q=q)
    P, dtype = case["page"], s["q"].dtype
    pos = s["positions"].long()
    cos, sin = s["cos"][pos], s["sin"][pos]
    q = _turned(s["q"], s["q_norm"], cos, sin, case["interleaved"]).to(dtype)
    k = _turned(s["k"], s["k_norm"], cos, sin, case["interleaved"])
    if not case["cached"]:
        return q, k.to(dtype)
    b, i, pos = _token_places(s)
    page, row = s["table"].long()[b, pos // P], pos % P
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
    return dict(_state(s), q=q)


def _state(s):
    return {"k": s["cache_k"], "v": s["cache_v"], "k_scale": s["scale_k"], "v_scale": s["scale_v"]}


def _fork(s):
    case = s["case"]
    P, table, refs = case["page"], s["table"], s["refs"]
    if own:
        sdpa = s["sdpa"]
        pairs = sdpa.sdpa_pages_fork(refs, table, s["lens"], s["src"], s["dst"], P)
        sdpa.sdpa_cache_copy_pages(s["handle"], pairs.src, pairs.dst, pairs.rows)
        missing = sdpa.sdpa_pages_take(refs, table, s["lens"], s["to_lens"], P)
        return dict(_state(s), refs=refs, table=table, src=pairs.src, dst=pairs.dst, rows=pairs.rows, missing=pairs.missing + missing)
    src, dst = s["src"].long(), s["dst"].long()
    entries = torch.arange(table.shape[1], device=DEV)
    lens = s["lens"].long()
    count, begun = lens[src] // P, lens[src] % P
    old = table[dst]
    refs.index_add_(0, old[old >= 0].long(), torch.full((1,), -1, dtype=torch.int32, device=DEV).expand(int((old >= 0).sum())))
    new = torch.where(entries[None, :] < count[:, None], table[src], -1)
    refs.index_add_(0, new[new >= 0].long(), torch.ones(1, dtype=torch.int32, device=DEV).expand(int((new >= 0).sum())))
    last = table[src, count.clamp(max=table.shape[1] - 1)]
    wants = (begun > 0) & (last >= 0)
    free = (refs <= 0).nonzero().flatten()
    rank = wants.long().cumsum(0) - 1
    got = wants & (rank < free.numel())
    page = free[rank.clamp(0, free.numel() - 1)]
    refs[page[got]] = 1
    new[got, count[got]] = page[got].to(torch.int32)
    table[dst] = new
    copy_src = torch.where(got, last, -1)
    copy_dst = torch.where(got, page, -1).to(torch.int32)
    rows = torch.where(got, begun, 0).to(torch.int32)
    a, b = copy_src[got].long(), copy_dst[got].long()
    _copied(s, a, b, rows[got])
    # room for the new tokens
    to = s["to_lens"].long()
    lo, hi = (lens + P - 1) // P, (to + P - 1) // P
    wanted = (entries[None, :] >= lo[:, None]) & (entries[None, :] < hi[:, None])
    r, e = wanted.nonzero(as_tuple=True)
    free = (refs <= 0).nonzero().flatten()[:r.numel()]
    table[r, e] = -1
    table[r[:free.numel()], e[:free.numel()]] = free.to(torch.int32)
    refs[free] = 1
    missing = (wants.sum() - got.sum() + r.numel() - free.numel()).to(torch.int32).view(1)
    return dict(_state(s), refs=refs, table=table, src=copy_src, dst=copy_dst, rows=rows, missing=missing)


def _copied(s, src, dst, rows):
    keep = None if rows is None else (torch.arange(s["case"]["page"], device=DEV)[None, :] < rows[:, None])[:, :, None, None]
    for name in ("k", "v"):
        cache, scale = s["cache_" + name], s["scale_" + name]
        x = cache.view(torch.uint8 if scale is not None else torch.int16)
        x[dst] = x[src] if keep is None else torch.where(keep, x[src], x[dst])
        if scale is not None:
            scale[dst] = scale[src]


def _copy(s):
    if own:
        s["sdpa"].sdpa_cache_copy_pages(s["handle"], s["src"], s["dst"], s["rows"])
    else:
        _copied(s, s["src"].long(), s["dst"].long(), s["rows"])
    return _state(s)


def _compact(s):
    if own:
        s["sdpa"].sdpa_cache_compact(s["handle"], s["table"], s["kept"], s["new_table"], s["kept_lens"])
        return _state(s)
    P = s["case"]["page"]
    b, i = (torch.arange(s["kept"].shape[1], device=DEV)[None, :] < s["kept_lens"][:, None]).nonzero(as_tuple=True)
    pos = s["kept"][b, i].long()
    src, dst = s["table"].long()[b, pos // P], s["new_table"].long()[b, i // P]
    for name in ("k", "v"):
        cache, scale = s["cache_" + name], s["scale_" + name]
        if scale is None:
            cache[dst, i % P] = cache[src, pos % P]
            continue
        now = torch.zeros_like(scale).index_reduce_(0, dst, scale[src], "amax")
        codes = cache.view(torch.uint8)
        x = codes[src, pos % P].view(E4M3).float() * (scale[src] / now[dst])[:, :, None]
        codes[dst, i % P] = x.to(E4M3).view(torch.uint8)
        scale.copy_(torch.where(now > 0, now, scale))
    return _state(s)


def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "norm": _exact_norm, "fork": _exact_fork, "copy": _exact_copy,
            "compact": _exact_compact}[case["op"]](s, case, seed)


def _exact_attend(s, case, seed):
    new, lens = _lengths(case, seed)
    P, H, Hkv, D = case["page"], case["heads"], case["kv_heads"], case["dim"]
    out = torch.zeros(sum(new), H, D, dtype=torch.float64, device=DEV)
    lse = torch.full((sum(new), H), -math.inf, dtype=torch.float64, device=DEV)
    row = 0
    for b, (n, L) in enumerate(zip(new, lens)):
        for r0 in range(0, n, 512):
            r1 = min(n, r0 + 512)
            pos = torch.arange(L - n + r0, L - n + r1, device=DEV)
            lo = max(0, L - n + r0 - case["window"] + 1)
            keys = [x for x in range(min(case["sinks"], lo))] + list(range(lo, L - n + r1))
            keys = torch.tensor(keys, device=DEV)
            pages = s["table"][b].long()[keys // P]
            # (key, row): whether the row sees the key
            behind = pos[:, None] - keys[None, :]
            sees = (behind >= 0) & ((behind < case["window"]) | (keys < case["sinks"])[None, :])
            for h in range(Hkv):
                kv = []
                for name in ("k", "v"):
                    x = s["cache_" + name][:, :, h].view(torch.uint8 if case["cache"] == "e4m3" else torch.int16)[pages, keys % P]
                    x = x.view(s["cache_" + name].dtype).double()
                    if case["cache"] == "e4m3":
                        x = x * s["scale_" + name][pages, h].double()[:, None]
                    kv.append(x)
                for g in range(h * (H // Hkv), (h + 1) * (H // Hkv)):
                    z = s["q"][row + r0:row + r1, g].double() @ kv[0].T / math.sqrt(D)
                    z = torch.where(sees, z, -math.inf)
                    lse[row + r0:row + r1, g] = torch.logsumexp(z, -1)
                    out[row + r0:row + r1, g] = torch.softmax(z, -1) @ kv[1]
        row += n
    return (out, lse) if case["lse"] else out


def _exact_norm(s, case, seed):
    new, lens = _lengths(case, seed)
    P, half = case["page"], case["rot"] // 2
    start = [sum(new[:b]) for b in range(len(new))]
    at = torch.cat([torch.arange(L - n, L, device=DEV) for n, L in zip(new, lens)])
    turn = torch.complex(s["cos"].double(), s["sin"].double())[at][:, None]

    def turned(x, weight):
        x = x.double()
        x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS) * weight.double()
        r, rest = x[..., :2 * half], x[..., 2 * half:]
        pairs = r.unflatten(-1, (half, 2)) if case["interleaved"] else r.unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        r = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([r, rest], -1)

    q, k = turned(s["q"], s["q_norm"]), turned(s["k"], s["k_norm"])
    if not case["cached"]:
        return q, k
    got = {"k_scale": None, "v_scale": None}
    for name, x in (("k", k), ("v", s["v"].double())):
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
    return {"k": got["k"], "v": got["v"], "k_scale": got["k_scale"], "v_scale": got["v_scale"], "q": q}


def _held(s):
    """The cache as numbers in 64 bits, laid out as run's."""
    return {k: None if t is None else t.double() for k, t in _state(s).items()}


def _move(held, src, dst, count):
    for name in ("k", "v"):
        held[name][dst, :count] = held[name][src, :count].clone()
        if held[name + "_scale"] is not None:
            held[name + "_scale"][dst] = held[name + "_scale"][src].clone()


def _exact_fork(s, case, seed):
    P = case["page"]
    table, refs, lens, to = (s[n].tolist() for n in ("table", "refs", "lens", "to_lens"))
    src, dst = s["src"].tolist(), s["dst"].tolist()
    held = _held(s)
    for d in dst:
        for p in table[d]:
            if p >= 0:
                refs[p] -= 1
    for a, d in zip(src, dst):
        table[d] = [p if e < lens[a] // P else -1 for e, p in enumerate(table[a])]
        for p in table[d]:
            if p >= 0:
                refs[p] += 1
    free = iter([p for p, n in enumerate(refs) if n <= 0])
    pairs, missing = [], 0
    for a, d in zip(src, dst):
        e = lens[a] // P
        pair = (-1, -1, 0)
        if lens[a] % P and table[a][e] >= 0:
            p = next(free, None)
            if p is None:
                missing += 1
            else:
                refs[p] = 1
                table[d][e] = p
                pair = (table[a][e], p, lens[a] % P)
        pairs.append(pair)
    for a, d, n in pairs:
        if d >= 0:
            _move(held, a, d, n)
    for r, row in enumerate(table):
        for e in range(-(-lens[r] // P), -(-to[r] // P)):
            p = next(free, None)
            row[e] = -1 if p is None else p
            missing += p is None
            if p is not None:
                refs[p] = 1
    return dict(held, refs=_i32(refs), table=_i32(table), src=_i32([x[0] for x in pairs]), dst=_i32([x[1] for x in pairs]),
                rows=_i32([x[2] for x in pairs]), missing=_i32([missing]))


def _exact_copy(s, case, seed):
    held = _held(s)
    rows = [case["page"]] * case["pages"] if s["rows"] is None else s["rows"].tolist()
    for a, d, n in zip(s["src"].tolist(), s["dst"].tolist(), rows):
        _move(held, a, d, n)
    return held


def _exact_compact(s, case, seed):
    P, held = case["page"], _held(s)
    for b, n in enumerate(_kept_counts(case, seed)):
        pos = s["kept"][b, :n].long()
        pages = s["table"][b].long()[pos // P]
        for e in range(-(-n // P)):
            part = slice(e * P, min(n, (e + 1) * P))
            page, rows = int(s["new_table"][b, e]), pos[part] % P
            for name in ("k", "v"):
                x, scale = held[name][pages[part], rows], held[name + "_scale"]
                if scale is not None:
                    each = scale[pages[part]]
                    scale[page] = each.amax(0)
                    x = x * each[:, :, None] / scale[page][None, :, None]
                held[name][page, :x.shape[0]] = x
    return held


def work(case):
    if not case.get("ragged") and case["op"] != "compact":
        return _work(case, 0)
    each = [_work(case, seed) for seed in range(16)]     # lengths differ from seed to seed
    return {key: sum(w[key] for w in each) / len(each) for key in each[0]}


def _work(case, seed):
    Hkv, D, P = case["kv_heads"], case["dim"], case["page"]
    wide = 1 if case["cache"] == "e4m3" else 2
    token = 2 * Hkv * D * wide                        # a token's key and value
    scales = 8 * Hkv if wide == 1 else 0              # a page's
    if case["op"] == "attend":
        new, lens = _lengths(case, seed)
        W, S, H = case["window"], case["sinks"], case["heads"]
        # tokens that some new token sees, their pages, and (token, new token) pairs
        tokens = pages = pairs = 0
        for n, L in zip(new, lens):
            lo = max(0, L - n + 1 - W)
            few = min(S, lo)
            tokens += L - lo + few
            pages += -(-L // P) - lo // P + (min(-(-few // P), lo // P) if few else 0)
            for p in range(L - n, L):
                begin = max(0, p + 1 - W)
                pairs += p + 1 - begin + min(S, begin)
        moved = tokens * token + pages * (4 + scales) + 2 * 2 * sum(new) * H * D + (4 * sum(new) * H if case["lse"] else 0)
        return {"bytes": moved, "flops": 4.0 * H * D * pairs}
    if case["op"] == "norm":
        new, lens = _lengths(case, seed)
        total, H = sum(new), case["heads"]
        places = len({p for n, L in zip(new, lens) for p in range(L - n, L)})
        moved = 2 * 2 * total * H * D + 4 * case["rot"] * places + 8 * D
        flops = total * (H + Hkv) * (4.0 * D + 3.0 * case["rot"])
        if not case["cached"]:
            return {"bytes": moved + 2 * 2 * total * Hkv * D + 4 * total, "flops": flops}
        pages = sum((L - 1) // P - (L - n) // P + 1 for n, L in zip(new, lens))
        return {"bytes": moved + total * (2 * 2 * Hkv * D + token) + pages * (4 + 2 * scales), "flops": flops}
    if case["op"] == "fork":
        moved = 0
        for L in _fork_lengths(case, seed):
            entries = -(-(case["kv_len"] + case["room"]) // P)
            fresh = -(-(L + case["room"]) // P) - L // P
            each = 4 * entries * 2 + 4 * (L // P) + 8 * (L // P) + 8 * fresh + (2 * (L % P) * token + 2 * scales if L % P else 0)
            moved += (case["width"] - 1) * each
        return {"bytes": moved, "flops": 0.0}
    if case["op"] == "copy":
        rows = (P + 1) / 2 if case["partly"] else P
        return {"bytes": 2.0 * case["pages"] * (rows * token + scales), "flops": 0.0}
    counts = _kept_counts(case, seed)
    old = -(-case["kv_len"] // P)
    moved = sum(n * (2 * token + 4) + (min(n, old) + -(-n // P)) * (4 + scales) for n in counts)
    return {"bytes": moved, "flops": 0.0}
