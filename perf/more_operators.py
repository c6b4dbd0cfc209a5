"""Cases and plain forms of the operators of a decode step round the paged KV cache: places for the
step's tokens (page tables and slot maps from lengths), the norm and rotation of queries and keys on
their way into the cache, and attention of sequences that share a long prefix.

A pool of pages is a uint8 tensor [pages, page bytes]. A page holds `page` tokens of every KV head;
the part of one head (T tokens, D elements a token) is, in this order,

  q8    K codes int8 [T][D], V codes int8 [T][D], K scales fp16 [T][D/32], V scales fp16 [D/32][T]
  f16   K fp16 [T][D], V fp16 [T][D]

A q8 element stands for code * scale, rounded once to fp16 and saturated at +-65504. `table`
(int32 [sequences, pages a sequence], -1 for none) maps a sequence's tokens to pages, `lens`
(int32) holds the sequences' lengths and `refs` (int32) how many sequences hold a page.
"""
import math
import random

import torch

own = False

GROUP = 32
FP16_MAX = 65504.0


# ---- cases -----------------------------------------------------------------------------

def _extend(name, rows, page, pages, past, reject, prompts, prompt, slots):
    """Rows of up to `past` tokens, of which `reject` are taken back; `prompts` rows get up to `prompt`
    tokens each, the others `reject` + 1."""
    return {"name": name, "op": "extend", "rows": rows, "page": page, "pages": pages, "past": past, "reject": reject,
            "prompts": prompts, "prompt": prompt, "slots": slots}


def _rope(name, cache, batch, new, past, heads, kv_heads, dim, page, rot, interleaved, norm, scaled):
    return {"name": name, "op": "rope", "cache": cache, "batch": batch, "new": new, "past": past, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "rot": rot, "interleaved": interleaved, "norm": norm,
            "scaled": scaled}


def _prefix(name, kind, groups, rows, heads, kv_heads, dim, page, prefix, tail, ragged, f32=False):
    return {"name": name, "op": "prefix", "kind": kind, "groups": groups, "rows": rows, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "prefix": prefix, "tail": tail, "ragged": ragged, "f32": f32}


def listed():
    return [
        # a served batch of 64 in speculative decoding: four drafted tokens taken back, five more asked
        _extend("extend_draft64", 64, 16, 4096, 900, 4, 0, 0, 320),
        # a large server's step: 1000 sequences of one token, some prompts in chunks, a pool of 4 million tokens
        _extend("extend_mixed1000", 1000, 16, 262144, 3500, 0, 24, 2048, 32768),
        # one user's decode step: query and key norms, rotation, int8 cache; latency
        _rope("rope_q8_decode1", "q8", 1, 1, 1000, 32, 8, 128, 16, 128, False, True, False),
        # the same for a served batch
        _rope("rope_q8_decode64", "q8", 64, 1, 1500, 32, 8, 128, 16, 128, False, True, False),
        # a prefill chunk far into a long context whose frequencies are scaled; 70B-like heads, fp16 cache
        _rope("rope_f16_chunk8192", "f16", 1, 8192, 120000, 64, 8, 128, 64, 128, False, False, True),
        # dense rotation of a quarter of heads of 256 in interleaved pairs, an odd number of tokens, with norms
        _rope("rope_dense_part256", "", 1, 4099, 0, 16, 4, 256, 16, 64, True, True, False),
        # eight samples of one prompt of a thousand tokens: the smallest call
        _prefix("prefix_q8_8x1000", "q8", 1, 8, 32, 8, 128, 16, 1000, 32, False),
        # a 70B-like layer (64 heads, 8 KV heads), fp16 cache, a long system prompt and short chats after it
        _prefix("prefix_f16_64x8192", "f16", 1, 64, 64, 8, 128, 64, 8192, 512, False),
        # a 7B-like layer (32 heads, 8 KV heads), int8 cache, a document that 128 questions share: the most products
        _prefix("prefix_q8_128x16384", "q8", 1, 128, 32, 8, 128, 32, 16384, 1024, False),
        # several prompts with some samples each, no shared KV heads, heads of 64, fp32 output
        _prefix("prefix_f16_mha64_groups", "f16", 5, 41, 12, 12, 64, 32, 4001, 300, True, True),
        # one KV head for all heads, heads of 256, large pages
        _prefix("prefix_q8_mqa256", "q8", 1, 48, 16, 1, 256, 128, 6007, 100, False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["extend", "rope", "rope", "prefix", "prefix", "prefix"])
    page = rng.choice([16, 32, 64, 128])
    if op == "extend":
        rows = _log(rng, 1, 1024)
        past = _log(rng, 1, 4000)
        pages = min(262144, rows * (-(-past // page) + 1) + _log(rng, 1, 20000))
        past = max(1, min(past, (pages // rows - 1) * page))
        prompts = rng.randint(0, rows) if rng.random() < 0.5 else 0
        prompt = _log(rng, 1, 2048)
        reject = rng.choice([0, 0, 1, 4, 7])
        most = rows * (reject + 1) + prompts * prompt
        case = _extend("", rows, page, pages, past, reject, prompts, prompt, min(65536, _log(rng, 1, 2 * most + 1)))
    else:
        dim = rng.choice([64, 128, 128, 256])
        kv_heads = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    if op == "rope":
        batch = _log(rng, 1, 256)
        new = 1 if rng.random() < 0.5 else _log(rng, 1, max(1, 8192 // batch))
        while batch * new * kv_heads * (group + 2) * dim > 8192 * 80 * 128:
            batch, new = max(1, batch // 2), max(1, new // 2)
        rot = rng.choice([dim, dim, dim // 2, dim // 4, 16, 48])
        case = _rope("", rng.choice(["q8", "f16", ""]), batch, new, _log(rng, 1, 200000), kv_heads * group, kv_heads, dim,
                     page, rot, rng.random() < 0.4, rng.random() < 0.5, rng.random() < 0.4)
    if op == "prefix":
        rows = _log(rng, 1, 256)
        groups = 1 if rng.random() < 0.5 else rng.randint(1, max(1, rows // 2))
        prefix, tail = _log(rng, 1, 32768), _log(rng, 1, 2048)
        # no more products with the prefixes than the largest listed case, nor more cached elements
        most = 128 * 32 * 16384 * 128
        prefix = max(1, min(prefix, most // (rows * kv_heads * group * dim), (1 << 27) // (groups * kv_heads * dim)))
        tail = max(1, min(tail, (1 << 27) // (rows * kv_heads * dim)))
        case = _prefix("", rng.choice(["q8", "f16"]), groups, rows, kv_heads * group, kv_heads, dim, page, prefix, tail,
                       rng.random() < 0.6, rng.random() < 0.3)
    del case["name"]
    return case


def _shape(case):
    """(rows of each group, prefix of each group, length of each row). They belong to the case, not to a seed."""
    r = random.Random(case["rows"] * 1000003 + case["prefix"])
    groups, rows, prefix, tail = case["groups"], case["rows"], case["prefix"], case["tail"]
    if not case["ragged"]:
        sizes = [rows // groups + (g < rows % groups) for g in range(groups)]
        lens = [prefix + 1 + b * (tail - 1) // max(1, rows - 1) for b in range(rows)]
        return sizes, [prefix] * groups, lens
    cuts = sorted(r.sample(range(1, rows), groups - 1)) if groups > 1 else []
    sizes = [b - a for a, b in zip([0] + cuts, cuts + [rows])]
    prefixes = [max(1, int(prefix * (1 - 0.8 * r.random()))) for _ in sizes]
    prefixes[0] = prefix
    lens = [p + 1 + int((tail - 1) * r.random() ** 2) for n, p in zip(sizes, prefixes) for _ in range(n)]
    if rows > 6 and sizes[-1] > 2:
        lens[-1] = 0                                       # a padded place of the batch
        lens[-2] = 1                                       # a row that is shorter than its group's prefix
    return sizes, prefixes, lens


# ---- pools -----------------------------------------------------------------------------

def _page_bytes(kind, kv_heads, dim, page):
    return kv_heads * page * (4 * dim if kind == "f16" else 2 * dim + 4 * (dim // GROUP))


def _parts(pool, kind, kv_heads, dim, page):
    """Views of a pool: (K, V) or (K codes, V codes, K scales, V scales)."""
    p = pool.view(pool.shape[0], kv_heads, -1)
    td, g = page * dim, dim // GROUP
    if kind == "f16":
        p = p.view(torch.float16)
        return p[:, :, :td].unflatten(-1, (page, dim)), p[:, :, td:].unflatten(-1, (page, dim))
    codes, scales = p.view(torch.int8), p.view(torch.float16)
    return (codes[:, :, :td].unflatten(-1, (page, dim)), codes[:, :, td:2 * td].unflatten(-1, (page, dim)),
            scales[:, :, td:td + page * g].unflatten(-1, (page, g)), scales[:, :, td + page * g:].unflatten(-1, (g, page)))


def _encode(x):
    """fp16 [..., D] -> int8 codes [..., D] and fp16 scales [..., D/32], decided on 64-bit quotients."""
    g = x.double().unflatten(-1, (-1, GROUP))
    t = g.abs().amax(-1) / 127
    d = t.half()
    d = torch.where(d.double() < t, (d.view(torch.int16) + 1).view(torch.float16), d)   # smallest fp16 >= t
    step = d.double()[..., None]
    q = torch.where(step > 0, torch.round(g / torch.where(step > 0, step, 1.0)), 0.0)
    return q.to(torch.int8).flatten(-2), d


def _decode(codes, scales):
    """int8 [..., D], fp16 [..., D/32] -> the fp16 values they stand for, in fp32."""
    v = codes.float().unflatten(-1, (-1, GROUP)) * scales.float()[..., None]
    return v.clamp(-FP16_MAX, FP16_MAX).half().float().flatten(-2)


def _heads(shape, gen):
    """Heads of keys, values or queries: centred, channels of different size."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16)
    return x * (torch.rand(shape[-1], generator=gen, device="cuda") * 1.2 + 0.3).half()


def _fill(pool, kind, kv_heads, dim, page, gen):
    step = max(1, (1 << 26) // (kv_heads * dim * page))
    for at in range(0, pool.shape[0], step):
        part = _parts(pool[at:at + step], kind, kv_heads, dim, page)
        for i in (0, 1):
            x = _heads((min(step, pool.shape[0] - at), kv_heads, page, dim), gen)
            if kind == "f16":
                part[i].copy_(x)
            else:
                codes, scales = _encode(x)
                part[i].copy_(codes)
                part[2 + i].copy_(scales if i == 0 else scales.transpose(-1, -2))


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _freqs(case):
    """Radians a token of each rotated pair, fp64. Scaled for a context eight times as long: pairs that turn less
    than once in the trained 16384 tokens turn eight times slower, those of over 32 turns as before."""
    half = case["rot"] // 2
    f = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    if case["scaled"]:
        turns = 16384 * f / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        f = f * (keep + (1 - keep) / 8)
    return f.cuda()


# ---- states ------------------------------------------------------------------------------

def _prepare_extend(case, seed, gen):
    r = random.Random(seed)
    rows, page, pages = case["rows"], case["page"], case["pages"]
    kept = [r.randint(1, case["past"]) for _ in range(rows)]
    for b in r.sample(range(rows), case["prompts"]):
        kept[b] = 0
    lens = [n + case["reject"] if n else 0 for n in kept]
    add = [case["reject"] + 1 if n else r.randint(1, case["prompt"]) for n in kept]
    width = -(-(case["past"] + max(2 * case["reject"] + 1, case["prompt"])) // page)
    held = -(-_ints(lens) // page)
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    j = torch.arange(width, device="cuda")
    at = (held.cumsum(0) - held)[:, None] + j
    taken = (j < held[:, None]) & (at < pages)
    table = torch.where(taken, order[at.clamp(max=pages - 1)], -1)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[table[taken].long()] = 1
    pool = torch.empty((pages, _page_bytes("q8", 1, 64, page)), dtype=torch.uint8, device="cuda")
    return {"case": case, "pool": pool, "table": table, "lens": _ints(lens), "refs": refs, "to": _ints(kept), "add": _ints(add)}


def _prepare_rope(case, seed, gen):
    batch, new, past, page, dim = case["batch"], case["new"], case["past"], case["page"], case["dim"]
    count, heads, kv_heads = batch * new, case["heads"], case["kv_heads"]
    # one projection's output: the queries, keys and values of a token side by side
    qkv = _heads((count, heads + 2 * kv_heads, dim), gen).flatten(1)
    at = torch.arange(past, past + new, device="cuda", dtype=torch.int32)
    state = {"case": case, "qkv": qkv, "positions": at.repeat(batch), "freqs": _freqs(case), "q_weight": None, "k_weight": None}
    if case["norm"]:
        state["q_weight"], state["k_weight"] = (torch.rand((2, dim), generator=gen, device="cuda") + 0.5).half()
    if case["cache"]:
        # only the pages of the new tokens are in this pool: the earlier ones were given up, or are never looked at
        first, last = past // page, (past + new - 1) // page
        each = last - first + 1
        pool = torch.empty((batch * each + 3, _page_bytes(case["cache"], kv_heads, dim, page)), dtype=torch.uint8, device="cuda")
        _fill(pool, case["cache"], kv_heads, dim, page, gen)
        order = torch.randperm(pool.shape[0], generator=gen, device="cuda").int()
        state["table"] = torch.full((batch, last + 1), -1, dtype=torch.int32, device="cuda")
        state["table"][:, first:] = order[:batch * each].view(batch, each)
        state["pool"] = pool
        state["seqs"] = torch.arange(batch, device="cuda", dtype=torch.int32).repeat_interleave(new)
    return state


def _prepare_prefix(case, seed, gen):
    sizes, prefixes, lens = _shape(case)
    page, kind, kv_heads, dim = case["page"], case["kind"], case["kv_heads"], case["dim"]
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + n)
    lead = [starts[g] for g, n in enumerate(sizes) for _ in range(n)]
    prefix = [prefixes[g] for g, n in enumerate(sizes) for _ in range(n)]
    whole = [0 if b == i else min(p, lens[b]) // page for i, (b, p) in enumerate(zip(lead, prefix))]   # pages of the first row's
    held = [-(-n // page) for n in lens]
    own_pages = [max(0, h - w) for h, w in zip(held, whole)]
    pages = sum(own_pages) + 3
    width = -(-max(lens) // page)
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    w, h, n = (_ints(v)[:, None] for v in (whole, held, own_pages))
    j = torch.arange(width, device="cuda")
    at = (n.cumsum(0) - n) + j - w
    mine = torch.where((j >= w) & (j < h), order[at.clamp(0, pages - 1)], -1)
    lead_t = torch.tensor(lead, device="cuda")
    table = torch.where(j < torch.minimum(w, h), mine[lead_t], mine)
    pool = torch.empty((pages, _page_bytes(kind, kv_heads, dim, page)), dtype=torch.uint8, device="cuda")
    _fill(pool, kind, kv_heads, dim, page, gen)
    # the page that the prefix ends in is each row's own, with the prefix's tokens in it
    copies = [(i, b) for i, (b, x) in enumerate(zip(lead, whole)) if b != i and prefix[i] % page and held[i] > x and held[b] > x]
    if copies:
        i, b = (torch.tensor(v, device="cuda") for v in zip(*copies))
        pool[table[i, w[i, 0].long()].long()] = pool[table[b, w[i, 0].long()].long()]
    q = torch.randn((case["rows"], case["heads"], dim), generator=gen, device="cuda") * 1.5
    return {"case": case, "pool": pool, "table": table, "lens": _ints(lens), "q": q.half(), "starts": _ints(starts),
            "prefix": _ints(prefixes), "group": _ints([g for g, n in enumerate(sizes) for _ in range(n)]).long(),
            "rank": _ints([i for n in sizes for i in range(n)]).long(), "most": max(sizes)}


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    return {"extend": _prepare_extend, "rope": _prepare_rope, "prefix": _prepare_prefix}[case["op"]](case, seed, gen)


# ---- the operators -----------------------------------------------------------------------

def _handle(state, kind, kv_heads, dim):
    """The framework's handle of the pool, which a program makes once and keeps."""
    import dequant_gemv_q4g32_amd as qg
    if "handle" not in state:
        state["handle"] = qg.KVPool(state["pool"], kind, kv_heads, dim, state["case"]["page"])
    return qg, state["handle"]


def _run_extend(s):
    """The step's rejected tokens are taken back, then every row gets places for its next ones."""
    c = s["case"]
    table, lens, refs, to, add, page, slots = s["table"], s["lens"], s["refs"], s["to"], s["add"], c["page"], c["slots"]
    if own:
        qg, kv = _handle(s, "q8", 1, 64)
        qg.kv_trim(kv, table, lens, refs, to)
        granted, seqs, positions = qg.kv_extend(kv, table, lens, refs, add, slots)
    else:
        width, j = table.shape[1], torch.arange(table.shape[1], device="cuda")
        cut = (to >= 0) & (to < lens)
        kept = torch.where(cut, to, lens)
        given = (j >= ((kept + page - 1) // page)[:, None]) & (j < ((lens + page - 1) // page)[:, None])
        given &= table >= 0
        refs.index_add_(0, table.clamp(min=0).flatten().long(), -given.flatten().int())
        table.masked_fill_(given, -1)
        lens.copy_(kept)
        n = add.clamp(min=0).long()
        ends = n.cumsum(0)
        held, want = (lens + page - 1) // page, (lens + n + page - 1) // page
        last = table.gather(1, (lens // page).clamp(max=width - 1).long()[:, None])[:, 0]
        alone = (lens % page == 0) | ((last >= 0) & (refs[last.clamp(min=0).long()] == 1))
        ok = (n > 0) & (lens + n <= width * page) & (ends <= slots) & alone
        need = torch.where(ok, want - held, 0)
        upto = need.cumsum(0)
        free = refs <= 0
        ranks = free.cumsum(0)                                                    # free pages up to each
        ok &= (need == 0) | (upto <= ranks[-1])
        need = torch.where(ok, need, 0)
        new = ok[:, None] & (j >= held[:, None]) & (j < want[:, None])
        at = (upto - need)[:, None] + j - held[:, None]
        pages = torch.searchsorted(ranks, torch.where(new, at, 0) + 1)
        table.copy_(torch.where(new, pages.int(), table))
        refs.masked_fill_(free & (ranks <= need.sum()), 1)
        i = torch.arange(slots, device="cuda")
        row = torch.searchsorted(ends, i, right=True)
        inside = row < n.numel()
        row = row.clamp(max=n.numel() - 1)
        inside &= ok[row]
        seqs = torch.where(inside, row, -1).int()
        positions = torch.where(inside, lens[row] + i - (ends - n)[row], -1).int()
        granted = torch.where(ok, n, 0).int()
        lens.add_(granted)
    return {"granted": granted, "seqs": seqs, "positions": positions, "table": table, "lens": lens, "refs": refs}


def _rotated(x, positions, freqs, weight, interleaved):
    """Heads [count, heads, D] normed (if there are weights) and rotated, in fp32 with angles in 64 bits."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    angle = positions.double()[:, None] * freqs
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    half = freqs.numel()
    part, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :half], part[..., half:])
    a, b = a * cos - b * sin, b * cos + a * sin
    part = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((part, rest), -1).half()


def _run_rope(s):
    c = s["case"]
    heads, kv_heads, dim, page = c["heads"], c["kv_heads"], c["dim"], c["page"]
    q, k, v = s["qkv"].split([heads * dim, kv_heads * dim, kv_heads * dim], 1)
    if own:
        import dequant_gemv_q4g32_amd as qg
        if "rotary" not in s:
            s["rotary"] = qg.Rotary(dim, s["freqs"], interleaved=c["interleaved"], q_weight=s["q_weight"],
                                    k_weight=s["k_weight"], eps=1e-6)
        if not c["cache"]:
            q, k = qg.qk_rope(s["rotary"], q, k, s["positions"])
            return {"q": q, "k": k}
        _, kv = _handle(s, c["cache"], kv_heads, dim)
        q = qg.kv_append_rope(kv, s["table"], s["rotary"], q, k, v, s["positions"], s["seqs"])
        if c["cache"] == "f16":
            return {"q": q, "pool": s["pool"].view(torch.float16)}
        k, v = qg.kv_gather(kv, s["table"], s["positions"], s["seqs"])
        return {"q": q, "k": k, "v": v}
    q = _rotated(q.unflatten(1, (-1, dim)), s["positions"], s["freqs"], s["q_weight"], c["interleaved"])
    k = _rotated(k.unflatten(1, (-1, dim)), s["positions"], s["freqs"], s["k_weight"], c["interleaved"])
    if not c["cache"]:
        return {"q": q.flatten(1), "k": k.flatten(1)}
    v = v.unflatten(1, (-1, dim))
    pos = s["positions"].long()
    at, off = s["table"][s["seqs"].long(), pos // page].long(), pos % page
    parts = _parts(s["pool"], c["cache"], kv_heads, dim, page)
    if c["cache"] == "f16":
        parts[0][at, :, off] = k
        parts[1][at, :, off] = v
        return {"q": q.flatten(1), "pool": s["pool"].view(torch.float16)}
    (kc, ks), (vc, vs) = _encode(k), _encode(v)
    parts[0][at, :, off] = kc
    parts[1][at, :, off] = vc
    parts[2][at, :, off] = ks
    parts[3][at, :, :, off] = vs
    k, v = _decode(parts[0][at, :, off], parts[2][at, :, off]), _decode(parts[1][at, :, off], parts[3][at, :, :, off])
    return {"q": q.flatten(1), "k": k.half().flatten(1), "v": v.half().flatten(1)}


def _entries(s, at):
    """Cached K and V of the pages `at` [n, pages], fp32 [n, kv heads, tokens, dim]."""
    c = s["case"]
    parts = _parts(s["pool"], c["kind"], c["kv_heads"], c["dim"], c["page"])
    if c["kind"] == "f16":
        k, v = (p[at].float() for p in parts)
    else:
        k, v = _decode(parts[0][at], parts[2][at]), _decode(parts[1][at], parts[3][at].transpose(-1, -2))
    return (x.transpose(1, 2).flatten(2, 3) for x in (k, v))


def _run_prefix(s):
    c = s["case"]
    scale, most = 1.0 / math.sqrt(c["dim"]), max(_shape(c)[2])
    if own:
        qg, kv = _handle(s, c["kind"], c["kv_heads"], c["dim"])
        out, lse = qg.prefix_attention(kv, s["q"], s["table"], s["lens"], s["starts"], s["prefix"], max_len=most,
                                       max_tail=c["tail"], scale=scale, out_f32=c["f32"], return_lse=True)
        return {"out": out, "lse": lse}
    page, kv_heads, dim = c["page"], c["kv_heads"], c["dim"]
    table, lens, prefix = s["table"], s["lens"].long(), s["prefix"].long()
    group, rank, heads = s["group"], s["rank"], c["heads"] // c["kv_heads"]
    # the prefixes, once a group: whole pages of its first row
    first = s["starts"][:-1].long()
    whole = torch.minimum(prefix, lens[first]) // page
    pages = max(1, c["prefix"] // page)
    k, v = _entries(s, table[first, :pages].clamp(min=0).long())
    q = s["q"].float().unflatten(1, (kv_heads, heads))
    together = q.new_zeros((first.numel(), kv_heads, s["most"], heads, dim))
    together[group, :, rank] = q
    j = torch.arange(k.shape[2], device="cuda")
    score = torch.matmul(together.flatten(2, 3), k.transpose(-1, -2).contiguous()) * scale
    score = score.unflatten(2, (s["most"], heads))[group, :, rank]                # [rows, kv heads, heads, tokens]
    seen = j < torch.minimum(lens, whole[group] * page)[:, None]
    score = torch.where(seen[:, None, None], score, -math.inf)
    # each row's own tokens
    at = whole[group][:, None] + torch.arange(-(-(c["tail"] + page) // page), device="cuda")
    kt, vt = _entries(s, table.gather(1, at.clamp(max=table.shape[1] - 1)).clamp(min=0).long())
    j = whole[group][:, None] * page + torch.arange(kt.shape[2], device="cuda")
    tail = torch.matmul(q, kt.transpose(-1, -2).contiguous()) * scale
    tail = torch.where((j < lens[:, None])[:, None, None], tail, -math.inf)
    top = torch.maximum(score.amax(-1, keepdim=True), tail.amax(-1, keepdim=True))
    top = torch.where(top > -math.inf, top, 0.0)
    score, tail = torch.exp(score - top), torch.exp(tail - top)
    total = score.sum(-1, keepdim=True) + tail.sum(-1, keepdim=True)
    weights = score.new_zeros((first.numel(), kv_heads, s["most"], heads, score.shape[-1]))
    weights[group, :, rank] = score
    out = torch.matmul(weights.flatten(2, 3), v).unflatten(2, (s["most"], heads))[group, :, rank] + torch.matmul(tail, vt)
    out = (out / torch.where(total > 0, total, 1.0)).flatten(1, 2)
    lse = (top + torch.log(total)).flatten(1)
    return {"out": out if c["f32"] else out.half(), "lse": lse}


def run(state):
    return {"extend": _run_extend, "rope": _run_rope, "prefix": _run_prefix}[state["case"]["op"]](state)


# ---- the same from the definitions, in 64 bits ----------------------------------------------

def _cached(s, page_ids, offs):
    """The fp16 values (in fp64) of K and V at (page, offset) pairs: two tensors [n, kv heads, dim]."""
    c = s["case"]
    flat = s["pool"].reshape(s["pool"].shape[0], c["kv_heads"], -1)
    td, heads = c["page"] * c["dim"], torch.arange(c["kv_heads"], device="cuda")[None, :, None]
    at, off = page_ids[:, None, None], offs[:, None, None]
    d = torch.arange(c["dim"], device="cuda")[None, None, :]
    got = []
    for which in (0, 1):
        if c["kind"] == "f16":
            got.append(flat.view(torch.float16)[at, heads, which * td + off * c["dim"] + d].double())
            continue
        code = flat.view(torch.int8)[at, heads, which * td + off * c["dim"] + d].double()
        groups = c["dim"] // GROUP
        place = off * groups + d // GROUP if which == 0 else c["page"] * groups + (d // GROUP) * c["page"] + off
        x = code * flat.view(torch.float16)[at, heads, td + place].double()
        got.append(x.clamp(-FP16_MAX, FP16_MAX).half().double())
    return got


def _held(x):
    """fp16 [n, heads, D] as int8 groups of 32 hold them, in fp64."""
    x = x.double().unflatten(-1, (-1, GROUP))
    t = x.abs().amax(-1, keepdim=True) / 127
    unit = torch.exp2(torch.floor(torch.log2(t.clamp(min=2.0 ** -14))) - 10)      # spacing of fp16 numbers at t
    d = torch.ceil(t / unit) * unit
    return (torch.round(x / d.clamp(min=2.0 ** -24)) * d).clamp(-FP16_MAX, FP16_MAX).half().double().flatten(-2)


def _exact_rope(case, s):
    dim, half = case["dim"], case["rot"] // 2
    x = s["qkv"].double().unflatten(1, (-1, dim))
    q, k, v = x.split([case["heads"], case["kv_heads"], case["kv_heads"]], 1)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["positions"].double()[:, None, None] * s["freqs"])
    got = []
    for x, weight in ((q, s["q_weight"]), (k, s["k_weight"])):
        if weight is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.double()
        y = x.clone()
        at = torch.arange(half, device="cuda")
        i, j = (2 * at, 2 * at + 1) if case["interleaved"] else (at, at + half)
        z = torch.complex(x[..., i], x[..., j]) * turn
        y[..., i], y[..., j] = z.real, z.imag
        got.append(y)
    q, k = got
    if not case["cache"]:
        return {"q": q.flatten(1), "k": k.flatten(1)}
    if case["cache"] == "q8":
        return {"q": q.flatten(1), "k": _held(k.half()).flatten(1), "v": _held(v).flatten(1)}
    pool = s["pool"].view(torch.float16).double()
    part = pool.view(pool.shape[0], case["kv_heads"], 2, case["page"], dim)
    page = s["table"][s["seqs"].long(), s["positions"].long() // case["page"]].long()
    part[page, :, :, s["positions"].long() % case["page"]] = torch.stack((k, v), 2)
    return {"q": q.flatten(1), "pool": pool}


def exact(case, seed):
    if case["op"] == "extend":
        return None                                       # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    out = torch.zeros((case["rows"], case["heads"], case["dim"]), dtype=torch.float64, device="cuda")
    lse = torch.full((case["rows"], case["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    group, page = case["heads"] // case["kv_heads"], case["page"]
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        j = torch.arange(n, device="cuda")
        k, v = _cached(s, s["table"][b, j // page].long(), j % page)
        for h in range(case["kv_heads"]):
            q = s["q"][b, h * group:(h + 1) * group].double()
            w = q @ k[:, h].T.contiguous() / math.sqrt(case["dim"])
            z = torch.logsumexp(w, -1)
            out[b, h * group:(h + 1) * group] = torch.exp(w - z[:, None]) @ v[:, h].contiguous()
            lse[b, h * group:(h + 1) * group] = z
    return {"out": out, "lse": lse}


def work(case):
    if case["op"] == "extend":
        rows, page = case["rows"], case["page"]
        moved = rows * (case["reject"] + 1) + case["prompts"] * case["prompt"] // 2
        return {"bytes": 4 * case["pages"] + 28 * rows + 8 * case["slots"] + 8 * (moved // page), "flops": 0}
    kv_heads, dim, page, heads = case["kv_heads"], case["dim"], case["page"], case["heads"]
    kind = case["cache"] if case["op"] == "rope" else case["kind"]
    token = kv_heads * (2 * dim + 4 * (dim // GROUP) if kind == "q8" else 4 * dim)
    if case["op"] == "rope":
        count = case["batch"] * case["new"]
        read = 2 * dim * (heads + (2 if kind else 1) * kv_heads)
        write = 2 * dim * heads + (token if kind else 2 * dim * kv_heads)
        back = token + 4 * dim * kv_heads if kind == "q8" else 0
        return {"bytes": count * (read + write + back + 12), "flops": count * (heads + kv_heads) * dim * (3 + 4 * case["norm"])}
    sizes, prefixes, lens = _shape(case)
    at, cached, products = 0, 0, sum(lens)
    for n, p in zip(sizes, prefixes):
        mine = lens[at:at + n]
        shared = min(p, max(mine))
        cached += shared + sum(max(0, x - shared) for x in mine)
        at += n
    bytes_ = cached * token + case["rows"] * heads * (dim * (2 + (4 if case["f32"] else 2)) + 4) + 4 * (cached // page + case["rows"])
    return {"bytes": bytes_, "flops": 4 * products * heads * dim}
