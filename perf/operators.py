"""Cases and plain forms of the paged KV-cache operators.

A pool of pages is a uint8 tensor [layers, pages, page bytes]. A page holds `page` tokens of
every KV head; the part of one head (T tokens, D elements a token) is, in this order,

  q8    K codes int8 [T][D], V codes int8 [T][D], K scales fp16 [T][D/32], V scales fp16 [D/32][T]
  f16   K fp16 [T][D], V fp16 [T][D]

A q8 element stands for code * scale, rounded once to fp16 and saturated at +-65504. `table`
(int32 [sequences, pages a sequence], -1 for none) maps a sequence's tokens to pages, `lens`
(int32) holds the sequences' lengths and `refs` (int32) how many sequences hold a page.
"""
import functools
import math
import random

import torch

own = False

GROUP = 32
FP16_MAX = 65504.0


# ---- cases -----------------------------------------------------------------------------

def _attn(name, kind, batch, heads, kv_heads, dim, page, max_len, ragged, window=0, f32=False):
    return {"name": name, "op": "attention", "kind": kind, "batch": batch, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "page": page, "max_len": max_len, "ragged": ragged, "window": window, "f32": f32}


def _rows(name, op, kind, batch, new, past, kv_heads, dim, page):
    return {"name": name, "op": op, "kind": kind, "batch": batch, "new": new, "past": past, "kv_heads": kv_heads,
            "dim": dim, "page": page}


def _pages(name, op, kind, layers, kv_heads, dim, page, pages, rows, count):
    return {"name": name, "op": op, "kind": kind, "layers": layers, "kv_heads": kv_heads, "dim": dim, "page": page,
            "pages": pages, "rows": rows, "count": count}


def listed():
    return [
        # one chat turn of a single user, cache of a thousand tokens: latency
        _attn("attn_q8_1x1000", "q8", 1, 32, 8, 128, 16, 1000, False),
        # a served batch of a 7B-like model (32 heads, 8 KV heads of 128), each sequence of its own length
        _attn("attn_q8_32x8192_ragged", "q8", 32, 32, 8, 128, 16, 8192, True),
        # the same layer of a 70B-like model (64 heads, 8 KV heads) with an fp16 cache, full batch: the largest
        _attn("attn_f16_64x8192", "f16", 64, 64, 8, 128, 64, 8192, False),
        # one very long document: all parallelism has to come from the cache's length
        _attn("attn_q8_1x131072", "q8", 1, 64, 8, 128, 32, 131072, False),
        # no shared KV heads, head size 64, a sliding window, a batch of odd size
        _attn("attn_f16_mha64_window", "f16", 37, 12, 12, 64, 32, 4001, True, window=1025),
        # one KV head for all heads, head size 256, fp32 output
        _attn("attn_q8_mqa256_f32", "q8", 48, 16, 1, 256, 128, 6007, True, f32=True),
        # one decode step's tokens of 64 sequences written to the cache, and read back as later steps see them
        _rows("append_q8_decode64", "append", "q8", 64, 1, 1500, 8, 128, 16),
        # a prefill chunk of 2048 tokens after 6144 cached ones: written, then the whole prefix read dense
        _rows("append_q8_chunk2048", "append", "q8", 1, 2048, 6144, 8, 128, 16),
        # beams of one 16-layer cache part exchanged: the losers are freed, the winners forked in their place
        _pages("beams_f16_16layers", "beams", "f16", 16, 8, 128, 16, 600, 16, 8),
        # duplicating the pages of preempted or branched sequences in every layer
        _pages("copy_f16_8layers", "copy", "f16", 8, 8, 128, 32, 640, 0, 256),
        # a fragmented small pool and a fragmented large one moved together, so that the tail can be given back
        _pages("compact_f16_small", "compact", "f16", 2, 2, 64, 16, 301, 9, 0),
        _pages("compact_f16_32layers", "compact", "f16", 32, 8, 128, 16, 1000, 24, 0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["q8", "f16"])
    dim = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    op = rng.choice(["attention", "attention", "attention", "append", "beams", "copy", "compact"])
    if op == "attention":
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16, 20])
        batch, max_len = _log(rng, 1, 256), _log(rng, 1, 131072)
        # no more cached elements than the largest listed case
        most = 64 * 8192 * 8 * 128
        max_len = max(1, min(max_len, most // (batch * kv_heads * dim)))
        while batch * max_len * kv_heads * group > 64 * 8192 * 64:
            group = group // 2
        window = 0 if rng.random() < 0.7 else rng.randint(1, max_len)
        return {k: v for k, v in _attn("", kind, batch, kv_heads * group, kv_heads, dim, page, max_len, rng.random() < 0.6,
                                       window, rng.random() < 0.3).items() if k != "name"}
    if op == "append":
        batch = _log(rng, 1, 128)
        new = 1 if rng.random() < 0.5 else _log(rng, 1, max(1, 4096 // batch))
        past = _log(rng, 1, max(1, 16384 // batch))
        return {k: v for k, v in _rows("", op, kind, batch, new, past, kv_heads, dim, page).items() if k != "name"}
    layers, rows = _log(rng, 1, 32), _log(rng, 2, 64)
    per_page = kv_heads * page * dim * 4
    pages = max(4 * rows, min(_log(rng, 256, 4096), (2 << 30) // (per_page * layers)))
    layers = max(1, min(layers, (2 << 30) // (per_page * pages)))
    count = {"beams": rng.randint(1, max(1, rows // 2)), "copy": rng.randint(1, pages // 2), "compact": 0}[op]
    return {k: v for k, v in _pages("", op, "f16", layers, kv_heads, dim, page, pages, 0 if op == "copy" else rows,
                                    count).items() if k != "name"}


def _lens(case):
    """The lengths of a case's sequences. They belong to the case; a seed only orders them."""
    batch, most = case["batch"], case["max_len"]
    if not case["ragged"]:
        return [most] * batch
    r = random.Random(batch * 1000003 + most)
    lens = [max(1, int(most * r.random() ** 1.5)) for _ in range(batch)]
    lens[0] = most
    if batch > 4:
        lens[1] = 0                       # a padded place of the batch
        lens[2] = 1
    return lens


# ---- pools -----------------------------------------------------------------------------

def _page_bytes(kind, kv_heads, dim, page):
    return kv_heads * page * (4 * dim if kind == "f16" else 2 * dim + 4 * (dim // GROUP))


def _parts(pool, kind, kv_heads, dim, page):
    """Views of one layer's pool [pages, page bytes]: (K, V) or (K codes, V codes, K scales, V scales)."""
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


def _keys(shape, gen):
    """Cached entries: centred, channels of different size, a few large ones."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float16)
    size = torch.rand(shape[-1], generator=gen, device="cuda") * 1.2 + 0.3
    return x * size.half()


def _fill(pool, kind, kv_heads, dim, page, gen):
    step = max(1, (1 << 26) // (kv_heads * dim * page))
    for at in range(0, pool.shape[0], step):
        part = _parts(pool[at:at + step], kind, kv_heads, dim, page)
        for i in (0, 1):
            x = _keys((min(step, pool.shape[0] - at), kv_heads, page, dim), gen)
            if kind == "f16":
                part[i].copy_(x)
            else:
                codes, scales = _encode(x)
                part[i].copy_(codes)
                part[2 + i].copy_(scales if i == 0 else scales.transpose(-1, -2))


def _table(lens, page, spare, gen, width):
    """A page table [sequences, width] of distinct pages in random order, and the pool's number of pages."""
    held = [-(-n // page) for n in lens]
    pages = sum(held) + spare
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(held):
        table[i, :n] = order[at:at + n]
        at += n
    return table, pages, order[at:]


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    kv_heads, dim, page, kind = case["kv_heads"], case["dim"], case["page"], case["kind"]
    size = _page_bytes(kind, kv_heads, dim, page)
    op = case["op"]
    ints = functools.partial(torch.tensor, dtype=torch.int32, device="cuda")
    if op == "attention":
        lens = _lens(case)
        random.Random(seed).shuffle(lens)
        table, pages, _ = _table(lens, page, 3, gen, -(-case["max_len"] // page))
        pool = torch.empty((1, pages, size), dtype=torch.uint8, device="cuda")
        _fill(pool[0], kind, kv_heads, dim, page, gen)
        q = torch.randn((case["batch"], case["heads"], dim), generator=gen, device="cuda") * 1.5
        return {"case": case, "pool": pool, "table": table, "lens": ints(lens), "q": q.half()}
    if op == "append":
        lens = [case["past"] + case["new"]] * case["batch"]
        table, pages, _ = _table(lens, page, 3, gen, -(-lens[0] // page))
        pool = torch.empty((1, pages, size), dtype=torch.uint8, device="cuda")
        _fill(pool[0], kind, kv_heads, dim, page, gen)
        rows = torch.arange(case["batch"], device="cuda", dtype=torch.int32)
        # what a step reads back: the prefix with the new chunk, or the new tokens alone
        first = case["past"] if case["new"] == 1 else 0
        new = torch.arange(case["past"], lens[0], device="cuda", dtype=torch.int32)
        back = torch.arange(first, lens[0], device="cuda", dtype=torch.int32)
        shape = (case["batch"] * case["new"], kv_heads * dim)
        k, v = (_keys((shape[0], kv_heads, dim), gen).view(shape) for _ in (0, 1))
        return {"case": case, "pool": pool, "table": table, "k": k, "v": v,
                "seqs": rows.repeat_interleave(new.numel()), "positions": new.repeat(case["batch"]),
                "back_seqs": rows.repeat_interleave(back.numel()), "back": back.repeat(case["batch"])}
    layers, pages = case["layers"], case["pages"]
    pool = torch.empty((layers, pages, size), dtype=torch.uint8, device="cuda")
    for layer in range(layers):
        _fill(pool[layer], kind, kv_heads, dim, page, gen)
    r = random.Random(seed)
    if op == "copy":
        order = torch.randperm(pages, generator=gen, device="cuda").int()
        return {"case": case, "pool": pool, "src": order[:case["count"]].contiguous(),
                "dst": order[pages // 2:pages // 2 + case["count"]].contiguous()}
    held = max(1, (pages - case["count"]) * 2 // 3 // case["rows"])     # pages a sequence holds at most
    lens = [r.randint((held - 1) * page + 1, held * page) for _ in range(case["rows"])]
    table, _, free = _table(lens, page, pages - sum(-(-n // page) for n in lens), gen, held + 2)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[table[table >= 0].long()] = 1
    state = {"case": case, "pool": pool, "table": table, "lens": ints(lens), "refs": refs}
    if op == "beams":
        who = r.sample(range(case["rows"]), 2 * case["count"])
        state["src"], state["dst"] = ints(who[:case["count"]]), ints(who[case["count"]:])
        state["new"] = free[:case["count"]].contiguous()
    return state


# ---- the operators -----------------------------------------------------------------------

def _handle(state):
    """The framework's handle of the pool, which a program makes once and keeps."""
    import dequant_gemv_q4g32_amd as qg
    if "handle" not in state:
        c = state["case"]
        state["handle"] = qg.KVPool(state["pool"], c["kind"], c["kv_heads"], c["dim"], c["page"])
    return qg, state["handle"]


def _attention(s):
    c = s["case"]
    scale = 1.0 / math.sqrt(c["dim"])
    if own:
        qg, kv = _handle(s)
        out, lse = qg.paged_attention(kv, s["q"], s["table"], s["lens"], max_len=c["max_len"], scale=scale,
                                      window=c["window"], out_f32=c["f32"], return_lse=True)
        return {"out": out, "lse": lse}
    parts = _parts(s["pool"][0], c["kind"], c["kv_heads"], c["dim"], c["page"])
    at = s["table"].clamp(min=0).long()
    if c["kind"] == "f16":
        k, v = (p[at].float() for p in parts)                                   # [batch, pages, kv heads, page, dim]
    else:
        k = _decode(parts[0][at], parts[2][at])
        v = _decode(parts[1][at], parts[3][at].transpose(-1, -2))
    k, v = (x.transpose(1, 2).flatten(2, 3) for x in (k, v))                    # [batch, kv heads, tokens, dim]
    q = s["q"].float().unflatten(1, (c["kv_heads"], -1))
    score = torch.matmul(k, q.transpose(-1, -2).contiguous()).transpose(-1, -2) * scale
    j, n = torch.arange(k.shape[2], device="cuda"), s["lens"][:, None]
    seen = (j < n) & (j >= n - c["window"]) if c["window"] else j < n
    seen = seen[:, None, None, :]
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total)).flatten(1)
    out = out.flatten(1, 2)
    return {"out": out if c["f32"] else out.half(), "lse": lse}


def _append(s):
    c = s["case"]
    if own:
        qg, kv = _handle(s)
        qg.kv_append(kv, s["table"], s["k"], s["v"], s["positions"], s["seqs"])
        k, v = qg.kv_gather(kv, s["table"], s["back"], s["back_seqs"])
        return {"k": k, "v": v}
    parts = _parts(s["pool"][0], c["kind"], c["kv_heads"], c["dim"], c["page"])
    pos = s["positions"].long()
    at, off = s["table"][s["seqs"].long(), pos // c["page"]].long(), pos % c["page"]
    for i, x in enumerate((s["k"], s["v"])):
        x = x.unflatten(-1, (c["kv_heads"], c["dim"]))
        if c["kind"] == "f16":
            parts[i][at, :, off] = x
        else:
            codes, scales = _encode(x)
            parts[i][at, :, off] = codes
            if i == 0:
                parts[2][at, :, off] = scales
            else:
                parts[3][at, :, :, off] = scales
    pos = s["back"].long()
    at, off = s["table"][s["back_seqs"].long(), pos // c["page"]].long(), pos % c["page"]
    if c["kind"] == "f16":
        k, v = (p[at, :, off] for p in parts)
    else:
        k = _decode(parts[0][at, :, off], parts[2][at, :, off]).half()
        v = _decode(parts[1][at, :, off], parts[3][at, :, :, off]).half()
    return {"k": k.flatten(1), "v": v.flatten(1)}


def _values(s):
    return s["pool"].view(torch.float16)


def _copy(s):
    if own:
        qg, kv = _handle(s)
        qg.kv_copy_pages(kv, s["src"], s["dst"])
    else:
        s["pool"][:, s["dst"].long()] = s["pool"][:, s["src"].long()]
    return {"pool": _values(s)}


def _beams(s):
    table, lens, refs, page = s["table"], s["lens"], s["refs"], s["case"]["page"]
    if own:
        qg, kv = _handle(s)
        qg.kv_free(kv, table, lens, refs, s["dst"])
        qg.kv_fork(kv, table, lens, refs, s["src"], s["dst"], s["new"])
    else:
        src, dst, new = s["src"].long(), s["dst"].long(), s["new"].long()
        j = torch.arange(table.shape[1], device="cuda")
        held = (lens[dst, None] + page - 1) // page > j
        refs.index_add_(0, table[dst].clamp(min=0).flatten().long(), -held.flatten().int())
        n = lens[src]
        whole, rest = n // page, n % page > 0
        row = table[src]
        shared = j < whole[:, None]
        refs.index_add_(0, row.clamp(min=0).flatten().long(), shared.flatten().int())
        tail = row.gather(1, whole.clamp(max=row.shape[1] - 1).long()[:, None])[:, 0].long()
        tail = torch.where(rest, tail, new)
        refs[new] = torch.where(rest, 1, refs[new])
        s["pool"][:, new] = s["pool"][:, tail]
        is_tail = (j == whole[:, None]) & rest[:, None]
        table[dst] = torch.where(shared, row, torch.where(is_tail, s["new"][:, None], -1))
        lens[dst] = n
    return {"pool": _values(s), "table": table, "lens": lens, "refs": refs}


def _compact(s):
    if own:
        qg, kv = _handle(s)
        table, refs, remap, live = qg.kv_compact(kv, s["table"], s["refs"])
    else:
        held = s["refs"] > 0
        n = held.sum()
        j = torch.arange(held.numel(), device="cuda")
        src = torch.nonzero(held & (j >= n))[:, 0]
        dst = torch.nonzero(~held & (j < n))[:, 0]
        s["pool"][:, dst] = s["pool"][:, src]
        remap = torch.where(held, j, -1)
        remap[src] = dst
        refs = s["refs"].clone()
        refs[dst] = s["refs"][src]
        refs[src] = 0
        table = torch.where(s["table"] >= 0, remap[s["table"].clamp(min=0).long()], -1).int()
        remap, live = remap.int(), n.int().view(1)
    return {"pool": _values(s), "table": table, "refs": refs, "remap": remap, "live": live}


def run(state):
    return {"attention": _attention, "append": _append, "copy": _copy, "beams": _beams,
            "compact": _compact}[state["case"]["op"]](state)


# ---- the same from the definitions, in 64 bits ----------------------------------------------

def _cached(s, page_ids, offs):
    """The fp16 values (in fp64) of K and V at (page, offset) pairs: two tensors [n, kv heads, dim]."""
    c = s["case"]
    flat = s["pool"][0].reshape(s["pool"].shape[1], c["kv_heads"], -1)
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


def exact(case, seed):
    op = case["op"]
    if op in ("copy", "beams", "compact"):
        return None                                       # values are moved, none is computed
    s = prepare(case, seed)
    page = case["page"]
    if op == "append":
        k, v = torch.zeros((2, s["back"].numel(), case["kv_heads"], case["dim"]), dtype=torch.float64, device="cuda")
        most = 4096
        for at in range(0, k.shape[0], most):
            pos, seq = s["back"][at:at + most].long(), s["back_seqs"][at:at + most].long()
            k[at:at + most], v[at:at + most] = _cached(s, s["table"][seq, pos // page].long(), pos % page)
        per_seq = s["back"].numel() // case["batch"]
        rows = s["seqs"].long() * per_seq + s["positions"].long() - s["back"][0].long()
        for new, old in ((s["k"], k), (s["v"], v)):
            if case["kind"] == "f16":
                old[rows] = new.double().view(new.shape[0], case["kv_heads"], -1)
                continue
            x = new.double().view(new.shape[0], case["kv_heads"], -1, GROUP)
            t = x.abs().amax(-1, keepdim=True) / 127
            e = torch.floor(torch.log2(t.clamp(min=2.0 ** -14)))
            unit = torch.exp2(e - 10)                     # spacing of fp16 numbers at t
            d = torch.ceil(t / unit) * unit
            x = torch.round(x / d.clamp(min=2.0 ** -24)) * d
            old[rows] = x.clamp(-FP16_MAX, FP16_MAX).half().double().flatten(2)
        return {"k": k.flatten(1), "v": v.flatten(1)}
    out = torch.zeros((case["batch"], case["heads"], case["dim"]), dtype=torch.float64, device="cuda")
    lse = torch.full((case["batch"], case["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    group = case["heads"] // case["kv_heads"]
    for b, n in enumerate(s["lens"].tolist()):
        first = max(0, n - case["window"]) if case["window"] else 0
        if n <= first:
            continue
        j = torch.arange(first, n, device="cuda")
        k, v = _cached(s, s["table"][b, j // page].long(), j % page)
        for h in range(case["kv_heads"]):
            q = s["q"][b, h * group:(h + 1) * group].double()
            w = q @ k[:, h].T.contiguous() / math.sqrt(case["dim"])
            z = torch.logsumexp(w, -1)
            out[b, h * group:(h + 1) * group] = torch.exp(w - z[:, None]) @ v[:, h].contiguous()
            lse[b, h * group:(h + 1) * group] = z
    return {"out": out, "lse": lse}


def work(case):
    kv_heads, dim, page = case["kv_heads"], case["dim"], case["page"]
    token = kv_heads * (4 * dim if case["kind"] == "f16" else 2 * dim + 4 * (dim // GROUP))
    op = case["op"]
    if op == "attention":
        tokens = sum(min(n, case["window"]) if case["window"] else n for n in _lens(case))
        rows = case["batch"] * case["heads"]
        bytes_ = tokens * token + rows * (dim * (2 + (4 if case["f32"] else 2)) + 4) + 4 * (tokens // page + case["batch"])
        return {"bytes": bytes_, "flops": 4 * tokens * case["heads"] * dim}
    if op == "append":
        new = case["batch"] * case["new"]
        back = new if case["new"] == 1 else case["batch"] * (case["past"] + case["new"])
        dense = 4 * kv_heads * dim
        return {"bytes": (new + back) * (dense + token + 8), "flops": 2 * kv_heads * dim * (new + back)}
    size = 2 * case["layers"] * page * token
    if op == "copy":
        return {"bytes": case["count"] * (size + 8), "flops": 0}
    held = max(1, (case["pages"] - case["count"]) * 2 // 3 // case["rows"])
    if op == "beams":
        return {"bytes": case["count"] * (size + 8 * held * 3), "flops": 0}
    live = held * case["rows"]
    moved = live * (case["pages"] - live) // case["pages"]                     # pages past the live count, on average
    return {"bytes": moved * size + 8 * case["pages"] + 8 * live, "flops": 0}
