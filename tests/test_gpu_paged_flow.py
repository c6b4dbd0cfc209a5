"""GPU tests of the paged-cache operators as they are used together and where they could get in
each other's way: a decoding run with branches, ends and compaction against the oracle; both
ways the attention shares out its work; graphs that are replayed while the cache changes; streams;
two graphs at once; the binding's refusals."""
import ctypes

import numpy as np
import pytest

import dequant_gemv_q4g32_amd as qg
from oracle import paged

from paged_util import assert_same_bytes, attention_tolerance, check_attention, dev, download, random_cache, random_table, upload

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


# ---- a decoding run ------------------------------------------------------------------------------

@pytest.mark.parametrize("kind,heads,kv_heads,dim,tokens,layers", [("q8", 8, 2, 64, 16, 2), ("f16", 6, 3, 128, 32, 1),
                                                                   ("q8", 4, 1, 256, 16, 1)])
def test_decoding_run(kind, heads, kv_heads, dim, tokens, layers):
    """Prompts are appended, then tokens one at a time with attention after each; rows fork, grow
    apart and end, the pool is compacted in the middle. Host and oracle keep the same tables; every
    byte of the pool and every output is compared."""
    rng = np.random.default_rng(dim + tokens)
    rows, width, pages, cols = 5, 8, 30, kv_heads * dim
    c = random_cache(kind, layers, pages, kv_heads, dim, tokens, 3, poison=True)
    pool = upload(c)
    table = np.full((rows, width), -1, np.int32)
    lens, refs = np.zeros(rows, np.int32), np.zeros(pages, np.int32)
    t, n, r = dev(table), dev(lens), dev(refs)

    def push():
        t.copy_(dev(table)), n.copy_(dev(lens)), r.copy_(dev(refs))

    def same(what):
        torch.cuda.synchronize()
        assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(n.cpu().numpy(), lens), what
        assert np.array_equal(r.cpu().numpy(), refs), what
        assert_same_bytes(download(c, pool), c, what)

    def grow(s, count):
        for j in range(int(lens[s]), int(lens[s]) + count):
            if j % tokens == 0:
                free = np.flatnonzero(refs == 0)
                table[s, j // tokens] = free[rng.integers(len(free))]
                refs[table[s, j // tokens]] = 1
        at = np.arange(lens[s], lens[s] + count, dtype=np.int32)
        lens[s] += count
        return at, np.full(count, s, np.int32)

    def append(items):
        pos, seq = (np.concatenate([i[k] for i in items]).astype(np.int32) for k in (0, 1))
        push()
        for layer in range(layers):
            k, v = (rng.standard_normal((len(pos), cols)).astype(np.float16) for _ in range(2))
            qg.kv_append(pool, t, dev(k, np.float16), dev(v, np.float16), dev(pos), dev(seq), layer=layer)
            c.append(layer, table, k, v, pos, seq)

    def attend(what):
        for layer in range(layers):
            q = rng.standard_normal((rows, heads, dim)).astype(np.float16)
            out, lse = qg.paged_attention(pool, dev(q, np.float16), t, n, layer=layer, out_f32=bool(layer), return_lse=True)
            check_attention(out, lse, paged.attention(c, layer, q, table, lens, 10 ** 9, dim ** -0.5), int(lens.max()), dim)
        same(what)

    append([grow(0, 37), grow(1, tokens), grow(2, 5)])
    attend("prompts")
    for step in range(3):
        append([grow(s, 1) for s in (0, 1, 2)])
        attend(f"step {step}")
    spare = np.flatnonzero(refs == 0)[:2].astype(np.int32)
    src, dst = np.array([0, 2], np.int32), np.array([3, 4], np.int32)
    qg.kv_fork(pool, t, n, r, dev(src), dev(dst), dev(spare))
    paged.fork(c, table, lens, refs, src, dst, spare)
    same("fork")
    for step in range(tokens // 2):                       # both branches grow, past a page's end for some
        append([grow(s, 1) for s in (0, 2, 3, 4)])
    attend("branches")
    gone = np.array([0, 1], np.int32)
    qg.kv_free(pool, t, n, r, dev(gone))
    paged.free(c, table, lens, refs, gone)
    same("free")
    qg.kv_compact(pool, t, r, table_out=t, refs_out=r)
    new_table, refs[:], _, live = paged.compact(c, table, refs)
    table[:] = new_table
    same("compact")
    assert np.all(refs[live:] == 0) and np.all(table < live)
    append([grow(s, 3) for s in (0, 3)])
    attend("after")


# ---- the two ways to share out the work --------------------------------------------------------------

WAYS = [  # kind, heads, kv heads, dim, page tokens, lens, window
    ("q8", 32, 8, 128, 16, [1, 15, 16, 17, 31, 32, 33, 0, 200], 0), ("q8", 8, 8, 64, 32, [63, 64, 65, 127, 128, 129], 0),
    ("q8", 16, 1, 256, 128, [257, 300, 1, 0], 0), ("q8", 40, 2, 64, 64, [100, 0, 511], 0), ("q8", 33, 1, 128, 16, [130, 40], 0),
    ("f16", 15, 3, 128, 64, [100, 0, 511, 512, 513], 0), ("f16", 20, 4, 256, 16, [700, 90], 0), ("f16", 48, 1, 64, 32, [333], 0),
    ("q8", 8, 2, 128, 16, [400, 37, 5, 0, 64, 65], 33), ("f16", 8, 2, 64, 16, [400, 37, 5, 0, 64], 1),
    ("f16", 4, 4, 128, 32, [1000, 129, 128, 127], 128)]


@pytest.mark.parametrize("kind,heads,kv_heads,dim,tokens,lens,window", WAYS)
def test_split_and_whole_head_tiles(kind, heads, kv_heads, dim, tokens, lens, window):
    """A long max_len makes the call split its work over all workgroups, a short one gives each
    head tile a workgroup: the same small sequences under both."""
    rng = np.random.default_rng(dim * 3 + len(lens))
    short = -(-max(lens) // tokens)
    wide = 40000 // tokens
    pages = sum(-(-n // tokens) for n in lens) + 1
    c = random_cache(kind, 1, pages, kv_heads, dim, tokens, 5)
    table = random_table(rng, lens, tokens, pages, wide)
    q = (rng.standard_normal((len(lens), heads, dim)) * 1.5).astype(np.float16)
    ref = paged.attention(c, 0, q, table, lens, 10 ** 9, dim ** -0.5, window)
    pool = upload(c)
    assert qg.paged_attention_bytes(pool, len(lens), heads, wide * tokens) > 0
    for max_len in (wide * tokens, short * tokens):
        out, lse = qg.paged_attention(pool, dev(q, np.float16), dev(table), dev(lens), max_len=max_len, window=window,
                                      out_f32=True, return_lse=True)
        check_attention(out, lse, ref, max(lens), dim)


def _torch_reference(k, v, table, lens, q, scale, window):
    """fp64 on the GPU. k, v: fp16 [pages, kv heads, T, D] on the GPU."""
    batch, heads, dim = q.shape
    kv, tokens = k.shape[1], k.shape[2]
    out, bound = torch.zeros((2, batch, heads, dim), dtype=torch.float64, device="cuda")
    lse = torch.full((batch, heads), -float("inf"), dtype=torch.float64, device="cuda")
    reach = torch.zeros((batch, heads), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        first = max(0, n - window) if window else 0
        if n <= first:
            continue
        at = table[b, :-(-n // tokens)].long()
        kb, vb = (x[at].transpose(0, 1).flatten(1, 2)[:, first:n].double().contiguous() for x in (k, v))
        x = q[b].double().view(kv, heads // kv, dim)
        s = torch.matmul(x, kb.transpose(1, 2).contiguous()) * scale
        w = torch.softmax(s, -1)
        out[b] = torch.matmul(w, vb).view(heads, dim)
        bound[b] = torch.matmul(w, vb.abs()).view(heads, dim)
        lse[b] = torch.logsumexp(s, -1).view(heads)
        reach[b] = (torch.matmul(x.abs(), kb.abs().transpose(1, 2).contiguous()).amax(-1) * abs(scale)).view(heads)
    return tuple(t.cpu().numpy() for t in (out, lse, bound, reach))


def _filled(kind, kv_heads, dim, tokens, pages, seed):
    """A pool of random entries and its values as fp16 [pages, kv heads, T, D]."""
    gen = torch.Generator("cuda").manual_seed(seed)
    pool = qg.KVPool.zeros(kind, kv_heads, dim, tokens, pages)
    ids = torch.arange(pages, device="cuda", dtype=torch.int32)[:, None].contiguous()
    place = torch.arange(tokens, device="cuda", dtype=torch.int32).repeat(pages)
    seq = torch.arange(pages, device="cuda", dtype=torch.int32).repeat_interleave(tokens)
    k, v = torch.randn((2, pages * tokens, kv_heads * dim), generator=gen, device="cuda").half()
    qg.kv_append(pool, ids, k, v, place, seq)
    back = qg.kv_gather(pool, ids, place, seq)
    return pool, [x.view(pages, tokens, kv_heads, dim).transpose(1, 2) for x in back], gen


@pytest.mark.parametrize("seed", range(24))
def test_random_batches(seed):
    """Seeded random shapes, types, windows and ragged lengths, from batches that leave most waves
    without work to ones that give a wave parts of several sequences; pages shared at random."""
    rng = np.random.default_rng(1000 + seed)
    kind, dim, tokens = rng.choice(["q8", "f16"]), int(rng.choice([64, 128, 256])), int(rng.choice([16, 32, 64, 128, 256]))
    kv_heads, group = int(rng.choice([1, 2, 3, 5, 8])), int(rng.choice([1, 2, 3, 4, 7, 8, 16, 17, 24]))
    batch = int(rng.choice([1, 2, 5, 17, 60, 300]))
    most = int(np.exp(rng.uniform(0, np.log(max(20, 400000 // (batch * kv_heads))))))
    lens = np.minimum(most, (most * rng.random(batch) ** 1.5).astype(int) + rng.integers(0, 2, batch))
    lens[rng.integers(batch)] = most
    window = int(rng.integers(1, most + 1)) if rng.random() < 0.3 else 0
    pages = min(600, int(sum(-(-lens // tokens))) + 1)
    pool, values, gen = _filled(kind, kv_heads, dim, tokens, pages, seed)
    width = -(-most // tokens) + int(rng.integers(0, 3))
    table = dev(rng.integers(0, pages, (batch, width)))          # sequences may share pages
    q = (torch.randn((batch, group * kv_heads, dim), generator=gen, device="cuda") * 1.5).half()
    f32 = bool(rng.integers(2))
    out, lse = qg.paged_attention(pool, q, table, dev(lens), window=window, out_f32=f32, return_lse=True)
    ref = _torch_reference(*values, table, lens.tolist(), q, dim ** -0.5, window)
    check_attention(out, lse, ref, most, dim)


@pytest.mark.parametrize("seed,batch,kv_heads,group,dim,most", [
    (1, 300, 8, 4, 128, 600), (2, 300, 8, 1, 64, 70), (3, 700, 4, 2, 64, 33), (4, 90, 8, 8, 128, 1500), (5, 257, 3, 17, 128, 480),
    (6, 64, 1, 16, 256, 700), (7, 1000, 8, 1, 64, 500), (8, 31, 16, 2, 128, 5000)])
def test_split_over_many_sequences(seed, batch, kv_heads, group, dim, most):
    """Many sequences under a long max_len, so that a wave's part of the split starts and ends anywhere
    in them: some of one tile, some empty, some longer than a wave's part."""
    rng = np.random.default_rng(seed)
    kind, tokens = ("q8", "f16")[seed % 2], (16, 32, 64)[seed % 3]
    pool, values, gen = _filled(kind, kv_heads, dim, tokens, 200, seed)
    lens = rng.integers(0, most + 1, batch) * (rng.random(batch) < 0.9)
    table = dev(rng.integers(0, 200, (batch, 8192 // tokens)))
    q = (torch.randn((batch, group * kv_heads, dim), generator=gen, device="cuda") * 1.5).half()
    window = 0 if seed % 4 else 100
    out, lse = qg.paged_attention(pool, q, table, dev(lens), window=window, out_f32=True, return_lse=True)
    assert qg.paged_attention_bytes(pool, batch, group * kv_heads, 8192) > 0
    check_attention(out, lse, _torch_reference(*values, table, lens.tolist(), q, dim ** -0.5, window), most, dim)


@pytest.mark.parametrize("kind,batch,kv_heads,group,dim,most,window", [
    ("q8", 300, 2, 4, 128, 130, 0), ("f16", 530, 2, 3, 128, 250, 0), ("q8", 530, 2, 5, 128, 500, 77), ("q8", 260, 1, 16, 256, 500, 0),
    ("f16", 520, 1, 20, 256, 60, 0), ("q8", 520, 2, 1, 64, 100, 0), ("f16", 1100, 4, 2, 64, 40, 9), ("q8", 2100, 1, 3, 128, 1, 0),
    ("f16", 700, 1, 1, 256, 512, 0), ("q8", 1100, 1, 16, 256, 300, 0)])
def test_many_short_sequences(kind, batch, kv_heads, group, dim, most, window):
    """More short sequences than there are workgroups at once, each head tile with one or two waves."""
    rng = np.random.default_rng(batch + dim)
    tokens = int(rng.choice([16, 32, 64]))
    pool, values, gen = _filled(kind, kv_heads, dim, tokens, 300, batch)
    lens = rng.integers(0, most + 1, batch) * (rng.random(batch) < 0.9)
    lens[-1] = most
    table = dev(rng.integers(0, 300, (batch, -(-most // tokens))))
    q = (torch.randn((batch, group * kv_heads, dim), generator=gen, device="cuda") * 1.5).half()
    assert qg.paged_attention_bytes(pool, batch, group * kv_heads, most) == 0
    out, lse = qg.paged_attention(pool, q, table, dev(lens), max_len=most, window=window, out_f32=True, return_lse=True)
    check_attention(out, lse, _torch_reference(*values, table, lens.tolist(), q, dim ** -0.5, window), most, dim)


@pytest.mark.parametrize("kind,batch,kv_heads,group,dim,max_len,most,window", [
    ("q8", 8, 1, 20, 256, 16384, 700, 0), ("f16", 9, 1, 33, 256, 16384, 300, 40), ("q8", 40, 2, 17, 128, 8192, 400, 0),
    ("f16", 33, 3, 71, 128, 8192, 1500, 0), ("q8", 64, 1, 48, 64, 16384, 900, 5000), ("f16", 70, 4, 32, 64, 8192, 250, 0),
    ("q8", 600, 1, 40, 128, 512, 512, 0), ("f16", 700, 1, 33, 64, 512, 200, 70), ("q8", 230, 1, 64, 256, 512, 300, 0),
    ("f16", 200, 1, 45, 256, 512, 512, 0), ("q8", 1100, 1, 18, 64, 512, 90, 0), ("f16", 600, 1, 50, 128, 500, 500, 100)])
def test_more_than_sixteen_heads(kind, batch, kv_heads, group, dim, max_len, most, window):
    """Head tiles of 32 heads, full and ragged, whole and split; lens of all sizes under max_len."""
    rng = np.random.default_rng(batch + group)
    tokens = int(rng.choice([16, 32, 64]))
    pool, values, gen = _filled(kind, kv_heads, dim, tokens, 300, group)
    lens = rng.integers(0, most + 1, batch) * (rng.random(batch) < 0.9)
    lens[0] = most
    table = dev(rng.integers(0, 300, (batch, -(-max_len // tokens))))
    q = (torch.randn((batch, group * kv_heads, dim), generator=gen, device="cuda") * 1.5).half()
    q[1, -1, 3] = float("nan")                       # the last head of a ragged tile
    lens[1] = 33
    out, lse = qg.paged_attention(pool, q, table, dev(lens), max_len=max_len, window=window, out_f32=True, return_lse=True)
    assert torch.all(torch.isnan(out[1, -1])) and torch.isnan(lse[1, -1])
    q[1, -1] = 0
    again, lse2 = qg.paged_attention(pool, q, table, dev(lens), max_len=max_len, window=window, out_f32=True, return_lse=True)
    same = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    same[1, -1] = False
    assert torch.equal(again[same], out[same]) and torch.equal(lse2[same], lse[same])
    check_attention(again, lse2, _torch_reference(*values, table, lens.tolist(), q, dim ** -0.5, window), most, dim)


# ---- graphs ------------------------------------------------------------------------------------------

@pytest.mark.parametrize("kind,max_len", [("q8", 256), ("f16", 8192)])
def test_graph_follows_the_cache(kind, max_len):
    """A captured decode step (append, attention) and page step (free, fork, copy, compact in place),
    replayed while lengths, positions and rows change, with eager work between: every replay equals
    the eager result on the same state."""
    rng = np.random.default_rng(7)
    batch, heads, kv_heads, dim, tokens = 6, 8, 2, 128, 16
    width, pages = max_len // tokens, 120
    lens0 = np.array([20, 1, 100, 0, 63, 0], np.int32)

    def state():
        c = random_cache(kind, 2, pages, kv_heads, dim, tokens, 2)
        table = np.full((batch, width), -1, np.int32)
        table[:, :16] = np.arange(batch * 16).reshape(batch, 16)     # pages for 256 tokens a row
        refs = np.zeros(pages, np.int32)
        refs[:batch * 16] = 1
        s = {"pool": upload(c), "table": dev(table), "lens": dev(lens0), "refs": dev(refs), "pos": dev(lens0 - 1),
             "k": torch.zeros((batch, kv_heads * dim), dtype=torch.float16, device="cuda"),
             "v": torch.zeros((batch, kv_heads * dim), dtype=torch.float16, device="cuda"),
             "q": torch.zeros((batch, heads, dim), dtype=torch.float16, device="cuda"),
             "src": dev([0]), "dst": dev([5]), "new": dev([110]), "cs": dev([3, -1]), "cd": dev([100, 101])}
        return s

    def step(s):
        qg.kv_append(s["pool"], s["table"], s["k"], s["v"], s["pos"], layer=1)
        out, lse = qg.paged_attention(s["pool"], s["q"], s["table"], s["lens"], max_len=max_len, layer=1, return_lse=True)
        qg.kv_free(s["pool"], s["table"], s["lens"], s["refs"], s["dst"])
        qg.kv_fork(s["pool"], s["table"], s["lens"], s["refs"], s["src"], s["dst"], s["new"])
        qg.kv_copy_pages(s["pool"], s["cs"], s["cd"])
        _, _, remap, live = qg.kv_compact(s["pool"], s["table"], s["refs"], table_out=s["table"], refs_out=s["refs"])
        return {"out": out, "lse": lse, "remap": remap, "live": live}

    def feed(s, i):
        r = np.random.default_rng(100 + i)
        for key, scale in (("k", 1), ("v", 1), ("q", 1.5)):
            s[key].copy_(dev(r.standard_normal(tuple(s[key].shape)) * scale, np.float16))
        lens = s["lens"].cpu().numpy().copy()
        grow = r.integers(0, 2, batch).astype(np.int32)
        grow[(lens <= 0) | (lens >= 250) | (np.arange(batch) == 5)] = 0
        # a new page may be needed at a page's end: only rows within their page grow
        grow[lens % tokens == 0] = 0
        lens += grow
        s["lens"].copy_(dev(lens))
        s["pos"].copy_(dev(np.where(grow > 0, lens - 1, -1)))
        s["src"].copy_(dev([i % 3]))
        s["new"].copy_(dev([int(np.flatnonzero(s["refs"].cpu().numpy() == 0)[-1])]))

    eager, graphed = state(), state()
    feed(eager, 0), feed(graphed, 0)
    side = state()
    feed(side, 50)
    step(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(graphed)
    for i in range(1, 6):
        want = step(eager)
        g.replay()
        step(side)                                        # eager work on another pool in between
        torch.cuda.synchronize()
        for key in want:
            assert torch.equal(got[key], want[key]), f"replay {i}: {key}"
        for key in ("table", "lens", "refs"):
            assert torch.equal(graphed[key], eager[key]), f"replay {i}: {key}"
        assert torch.equal(graphed["pool"].pages, eager["pool"].pages), f"replay {i}: pages"
        feed(eager, i), feed(graphed, i)


def test_two_graphs_at_once():
    """Two captured calls on different data, replayed together on two streams: neither's workspace
    is the other's."""
    cases = []
    for seed in (1, 2):
        pool, values, gen = _filled("q8", 8, 128, 16, 400, seed)
        lens = [6000, 333, 40][::1 if seed == 1 else -1]
        rng = np.random.default_rng(seed)
        table = dev(rng.integers(0, 400, (3, 400)))
        q = torch.randn((3, 32, 128), generator=gen, device="cuda").half()
        want = qg.paged_attention(pool, q, table, dev(lens), return_lse=True)
        n = dev(lens)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = qg.paged_attention(pool, q, table, n, return_lse=True)
        cases.append((g, got, want, (pool, table, q, n)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(5):
        for _, got, _, _ in cases:
            got[0].zero_(), got[1].zero_()
        torch.cuda.synchronize()
        for _ in range(4):
            for s, case in zip(streams, cases):
                with torch.cuda.stream(s):
                    case[0].replay()
        torch.cuda.synchronize()
        for _, got, want, _ in cases:
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), rep


def test_streams():
    """Calls on a stream that is passed (a torch stream, its handle) or current, and two at once on
    two streams, equal the default stream's result; what they allocate belongs to the stream."""
    pool, _, gen = _filled("q8", 4, 128, 16, 300, 5)
    rng = np.random.default_rng(5)
    lens, table = dev([4000, 77, 1200]), dev(rng.integers(0, 300, (3, 256)))
    q = torch.randn((3, 16, 128), generator=gen, device="cuda").half()
    pos, seq = dev([5, 70, 900]), dev([0, 1, 2])
    want = qg.paged_attention(pool, q, table, lens, return_lse=True)
    want_rows = qg.kv_gather(pool, table, pos, seq)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for how in (a, a.cuda_stream, 0):
        got = qg.paged_attention(pool, q, table, lens, return_lse=True, stream=how)
        rows = qg.kv_gather(pool, table, pos, seq, stream=how)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got + rows, want + want_rows))
    for rep in range(4):
        with torch.cuda.stream(a):
            x = qg.paged_attention(pool, q, table, lens, return_lse=True)
        y = qg.paged_attention(pool, q, table, lens, return_lse=True, stream=b)
        torch.cuda.synchronize()
        assert all(torch.equal(m, n) for m, n in zip(x + y, want + want))


def test_given_workspace():
    """A workspace of the stated size, with the bytes behind it untouched, whatever it held before."""
    pool, _, gen = _filled("f16", 2, 64, 16, 200, 6)
    rng = np.random.default_rng(6)
    lens, table = dev([2500, 0, 31]), dev(rng.integers(0, 200, (3, 300)))
    q = torch.randn((3, 12, 64), generator=gen, device="cuda").half()
    want = qg.paged_attention(pool, q, table, lens, return_lse=True)
    need = qg.paged_attention_bytes(pool, 3, 12, 300 * 16)
    assert need > 0
    buf = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        got = qg.paged_attention(pool, q, table, lens, return_lse=True, workspace=buf[:need])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.all(buf[need:] == 0xFF)
    with pytest.raises(qg.QGError):
        qg.paged_attention(pool, q, table, lens, workspace=buf[:need - 16])


# ---- refusals ---------------------------------------------------------------------------------------------

def test_binding_refusals():
    pool, _, gen = _filled("q8", 2, 64, 16, 8, 9)
    q = torch.zeros((2, 4, 64), dtype=torch.float16, device="cuda")
    table, lens = dev([[0, 1], [2, 3]]), dev([20, 3])
    rows = torch.zeros((2, 128), dtype=torch.float16, device="cuda")
    pos, refs = dev([0, 1]), dev(np.zeros(8))
    bad = [
        lambda: qg.paged_attention(pool, q.float(), table, lens), lambda: qg.paged_attention(pool, q[0], table, lens),
        lambda: qg.paged_attention(pool, q[:, :, :32], table, lens), lambda: qg.paged_attention(pool, q.cpu(), table, lens),
        lambda: qg.paged_attention(pool, q.transpose(0, 1), table, lens),
        lambda: qg.paged_attention(pool, q, table.long(), lens), lambda: qg.paged_attention(pool, q, table.t(), lens),
        lambda: qg.paged_attention(pool, q, table[:1], lens), lambda: qg.paged_attention(pool, q, table, lens[:1]),
        lambda: qg.paged_attention(pool, q, table, lens, max_len=33),
        lambda: qg.paged_attention(pool, q, table, lens, out=torch.empty_like(q)[:1]),
        lambda: qg.paged_attention(pool, q, table, lens, out=torch.empty_like(q).double()),
        lambda: qg.paged_attention(pool, q, table, lens, lse=torch.zeros((4, 2), device="cuda")),
        lambda: qg.paged_attention(pool, q, table, lens, workspace=torch.zeros(64, device="cuda")),
        lambda: qg.kv_append(pool, table, rows.float(), rows, pos), lambda: qg.kv_append(pool, table, rows[:, :64], rows, pos),
        lambda: qg.kv_append(pool, table, rows, rows[:1], pos), lambda: qg.kv_append(pool, table, rows, rows, pos.long()),
        lambda: qg.kv_append(pool, table, rows, rows, pos, dev([0])), lambda: qg.kv_gather(pool, table, pos, k=rows[:1]),
        lambda: qg.kv_copy_pages(pool, pos, dev([1])), lambda: qg.kv_copy_pages(pool, pos.cpu(), pos),
        lambda: qg.kv_fork(pool, table, lens, refs[:7], pos, pos, pos), lambda: qg.kv_fork(pool, table, lens[:1], refs, pos, pos, pos),
        lambda: qg.kv_free(pool, table, lens, refs.float(), pos), lambda: qg.kv_compact(pool, table, refs[:3]),
        lambda: qg.kv_compact(pool, table, refs, table_out=table[:1]),
        lambda: qg.KVPool(torch.zeros((4, 100), dtype=torch.uint8, device="cuda"), "q8", 2, 64, 16),
        lambda: qg.KVPool(pool.pages.float(), "q8", 2, 64, 16), lambda: qg.KVPool(pool.pages.cpu(), "q8", 2, 64, 16)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    refused = [lambda: qg.paged_attention(pool, q[:, :3], table, lens), lambda: qg.paged_attention(pool, q, table, lens, window=-1),
               lambda: qg.paged_attention(pool, q, table, lens, scale=float("nan")),
               lambda: qg.paged_attention(pool, q, table, lens, layer=1), lambda: qg.kv_append(pool, table, rows, rows, pos, layer=-1),
               lambda: qg.paged_attention(pool, torch.zeros(520, dtype=torch.float16, device="cuda")[4:516].view(2, 4, 64), table, lens)]
    for i, call in enumerate(refused):
        with pytest.raises(qg.QGError):
            call()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(KeyError):
        qg.KVPool(pool.pages, "q4", 2, 64, 16)
