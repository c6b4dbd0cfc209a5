"""GPU tests of a decode step's operators as they are used together: a prompt that several rows continue, places for
each step's tokens (kv_extend), norm and rotation on the way into the cache (kv_append_rope), attention that reads the
shared prompt once (prefix_attention), rejected tokens given back (kv_trim), forks and rows given up, against
the oracle doing the same; the same step captured and replayed; two of them at once; streams; given workspaces;
long prefixes against 64 bits; tokens past 4 GiB of a pool."""
import numpy as np
import pytest

import dequant_gemv_q4g32_amd as qg
from oracle import paged, step

from paged_util import assert_same_bytes, dev, download, random_cache, upload
from test_gpu_prefix_attention import check, shared_cache, starts_of

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def host(t):
    return t.cpu().numpy()


class Both:
    """A cache with its table on the GPU, and the oracle's copy of all of it."""

    def __init__(self, kind, rows, width, pages, heads, kv_heads, dim, tokens, seed):
        self.rng = np.random.default_rng(seed)
        self.heads, self.kv_heads, self.dim, self.tokens, self.rows = heads, kv_heads, dim, tokens, rows
        self.c = random_cache(kind, 1, pages, kv_heads, dim, tokens, seed, poison=True)
        self.pool = upload(self.c)
        self.table, self.lens, self.refs = np.full((rows, width), -1, np.int32), np.zeros(rows, np.int32), np.zeros(pages, np.int32)
        self.t, self.n, self.r = dev(self.table), dev(self.lens), dev(self.refs)
        w = [dev(self.rng.random(dim) + 0.5, np.float16) for _ in range(2)]
        self.rotary = qg.Rotary(dim, qg.rope_freqs(dim // 2, 10000.0, "linear", 4.0), True, *w)

    def same(self):
        for name, want, got in (("table", self.table, self.t), ("lens", self.lens, self.n), ("refs", self.refs, self.r)):
            assert np.array_equal(host(got), want), name
        assert_same_bytes(download(self.c, self.pool), self.c)

    def add(self, add, slots):
        """Tokens for rows that ask for add[r]; (granted, queries, seqs) of all slots."""
        granted, seqs, pos = qg.kv_extend(self.pool, self.t, self.n, self.r, dev(add), slots)
        want = step.extend(self.table, self.lens, self.refs, add, slots, self.tokens)
        for got, x in ((granted, want[0]), (seqs, want[2]), (pos, want[3])):
            assert np.array_equal(host(got), x)
        x = dev(self.rng.standard_normal((slots, (self.heads + 2 * self.kv_heads) * self.dim)), np.float16)
        q, k, v = x.split_with_sizes([n * self.dim for n in (self.heads, self.kv_heads, self.kv_heads)], 1)
        out = torch.zeros((slots, self.heads * self.dim), dtype=torch.float16, device="cuda")
        qg.kv_append_rope(self.pool, self.t, self.rotary, q, k, v, pos, seqs, q_out=out)
        zeros = [torch.zeros((slots, n * self.dim), dtype=torch.float16, device="cuda") for n in (self.heads, self.kv_heads)]
        turned = qg.qk_rope(self.rotary, q, k, pos, *zeros)
        assert torch.equal(out, turned[0])
        self.c.append(0, self.table, host(turned[1]), host(v), want[3], want[2])
        return want[0], out, want[2]

    def trim(self, to):
        qg.kv_trim(self.pool, self.t, self.n, self.r, dev(to))
        step.trim(self.table, self.lens, self.refs, to, self.tokens)

    def fork(self, src, dst):
        new = [int(p) for p in np.flatnonzero(self.refs == 0)[::-1][:len(dst)]]
        qg.kv_fork(self.pool, self.t, self.n, self.r, dev(src), dev(dst), dev(new))
        paged.fork(self.c, self.table, self.lens, self.refs, src, dst, new)

    def free(self, rows):
        qg.kv_free(self.pool, self.t, self.n, self.r, dev(rows))
        paged.free(self.c, self.table, self.lens, self.refs, rows)

    def attend(self, q, starts, prefix, f32=False):
        """Both attentions for a query a row. A page's places past its tokens hold anything, and are not read."""
        q = q.reshape(self.rows, self.heads, self.dim)
        tokens, scale = int(self.lens.max()), self.dim ** -0.5
        held = np.concatenate([np.abs(self.c.gather(0, self.table, np.arange(n), np.full(n, r))[1].astype(np.float64).ravel())
                               for r, n in enumerate(self.lens) if n])
        self.c.most = float(held.max(initial=0))
        with np.errstate(all="ignore"):
            want = paged.attention(self.c, 0, host(q), self.table, self.lens, tokens, scale)
        check(*qg.prefix_attention(self.pool, q, self.t, self.n, dev(starts), dev(prefix), out_f32=f32, return_lse=True), want, tokens,
              self.dim, self.c)
        check(*qg.paged_attention(self.pool, q, self.t, self.n, out_f32=f32, return_lse=True), want, tokens, self.dim, self.c)


@pytest.mark.parametrize("kind,heads,kv_heads,dim,prompts", [
    ("q8", 8, 2, 128, [70, 33]), ("f16", 4, 4, 64, [16, 100]), ("f16", 6, 1, 256, [45, 3]), ("q8", 12, 3, 64, [31, 64])])
def test_step_after_step(kind, heads, kv_heads, dim, prompts):
    """Rows 0-4 continue the first prompt, 5-7 the second, 8 none. Nine steps; every byte of the cache equals the
    oracle's after each."""
    tokens = 16
    s = Both(kind, 9, 10, 60, heads, kv_heads, dim, tokens, dim + heads)
    add = np.zeros(9, np.int32)
    add[[0, 5, 8]] = prompts + [1]
    granted, _, _ = s.add(add, sum(prompts) + 4)              # some slots stay empty
    assert granted.sum() == sum(prompts) + 1
    s.fork([0, 0, 0, 0, 5, 5], [1, 2, 3, 4, 6, 7])
    s.same()
    starts, prefix = [0, 5, 8], prompts
    for i in range(9):
        ask = np.ones(9, np.int32)
        ask[s.rng.integers(0, 9)] = 0                         # a row that waits
        before = s.refs.copy()
        last = np.where(s.lens % tokens > 0, s.table[np.arange(9), s.lens // tokens], -1)
        granted, q, seqs = s.add(ask, 8)                      # a slot for each row but one
        assert np.array_equal(granted, np.where((last >= 0) & (before[last] > 1), 0, ask))   # not into a page of others
        by_row = torch.zeros((9, heads * dim), dtype=torch.float16, device="cuda")
        by_row[dev(seqs[seqs >= 0], np.int64)] = q[dev(np.flatnonzero(seqs >= 0), np.int64)]
        s.attend(by_row, starts, prefix, f32=i % 2 == 0)
        to = np.full(9, -1, np.int32)
        if i % 3 == 1:                                        # the last tokens of some rows are rejected
            to[[1, 6]] = s.lens[[1, 6]] - 2
            to[3] = s.lens[3]
        s.trim(to)
        if i == 4:                                            # a row ends, another takes its place in the group
            s.free([2])
            s.fork([4], [2])
        if i == 6:                                            # a row falls back into its prompt, which it shares
            to[:] = -1
            to[7] = max(prompts[1] - 20, 0)
            s.trim(to)
            prefix = [prompts[0], to[7]]                      # what the group shares from now on
        s.same()


def decode_state(seed, kind="q8", rows=12, prompt=300, pages=160, width=32):
    """A prompt of row 0 that all rows continue, one cache for each call."""
    rng = np.random.default_rng(seed)
    heads, kv_heads, dim, tokens = 8, 2, 128, 16
    pool = upload(random_cache(kind, 2, pages, kv_heads, dim, tokens, seed))
    s = {"pool": pool, "table": dev(np.full((rows, width), -1)), "lens": dev(np.zeros(rows)), "refs": dev(np.zeros(pages)),
         "add": dev([prompt] + [0] * (rows - 1)), "to": dev([-1] * rows), "starts": dev([0, rows]), "prefix": dev([prompt]),
         "rotary": qg.Rotary(dim, qg.rope_freqs(dim)), "x": dev(rng.standard_normal((rows, (heads + 2 * kv_heads) * dim)), np.float16)}
    qg.kv_extend(pool, s["table"], s["lens"], s["refs"], s["add"], prompt)
    new = [pages - 1 - i for i in range(rows - 1)]
    qg.kv_fork(pool, s["table"], s["lens"], s["refs"], dev([0] * (rows - 1)), dev(range(1, rows)), dev(new))
    s["add"].copy_(dev([1] * rows))
    return s


def decode_step(s, layer=1, **how):
    """kv_trim, kv_extend, kv_append_rope, prefix_attention; all that they return."""
    pool, rows = s["pool"], s["lens"].numel()
    qg.kv_trim(pool, s["table"], s["lens"], s["refs"], s["to"], **how)
    granted, seqs, pos = qg.kv_extend(pool, s["table"], s["lens"], s["refs"], s["add"], rows, **how)
    q, k, v = s["x"].split_with_sizes([1024, 256, 256], 1)
    q = qg.kv_append_rope(pool, s["table"], s["rotary"], q, k, v, pos, seqs, q_out=s["x"].new_zeros(rows, 1024), layer=layer, **how)
    out, lse = qg.prefix_attention(pool, q.view(rows, 8, 128), s["table"], s["lens"], s["starts"], s["prefix"], layer=layer,
                                   return_lse=True, **how)
    return {"granted": granted, "seqs": seqs, "pos": pos, "q": q, "out": out, "lse": lse}


def feed(s, i):
    rng = np.random.default_rng(100 + i)
    s["x"].copy_(dev(rng.standard_normal(tuple(s["x"].shape)), np.float16))
    lens, rows = host(s["lens"]), s["lens"].numel()
    to = np.where(rng.random(rows) < 0.3, np.maximum(lens - rng.integers(0, 3, rows), 0), -1)
    s["to"].copy_(dev(to))
    s["add"].copy_(dev(rng.random(rows) < 0.8))
    s["starts"].copy_(dev([int(rng.integers(0, 3)), rows - int(rng.integers(0, 3))]))


def assert_same_state(a, b, what):
    for key in ("table", "lens", "refs"):
        assert torch.equal(a[key], b[key]), f"{what}: {key}"
    assert torch.equal(a["pool"].pages, b["pool"].pages), f"{what}: pages"


@pytest.mark.parametrize("kind", ["q8", "f16"])
def test_graph_follows_the_cache(kind):
    """A captured step, replayed while rows, lengths and groups change, with eager work between: every replay equals
    the eager result on the same state."""
    eager, graphed, side = decode_state(1, kind), decode_state(1, kind), decode_state(2, kind)
    feed(eager, 0), feed(graphed, 0), feed(side, 7)
    decode_step(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = decode_step(graphed)
    for i in range(1, 6):
        want = decode_step(eager)
        g.replay()
        decode_step(side)
        torch.cuda.synchronize()
        for key in want:
            assert torch.equal(got[key], want[key]), f"replay {i}: {key}"
        assert_same_state(graphed, eager, f"replay {i}")
        feed(eager, i), feed(graphed, i)


def test_two_graphs_at_once():
    """Two captured steps on their own caches, replayed together on two streams."""
    cases = []
    for seed in (3, 4):
        eager, graphed = decode_state(seed), decode_state(seed)
        feed(eager, seed), feed(graphed, seed)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = decode_step(graphed)
        cases.append((g, got, eager, graphed))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(6):
        for s, case in zip(streams, cases):
            with torch.cuda.stream(s):
                case[0].replay()
        wants = [decode_step(case[2]) for case in cases]
        torch.cuda.synchronize()
        for (_, got, eager, graphed), want in zip(cases, wants):
            for key in want:
                assert torch.equal(got[key], want[key]), (rep, key)
            assert_same_state(graphed, eager, rep)


def test_streams():
    """Steps on a stream that is passed or current, and two at once, equal the default stream's."""
    states = [decode_state(5) for _ in range(4)]
    for s in states:
        feed(s, 1)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for rep in range(3):
        want = decode_step(states[0])
        got = [decode_step(states[1], stream=a), decode_step(states[2], stream=b.cuda_stream)]
        with torch.cuda.stream(a):
            got.append(decode_step(states[3]))
        torch.cuda.synchronize()
        for x, s in zip(got, states[1:]):
            for key in want:
                assert torch.equal(x[key], want[key]), (rep, key)
            assert_same_state(s, states[0], rep)
    q = dev(np.random.default_rng(1).standard_normal((5, 1024)), np.float16)
    want = qg.qk_rope(states[0]["rotary"], q, q[:, :256], dev([0, 5, -1, 9, 70000]), torch.zeros_like(q), q.new_zeros(5, 256))
    torch.cuda.synchronize()
    got = qg.qk_rope(states[0]["rotary"], q, q[:, :256], dev([0, 5, -1, 9, 70000]), torch.zeros_like(q), q.new_zeros(5, 256), stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("kind,f32", [("q8", False), ("f16", True)])
def test_given_workspace(kind, f32):
    """A workspace of the stated size, with the bytes behind it untouched, whatever it held before."""
    lens = [700 + 13 * i for i in range(20)]
    c, table = shared_cache(kind, [12, 8], [700, 820], lens, 2, 128, 16, 4)
    pool, q = upload(c), dev(np.random.default_rng(1).standard_normal((20, 8, 128)), np.float16)
    args, more = [pool, q, dev(table), dev(lens), dev([0, 12, 20]), dev([700, 820])], {"out_f32": f32, "return_lse": True, "max_tail": 250}
    want = qg.prefix_attention(*args, **more)
    need = qg.prefix_attention_bytes(pool, 20, 8, 2, table.shape[1] * 16, 250)
    for fill in (0xFF, 0x00, 0x7F):
        buf = torch.full((need + 256,), fill, dtype=torch.uint8, device="cuda")
        got = qg.prefix_attention(*args, **more, workspace=buf[:need])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.all(buf[need:] == fill)
    with pytest.raises(qg.QGError):
        qg.prefix_attention(*args, **more, workspace=buf[:need - 16])


@pytest.mark.parametrize("kind,dim", [("q8", 128), ("f16", 64), ("f16", 128)])
@pytest.mark.parametrize("f32", [False, True])
def test_long_prefixes(kind, dim, f32):
    """20000 shared tokens, whose sums pass through many workgroups."""
    lens = [20000 + n for n in (0, 1, 300, 33, 5, 5)]
    c, table = shared_cache(kind, [6], [20000], lens, 1, dim, 64, 5)
    q = (np.random.default_rng(2).standard_normal((6, 5, dim)) * 2).astype(np.float16)
    out, lse = qg.prefix_attention(upload(c), dev(q, np.float16), dev(table), dev(lens), dev([0, 6]), dev([20000]), out_f32=f32, return_lse=True)
    check(out, lse, paged.attention(c, 0, q, table, lens, max(lens), dim ** -0.5), max(lens), dim, c)


def test_pages_past_4_gib():
    """A pool of 5 GB: the operators reach its last pages as they do its first."""
    heads, dim, tokens, lens, rows = 2, 256, 256, [300, 280, 511], 3
    pages = 5 * 2 ** 30 // qg.kv_page_bytes("f16", heads, dim, tokens)
    small = random_cache("f16", 1, 6, heads, dim, tokens, 3)
    pool = qg.KVPool(torch.empty((pages, qg.kv_page_bytes("f16", heads, dim, tokens)), dtype=torch.uint8, device="cuda"), "f16", heads, dim, tokens)
    low = qg.KVPool(torch.zeros_like(pool.pages[:6]), "f16", heads, dim, tokens)
    rng = np.random.default_rng(1)
    table = np.array([[0, 1], [0, 2], [0, 3]], np.int32)
    pool.pages[pages - 6:] = torch.from_numpy(small.pack()[0]).cuda()
    low.pages.copy_(pool.pages[pages - 6:])
    far = np.where(table >= 0, table + pages - 6, -1)
    x = dev(rng.standard_normal((rows, 6 * dim)), np.float16)
    rotary = qg.Rotary(dim, qg.rope_freqs(dim))
    got = []
    for p, t in ((pool, far), (low, table)):
        q = qg.kv_append_rope(p, dev(t), rotary, x[:, :2 * dim], x[:, 2 * dim:4 * dim], x[:, 4 * dim:], dev(np.array(lens) - 1))
        got.append((q, *qg.prefix_attention(p, q.view(rows, 2, dim), dev(t), dev(lens), dev([0, rows]), dev([256]), return_lse=True)))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert torch.equal(pool.pages[pages - 6:], low.pages)
    # places at the pool's end: all pages but the last three are held
    refs, lens_d, t = torch.ones(pages, dtype=torch.int32, device="cuda"), dev([0, 0]), dev(np.full((2, 4), -1))
    refs[pages - 3:] = 0
    granted, seqs, pos = qg.kv_extend(pool, t, lens_d, refs, dev([257, 256]), 600)
    assert host(granted).tolist() == [257, 256]
    assert host(t)[:, :2].tolist() == [[pages - 3, pages - 2], [pages - 1, -1]] and host(refs).min() == 1
