"""GPU tests of the attention over shared prefixes against the oracle's one-token attention (sharing
changes how it is computed, not what): groups of all sizes, prefixes that end anywhere, rows shorter than their
prefix, missing pages, garbage wherever nothing may be read, and groups that are none."""
import numpy as np
import pytest

import dequant_gemv_q4g32_amd as qg
from oracle import paged

from paged_util import attention_tolerance, dev, random_cache, upload

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def tolerance(out, lse, bound, reach, tokens, dim, f32, most):
    """As the one-token attention's, with two terms more.

    fp16 results: the shared tokens' weights are rounded to fp16 once, at most 2^-11 of each, so at most 2^-11 of the
    sum of w |v|.

    Small weights: a weight p = 2^(s - ref) below 2^-14 is a subnormal fp16 number (as a pair: its remainder is),
    off by up to 2^-25, half the distance of these. The reference was last moved to 7 below the largest score of
    that moment and scores found later only add to the sum, so the sum of the weights is at least 2^7: together at most
    2^-25 / 2^7 times the sum of |v|, tokens * most * 2^-32. The other tolerances are relative to the sum of w |v|, which
    can be smaller than that: where the largest weight meets a value near zero."""
    tol, tol_lse = attention_tolerance(out, lse, bound, reach, tokens, dim, f32)
    return tol + (0 if f32 else bound * 2.0 ** -11) + tokens * most * 2.0 ** -32, tol_lse


def check(got, got_lse, ref, tokens, dim, cache):
    out, lse, bound, reach = ref
    tol, tol_lse = tolerance(out, lse, bound, reach, tokens, dim, got.dtype == torch.float32, cache.most)
    g, gl = got.cpu().double().numpy(), got_lse.cpu().double().numpy()
    bad = ~(np.abs(g - out) <= tol)
    assert not bad.any(), (f"out: {int(bad.sum())} of {bad.size}, first {np.argwhere(bad)[0].tolist()}: got {g[bad][0]:.8g} "
                           f"want {out[bad][0]:.8g} tolerance {tol[bad][0]:.3g}")
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(gl), empty)
    bad = ~(np.abs(np.where(empty, 0, gl) - np.where(empty, 0, lse)) <= tol_lse)
    assert not bad.any(), f"lse: {np.argwhere(bad)[0].tolist()}: got {gl[bad][0]:.9g} want {lse[bad][0]:.9g} tolerance {tol_lse[bad][0]:.3g}"


def shared_cache(kind, sizes, prefixes, lens, kv_heads, dim, tokens, seed, spare=2, holes=()):
    """(oracle cache, table) of groups whose rows' tables name the first row's pages for the whole pages of the
    prefix. The page that a prefix ends in is a copy. Places that hold no token are poisoned."""
    rng = np.random.default_rng(seed)
    width = max(1, max(-(-n // tokens) for n in lens))
    table = np.full((len(lens), width), -1, np.int32)
    need = sum(-(-n // tokens) for n in lens) + spare
    order, at, copies, b = rng.permutation(need), 0, [], 0
    for size, prefix in zip(sizes, prefixes):
        lead = b
        for _ in range(size):
            n = -(-lens[b] // tokens)
            whole = 0 if b == lead else min(min(prefix, lens[lead]) // tokens, n)
            table[b, :whole] = table[lead, :whole]
            table[b, whole:n] = order[at:at + n - whole]
            if b != lead and min(prefix, lens[lead]) % tokens and whole < n:
                copies.append((table[lead, whole], table[b, whole]))
            at += n - whole
            b += 1
    while b < len(lens):                                  # rows in no group
        n = -(-lens[b] // tokens)
        table[b, :n] = order[at:at + n]
        at += n
        b += 1
    c = random_cache(kind, 1, need, kv_heads, dim, tokens, seed)
    c.most = float(127 * c.scales[1].max() if kind == "q8" else np.abs(c.values[1]).max())   # no value is larger
    for src, dst in copies:
        c.copy_page(src, dst)
    poison = random_cache(kind, 1, need, kv_heads, dim, tokens, seed + 1, poison=True)
    held = np.zeros((need, tokens), bool)
    for b, n in enumerate(lens):
        for j in range(n):
            if table[b, j // tokens] >= 0:
                held[table[b, j // tokens], j % tokens] = True
    for mine, theirs in zip(c._arrays, poison._arrays):
        mine[0] = np.where(held[:, None, :, None], mine[0], theirs[0])
    for b, j, page in holes:
        table[b, j] = page
    return c, table


def starts_of(sizes):
    return np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)


CASES = [
    # kind, rows of the groups, prefixes, tails (cycled over the rows), heads, kv heads, dim, tokens a page
    ("f16", [2], [16], [1], 8, 8, 64, 16), ("q8", [2], [16], [1], 8, 8, 128, 16), ("f16", [2], [16], [0], 2, 1, 256, 16),
    ("q8", [9], [200], [1, 30, 64], 8, 2, 128, 16), ("f16", [9], [200], [1, 30, 64], 8, 2, 128, 16),
    ("q8", [40], [517], [3, 0, 17], 12, 3, 64, 32), ("f16", [40], [517], [3, 0, 17], 12, 3, 64, 32),
    ("q8", [20], [333], [5, 40], 16, 1, 256, 64), ("f16", [20], [333], [5, 40], 16, 1, 256, 64),
    ("f16", [3, 1, 5, 2], [100, 70, 15, 48], [9, 1, 33], 4, 4, 64, 16), ("q8", [3, 1, 5, 2], [100, 70, 15, 48], [9, 1, 33], 4, 2, 128, 16),
    ("q8", [65], [64], [2], 7, 1, 128, 16), ("f16", [130], [257], [1], 2, 2, 128, 128), ("f16", [17], [1500], [20], 5, 1, 64, 256),
    ("q8", [33], [1041], [100, 1], 20, 2, 64, 16), ("q8", [5, 6], [2000, 1200], [40], 12, 2, 256, 16),
    ("f16", [1, 1, 1], [50, 60, 70], [4], 4, 2, 64, 16), ("q8", [2, 2], [0, 5], [40, 3], 4, 2, 64, 16)]


@pytest.mark.parametrize("kind,sizes,prefixes,tails,heads,kv_heads,dim,tokens", CASES)
@pytest.mark.parametrize("f32", [False, True])
def test_groups(kind, sizes, prefixes, tails, heads, kv_heads, dim, tokens, f32):
    owner = [g for g, n in enumerate(sizes) for _ in range(n)]
    lens = [prefixes[g] + tails[i % len(tails)] for i, g in enumerate(owner)]
    c, table = shared_cache(kind, sizes, prefixes, lens, kv_heads, dim, tokens, 11)
    rng = np.random.default_rng(3)
    q = (rng.standard_normal((len(lens), heads, dim)) * 1.5).astype(np.float16)
    out, lse = qg.prefix_attention(upload(c), dev(q, np.float16), dev(table), dev(lens), dev(starts_of(sizes)), dev(prefixes),
                                   max_tail=max(tails), out_f32=f32, return_lse=True)
    check(out, lse, paged.attention(c, 0, q, table, lens, max(lens), dim ** -0.5), max(lens), dim, c)


@pytest.mark.parametrize("kind,dim", [("q8", 128), ("f16", 64), ("f16", 256)])
def test_rows_of_any_length(kind, dim):
    """Empty rows, rows that end inside the prefix, inside its last page, at its end; a first row that is
    shorter than the prefix; rows before and behind all groups."""
    sizes, prefixes = [7, 4, 3], [200, 150, 64]
    lens = [230, 0, 1, 100, 199, 200, 201, 90, 170, 160, 150, 0, 70, 64, 33, 0]
    c, table = shared_cache(kind, sizes, prefixes, lens, 2, dim, 16, 5)
    rng = np.random.default_rng(4)
    q = rng.standard_normal((len(lens), 6, dim)).astype(np.float16)
    for f32 in (False, True):
        out, lse = qg.prefix_attention(upload(c), dev(q, np.float16), dev(table), dev(lens), dev(starts_of(sizes)), dev(prefixes),
                                       out_f32=f32, return_lse=True)
        check(out, lse, paged.attention(c, 0, q, table, lens, max(lens), dim ** -0.5), 230, dim, c)
        assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()


@pytest.mark.parametrize("starts", [[3, 3, 9], [2, 6, 6], [0, 20, 5], [-4, 4, 99], [5, 2, 12], [12, 12, 12]])
def test_starts(starts):
    """Rows in no group, empty groups, and starts that do not ascend or lie outside the batch: they count as the
    header says, and every row is right as long as its group's rows share what they claim."""
    lens = [100 + i for i in range(12)]
    c, table = shared_cache("f16", [12], [96], lens, 2, 64, 16, 9)
    rng = np.random.default_rng(4)
    q = rng.standard_normal((12, 4, 64)).astype(np.float16)
    out, lse = qg.prefix_attention(upload(c), dev(q, np.float16), dev(table), dev(lens), dev(starts), dev([96, 80]), out_f32=True,
                                   return_lse=True)
    check(out, lse, paged.attention(c, 0, q, table, lens, max(lens), 0.125), 111, 64, c)


@pytest.mark.parametrize("prefix", [-5, 0, 15, 16, 10 ** 9])
def test_prefixes_past_the_first_row(prefix):
    """A prefix past the first row's tokens counts as those: the rows are forks of one length here."""
    lens = [80] * 5
    c, table = shared_cache("q8", [5], [80], lens, 1, 64, 16, 2)
    q = np.random.default_rng(4).standard_normal((5, 3, 64)).astype(np.float16)
    out, lse = qg.prefix_attention(upload(c), dev(q, np.float16), dev(table), dev(lens), dev([0, 5]), dev([prefix]), return_lse=True)
    check(out, lse, paged.attention(c, 0, q, table, lens, 80, 0.125), 80, 64, c)


@pytest.mark.parametrize("kind", ["q8", "f16"])
@pytest.mark.parametrize("tokens", [16, 64])
def test_missing_pages(kind, tokens):
    """Entries that are no page, in the prefix and behind it: their tokens are not there. A prefix of no pages at all."""
    sizes, prefixes, lens = [6, 3], [400, 200], [430] * 6 + [210] * 3
    holes = [(b, j, e) for b in range(6) for j, e in ((1, -1), (400 // tokens - 1, 10 ** 6))]
    holes += [(b, j, -1) for b in (6, 7, 8) for j in range(200 // tokens)] + [(2, 400 // tokens, -7)]
    c, table = shared_cache(kind, sizes, prefixes, lens, 2, 128, tokens, 6, holes=holes)
    q = np.random.default_rng(4).standard_normal((9, 8, 128)).astype(np.float16)
    for f32 in (False, True):
        out, lse = qg.prefix_attention(upload(c), dev(q, np.float16), dev(table), dev(lens), dev(starts_of(sizes)), dev(prefixes),
                                       out_f32=f32, return_lse=True)
        check(out, lse, paged.attention(c, 0, q, table, lens, 430, 128 ** -0.5), 430, 128, c)


@pytest.mark.parametrize("kind", ["q8", "f16"])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0, 1e-30])
def test_scales(kind, scale):
    sizes, prefixes, lens = [12], [300], [310] * 12
    c, table = shared_cache(kind, sizes, prefixes, lens, 1, 64, 16, 8)
    q = np.random.default_rng(4).standard_normal((12, 4, 64)).astype(np.float16)
    out, lse = qg.prefix_attention(upload(c), dev(q, np.float16), dev(table), dev(lens), dev([0, 12]), dev(prefixes), scale=scale,
                                   out_f32=True, return_lse=True)
    check(out, lse, paged.attention(c, 0, q, table, lens, 310, scale), 310, 64, c)


@pytest.mark.parametrize("kind", ["q8", "f16"])
def test_rising_scores(kind):
    """Scores that grow along the prefix, by far more than fp16 weights span: the running reference moves again and again."""
    lens = [1024 + 5] * 8
    c, table = shared_cache(kind, [8], [1024], lens, 1, 64, 16, 8)
    if kind == "f16":
        for j in range(1024):
            c.values[0][0, table[0, j // 16], :, j % 16] = np.float16(j / 1024) * np.sign(c.values[0][0, table[0, j // 16], :, j % 16])
    else:
        for j in range(1024):
            c.scales[0][0, table[0, j // 16], :, j % 16] = np.float16(j / 1024 / 64)
    q = (np.random.default_rng(4).standard_normal((8, 4, 64)) * 4).astype(np.float16)
    for f32 in (False, True):
        out, lse = qg.prefix_attention(upload(c), dev(q, np.float16), dev(table), dev(lens), dev([0, 8]), dev([1024]), scale=2.0,
                                       out_f32=f32, return_lse=True)
        check(out, lse, paged.attention(c, 0, q, table, lens, 1029, 2.0), 1029, 64, c)


@pytest.mark.parametrize("kind", ["q8", "f16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_queries_that_are_not_finite(kind, value):
    """Such a head gives NaN where it sees a token, and changes no other; one that sees none gives zeros."""
    lens = [110, 105, 0, 101, 3]
    c, table = shared_cache(kind, [5], [96], lens, 2, 64, 16, 8)
    q = np.random.default_rng(4).standard_normal((5, 4, 64)).astype(np.float16)
    want = paged.attention(c, 0, q, table, lens, 110, 0.125)
    for b, h in ((0, 1), (2, 2), (3, 0), (4, 3)):
        q[b, h, 7] = value
    out, lse = qg.prefix_attention(upload(c), dev(q, np.float16), dev(table), dev(lens), dev([0, 5]), dev([96]), out_f32=True,
                                   return_lse=True)
    for b, h in ((0, 1), (3, 0), (4, 3)):
        assert torch.isnan(out[b, h]).all() and torch.isnan(lse[b, h]), (b, h)
        want[0][b, h] = want[1][b, h] = 0
        out[b, h] = lse[b, h] = 0
    check(out, lse, want, 110, 64, c)


def test_strides_layers_and_given_outputs():
    """q and out as parts of wider rows, a layer of several, a table with further columns, a workspace that holds anything."""
    rng = np.random.default_rng(7)
    sizes, prefixes, lens = [4, 3], [100, 40], [120, 101, 130, 111, 60, 41, 44]
    c, table = shared_cache("q8", sizes, prefixes, lens, 2, 128, 16, 8)
    packed = c.pack()
    pool = qg.KVPool(torch.from_numpy(np.concatenate([packed, np.full_like(packed, 0x7E), packed])).cuda()[::2], "q8", 2, 128, 16)
    wide = torch.randn((7, 1024 + 64), device="cuda").half()
    q = wide[:, :1024].unflatten(1, (8, 128))
    t = torch.full((7, table.shape[1] + 5), 10 ** 8, dtype=torch.int32, device="cuda")
    t[:, 2:2 + table.shape[1]] = dev(table)
    t = t[:, 2:2 + table.shape[1]]
    size = qg.prefix_attention_bytes(pool, 7, 8, 2, 130, 30)
    for f32 in (False, True):
        room = torch.full((7, 1024 + 8), 5.0, dtype=torch.float32 if f32 else torch.float16, device="cuda")
        out, lse = room[:, :1024].unflatten(1, (8, 128)), torch.empty((7, 8), device="cuda")
        work = torch.randint(0, 256, (size,), dtype=torch.uint8, device="cuda")
        got = qg.prefix_attention(pool, q, t, dev(lens), dev(starts_of(sizes)), dev(prefixes), max_len=130, max_tail=30, out=out,
                                  lse=lse, workspace=work, layer=1)
        assert got[0] is out and got[1] is lse
        check(out, lse, paged.attention(c, 0, q.cpu().numpy(), table, lens, 130, 128 ** -0.5), 130, 128, c)
        assert (room[:, 1024:] == 5).all()


@pytest.mark.parametrize("max_tail", [0, 40, 700])
def test_max_tail_chooses_the_launch_only(max_tail):
    """Tails longer than max_tail says, and by far shorter ones; a long tail's split over the workgroups."""
    lens = [600, 65, 640, 64, 300]
    c, table = shared_cache("f16", [5], [64], lens, 1, 64, 16, 8)
    q = np.random.default_rng(4).standard_normal((5, 2, 64)).astype(np.float16)
    out, lse = qg.prefix_attention(upload(c), dev(q, np.float16), dev(table), dev(lens), dev([0, 5]), dev([64]), max_tail=max_tail,
                                   out_f32=True, return_lse=True)
    check(out, lse, paged.attention(c, 0, q, table, lens, 640, 0.125), 640, 64, c)


def test_many_groups():
    """More groups than a wave has lanes, and than a workgroup has threads; sizes 0 to 3."""
    rng = np.random.default_rng(7)
    for groups in (70, 1023):
        sizes = rng.integers(0, 4, groups).tolist()
        prefixes = rng.integers(0, 50, groups).tolist()
        owner = [g for g, n in enumerate(sizes) for _ in range(n)]
        lens = [int(prefixes[g] + rng.integers(0, 5)) for g in owner]
        c, table = shared_cache("f16", sizes, prefixes, lens, 1, 64, 16, 3)
        q = rng.standard_normal((len(lens), 2, 64)).astype(np.float16)
        out, lse = qg.prefix_attention(upload(c), dev(q, np.float16), dev(table), dev(lens), dev(starts_of(sizes)), dev(prefixes),
                                       max_tail=5, out_f32=True, return_lse=True)
        check(out, lse, paged.attention(c, 0, q, table, lens, max(lens), 0.125), max(lens), 64, c)


@pytest.mark.parametrize("kind,sizes,prefixes,heads,kv_heads,dim,tokens", [
    ("f16", [12, 30, 9], [16, 40, 130], 8, 4, 64, 16), ("q8", [24, 40], [16, 33], 8, 4, 128, 16), ("f16", [16, 2, 25], [32, 500, 16], 4, 1, 256, 16),
    ("q8", [90], [128], 34, 2, 64, 32), ("q8", [4, 5, 3, 2], [1600, 1600, 1600, 1600], 4, 2, 128, 64), ("f16", [2, 3, 1], [1500, 900, 2000], 20, 1, 64, 16)])
@pytest.mark.parametrize("f32", [False, True])
def test_groups_round_the_choice_to_share(kind, sizes, prefixes, heads, kv_heads, dim, tokens, f32):
    """Many rows after less than a tile of shared tokens, few rows after many: read together, or for each row."""
    lens = [prefixes[g] + (7 * b) % 19 for b, g in enumerate(g for g, n in enumerate(sizes) for _ in range(n))]
    c, table = shared_cache(kind, sizes, prefixes, lens, kv_heads, dim, tokens, 21)
    q = (np.random.default_rng(4).standard_normal((len(lens), heads, dim)) * 1.5).astype(np.float16)
    out, lse = qg.prefix_attention(upload(c), dev(q, np.float16), dev(table), dev(lens), dev(starts_of(sizes)), dev(prefixes),
                                   max_tail=20, out_f32=f32, return_lse=True)
    check(out, lse, paged.attention(c, 0, q, table, lens, max(lens), dim ** -0.5), max(lens), dim, c)


@pytest.mark.parametrize("kind,dim,heads,kv_heads,tokens", [
    ("q8", 64, 32, 16, 16), ("f16", 64, 14, 14, 32), ("q8", 128, 60, 20, 16), ("f16", 128, 80, 16, 64), ("q8", 256, 16, 16, 16), ("f16", 256, 45, 15, 16),
    ("q8", 64, 256, 16, 16), ("f16", 64, 272, 16, 16)])
@pytest.mark.parametrize("f32", [False, True])
def test_many_groups_of_few_rows(kind, dim, heads, kv_heads, tokens, f32):
    """Enough of them that their tokens are read once for 16 query rows (or, with 16 heads of a KV head, for each
    row): rows shorter than their prefix, of no token, of equal and of different lengths, missing pages, queries that are
    not finite."""
    sizes, prefixes = [2, 3, 1, 5, 4, 2, 7, 2, 3, 2], [100, 64, 90, 33, 160, 47, 16, 96, 128, 70]
    owner = [g for g, n in enumerate(sizes) for _ in range(n)]
    lens = [prefixes[g] + (5 * b) % 23 for b, g in enumerate(owner)]
    lens[1], lens[4], lens[8], lens[18], lens[22] = 40, 0, 1, 17, 128
    c, table = shared_cache(kind, sizes, prefixes, lens, kv_heads, dim, tokens, 31)
    for b in (11, 12, 13, 14):                            # the group that starts at row 11 misses a page in its prefix
        table[b, 1] = -1
    rng = np.random.default_rng(5)
    q = (rng.standard_normal((len(lens), heads, dim)) * 1.5).astype(np.float16)
    want = paged.attention(c, 0, q, table, lens, max(lens), dim ** -0.5)
    args = [dev(table), dev(lens), dev(starts_of(sizes)), dev(prefixes)]
    out, lse = qg.prefix_attention(upload(c), dev(q, np.float16), *args, max_tail=30, out_f32=f32, return_lse=True)
    check(out, lse, want, max(lens), dim, c)
    odd = q.copy()
    odd[2, 1], odd[9, 0, 3], odd[20, heads - 1, dim - 1] = np.nan, np.inf, -np.inf
    got, got_lse = qg.prefix_attention(upload(c), dev(odd, np.float16), *args, max_tail=30, out_f32=f32, return_lse=True)
    bad = ~np.isfinite(odd).all(-1)
    seen = bad & ~np.isneginf(want[1])
    assert np.isnan(got.cpu().numpy()[seen]).all() and np.isnan(got_lse.cpu().numpy()[seen]).all()
    rest = torch.from_numpy(~bad).cuda()
    assert torch.equal(got[rest], out[rest]) and torch.equal(got_lse[rest], lse[rest])


@pytest.mark.parametrize("kind,dim", [("q8", 64), ("f16", 256)])
def test_long_rows_without_a_group(kind, dim):
    """More own tokens than max_tail says: the workspace's room for partial results spreads them less."""
    lens = [9000, 33, 5000]
    c, table = shared_cache(kind, [1], [8000], lens, 2, dim, 16, 9)
    q = (np.random.default_rng(4).standard_normal((3, 6, dim)) * 1.5).astype(np.float16)
    want = paged.attention(c, 0, q, table, lens, max(lens), dim ** -0.5)
    for max_tail in (0, 100, 9000):
        out, lse = qg.prefix_attention(upload(c), dev(q, np.float16), dev(table), dev(lens), dev([0, 1]), dev([8000]), max_tail=max_tail, return_lse=True)
        check(out, lse, want, max(lens), dim, c)


def test_nothing_to_see():
    """No sequences, no groups, no tokens at all, a table without entries."""
    c, table = shared_cache("f16", [3], [16], [20] * 3, 1, 64, 16, 8)
    pool, q, none = upload(c), torch.ones((3, 2, 64), dtype=torch.float16, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    for args in ((dev(table), dev([0, 0, -3]), dev([0, 3]), dev([16])), (torch.zeros((3, 0), dtype=torch.int32, device="cuda"), dev([5, 5, 5]), dev([0, 3]), dev([16])),
                 (dev(table), dev([0, 0, 0]), dev([0]), none)):
        out, lse = qg.prefix_attention(pool, q, *args, return_lse=True)
        assert torch.all(out == 0) and torch.all(lse == -float("inf"))
    out, lse = qg.prefix_attention(pool, q[:0], dev(table)[:0], none, dev([0]), none, return_lse=True)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    alone = qg.prefix_attention(pool, q, dev(table), dev([20] * 3), dev([0]), none, out_f32=True, return_lse=True)
    check(*alone, paged.attention(c, 0, q.cpu().numpy(), table, [20] * 3, 32, 0.125), 20, 64, c)


def test_equal_inputs_give_equal_bits():
    lens = [1000 + i for i in range(30)]
    c, table = shared_cache("q8", [30], [1000], lens, 2, 128, 16, 8)
    pool, q = upload(c), dev(np.random.default_rng(1).standard_normal((30, 8, 128)), np.float16)
    args = [pool, q, dev(table), dev(lens), dev([0, 30]), dev([1000])]
    first = qg.prefix_attention(*args, out_f32=True, return_lse=True)
    for _ in range(3):
        again = qg.prefix_attention(*args, out_f32=True, return_lse=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_binding_refusals():
    c, table = shared_cache("q8", [3], [16], [20] * 3, 1, 64, 16, 8)
    pool, q = upload(c), torch.zeros((3, 2, 64), dtype=torch.float16, device="cuda")
    t, lens, starts, prefix = dev(table), dev([20] * 3), dev([0, 3]), dev([16])
    for bad in (lambda: qg.prefix_attention(pool, q.float(), t, lens, starts, prefix), lambda: qg.prefix_attention(pool, q[:2], t, lens, starts, prefix),
                lambda: qg.prefix_attention(pool, q, t, lens[:2], starts, prefix), lambda: qg.prefix_attention(pool, q, t, lens, starts[:1], prefix),
                lambda: qg.prefix_attention(pool, q, t, lens, starts.cpu(), prefix), lambda: qg.prefix_attention(pool, q, t, lens, starts, prefix.long()),
                lambda: qg.prefix_attention(pool, q, t, lens, starts, prefix, max_len=33),
                lambda: qg.prefix_attention(pool, q, t, lens, starts, prefix, out=torch.zeros((3, 2, 64))),
                lambda: qg.prefix_attention(pool, q, t, lens, starts, prefix, workspace=torch.zeros(4, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(qg.QGError):
        qg.prefix_attention(pool, q, t, lens, starts, prefix, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(qg.QGError):
        qg.prefix_attention(pool, q, t, lens, starts, prefix, max_tail=-1)
