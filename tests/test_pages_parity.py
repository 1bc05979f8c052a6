"""The pages of a cache against the oracle: sequences forked, grown, freed, the cache compacted, pages copied, rows kept (GPU).

Everything is whole numbers or moved bytes: results are equal."""
import numpy as np
import pytest
import torch

from oracle import pages_oracle as po
from sdpa_testlib import lib
from serving_testlib import make_cache

pytestmark = pytest.mark.gpu

MARK, PAD = 0x5A5A5A5A, 64


def words(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Guarded:
    """An int32 tensor of a shape and row stride inside a buffer of marks."""

    def __init__(self, shape, stride=None, fill=7):
        shape = tuple(shape)
        strides = (stride or shape[-1], 1) if len(shape) == 2 else (1,)
        span = 1 + sum((n - 1) * s for n, s in zip(shape, strides))
        self.buf = torch.full((span + 2 * PAD,), MARK, dtype=torch.int32, device="cuda")
        self.t = self.buf.as_strided(shape, strides, PAD)
        self.inside = torch.zeros_like(self.buf, dtype=torch.bool)
        self.inside.as_strided(shape, strides, PAD).fill_(True)
        self.t.fill_(fill)

    def check(self):
        assert (self.buf[~self.inside] == MARK).all(), "written outside the tensor"
        return self.t.tolist()


def guarded(x, stride=None):
    x = np.asarray(x)
    g = Guarded(x.shape, stride)
    g.t.copy_(words(x))
    return g


def batch(rng, b, columns, page, spread, spare, shared=0.5, missing=0.1):
    """A page table whose rows share pages, lengths, and counts that hold some owners besides."""
    cap = columns * page
    lens = [int(rng.integers(0, cap + 1)) for _ in range(b)]
    lens = [n if rng.random() > 0.2 else int(rng.choice([0, 1, page, cap, n // page * page])) for n in lens]
    table, at = np.full((b, columns), -1, np.int64), 0
    for i, n in enumerate(lens):
        need = -(-n // page)
        take = 0
        if i and rng.random() < shared:
            j = int(rng.integers(0, i))
            take = min(need, -(-lens[j] // page), int(rng.integers(0, columns + 1)) if rng.random() < 0.5 else columns)
            table[i, :take] = table[j, :take]
            if take == need and n % page and rng.random() < 0.7:
                lens[i] = n = min(lens[j], need * page) if -(-lens[j] // page) == need else n
        table[i, take:need] = np.arange(at, at + need - take)
        at += need - take
    pages = max(1, at + spare) * spread
    order = rng.permutation(pages)
    table = np.where(table >= 0, order[table], -1)
    counts = np.where(rng.random(pages) < 0.1, 1, 0)                       # what else owns pages
    for row, n in zip(table, lens):
        need = -(-n // page)
        for c in range(columns):
            if c >= need:
                row[c] = rng.choice([-1, 0, 123456789])                    # (not reached: it may hold anything)
            elif rng.random() < missing:
                row[c] = rng.choice([-1, -5, pages, pages + 1000, 2 ** 31 - 1])
            else:
                counts[row[c]] += 1
    return table.tolist(), lens, counts.tolist()


SIZES = [
    # b, columns, page, spread, spare
    (1, 1, 16, 1, 1), (1, 1, 64, 1, 3), (3, 4, 16, 1, 5), (4, 17, 64, 1, 9), (7, 130, 16, 1, 40), (33, 9, 32, 2, 30), (64, 300, 16, 1, 900),
    (1, 3000, 16, 1, 10), (2, 700, 48, 9, 100), (300, 5, 128, 1, 400), (1500, 2, 16, 1, 2000), (40, 64, 16, 20, 300),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("b,columns,page,spread,spare", SIZES)
def test_fork(b, columns, page, spread, spare, in_place):
    m, rng = lib(), np.random.default_rng(b * 7 + columns)
    table, lens, counts = batch(rng, b, columns, page, spread, spare)
    said = [n + (1000 * columns * page if rng.random() < 0.05 and n == columns * page else 0) for n in lens]   # (clamped)
    for b_out in {1, b, 2 * b + 3}:
        parents = rng.integers(-2, b + 2, b_out)
        t, out, lens_out = guarded(table, columns + 3), Guarded((b_out, columns), columns + 5), Guarded((b_out,))
        refs = guarded(counts)
        refs_out = refs if in_place else Guarded((len(counts),))
        m.sdpa_cache_fork(t.t, words(said), words(parents), refs.t, out.t, lens_out.t, None if in_place else refs_out.t, page_size=page)
        rows, ns, cs = po.fork(table, lens, parents, counts, page)
        assert out.check() == rows and lens_out.check() == ns and refs_out.check() == cs
        assert t.check() == table and (in_place or refs.check() == counts)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("b,columns,page,spread,spare", SIZES)
def test_grow(b, columns, page, spread, spare, in_place):
    m, rng = lib(), np.random.default_rng(b * 11 + columns)
    table, lens, counts = batch(rng, b, columns, page, spread, spare)
    cap = columns * page
    one = [n + 1 for n in lens]
    some = [n + int(rng.integers(-5, 3 * page)) for n in lens]
    most = [cap + 1000 if rng.random() < 0.5 else -3 for _ in lens]
    granted = 0
    for new in (lens, one, some, most):
        t, refs = guarded(table, columns + 1), guarded(counts)
        out = t if in_place else Guarded((b, columns), columns + 2)
        refs_out = refs if in_place else Guarded((len(counts),))
        src, dst, missing = Guarded((b,)), Guarded((b,)), Guarded((1,))
        where = {} if in_place else dict(page_table_out=out.t, ref_counts_out=refs_out.t)
        m.sdpa_cache_grow(t.t, words(lens), words(new), refs.t, src.t, dst.t, missing.t, page_size=page, **where)
        rows, cs, a, z, lacked = po.grow(table, lens, new, counts, page)
        assert missing.check() == [lacked] and src.check() == a and dst.check() == z
        assert out.check() == (table if lacked else rows) and refs_out.check() == (counts if lacked else cs)
        granted += not lacked
    assert granted >= 1


def test_grow_by_exactly_what_is_free():
    m, page = lib(), 16
    for pages, lens, new in ((1, [0], [16]), (5, [0, 0], [48, 32]), (6, [0, 0], [48, 32]), (40000, [0] * 4, [160000] * 4)):
        columns = -(-max(new) // page)
        for take in (0, 1):
            counts = [0] * pages
            for i in range(0, pages - sum(n // page for n in new) + take):
                counts[(i * 7919) % pages] = 1
            free = counts.count(0)
            table = [[-1] * columns for _ in lens]
            t, refs, src, dst, missing = guarded(table), guarded(counts), Guarded((len(lens),)), Guarded((len(lens),)), Guarded((1,))
            m.sdpa_cache_grow(t.t, words(lens), words(new), refs.t, src.t, dst.t, missing.t, page_size=page)
            rows, cs, _, _, lacked = po.grow(table, lens, new, counts, page)
            assert lacked == max(0, sum(n // page for n in new) - free)
            assert missing.check() == [lacked] and t.check() == (table if lacked else rows) and refs.check() == (counts if lacked else cs)


@pytest.mark.parametrize("b,owners", [(8, 8), (8, 9), (100, 100), (4096, 4097), (1030, 1030)])
def test_grow_in_one_shared_page(b, owners):
    """All rows grow in the same partly filled page: with no other owner the last of them keeps it."""
    m, page = lib(), 16
    table, counts = [[3, -1]] * b, [0] * (b + 8)
    counts[3] = owners
    t, refs, src, dst, missing = guarded(table), guarded(counts), Guarded((b,)), Guarded((b,)), Guarded((1,))
    m.sdpa_cache_grow(t.t, words([5] * b), words([6] * b), refs.t, src.t, dst.t, missing.t, page_size=page)
    rows, cs, a, z, lacked = po.grow(table, [5] * b, [6] * b, counts, page)
    assert lacked == 0 and a.count(3) == b - (owners == b)
    assert t.check() == rows and refs.check() == cs and src.check() == a and dst.check() == z and missing.check() == [0]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("b,columns,page,spread,spare", SIZES)
def test_free(b, columns, page, spread, spare, in_place):
    m, rng = lib(), np.random.default_rng(b * 13 + columns)
    table, lens, counts = batch(rng, b, columns, page, spread, spare)
    for kept in ([0] * b, list(lens), [int(rng.integers(-5, n + 40)) for n in lens]):
        t, refs = guarded(table, columns + 1), guarded(counts)
        out = t if in_place else Guarded((b, columns), columns + 2)
        refs_out = refs if in_place else Guarded((len(counts),))
        where = {} if in_place else dict(page_table_out=out.t, ref_counts_out=refs_out.t)
        m.sdpa_cache_free(t.t, words(lens), words(kept), refs.t, page_size=page, **where)
        rows, cs = po.free(table, lens, kept, counts, page)
        assert out.check() == rows and refs_out.check() == cs


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("b,columns,page,spread,spare", SIZES)
def test_compact(b, columns, page, spread, spare, in_place):
    m, rng = lib(), np.random.default_rng(b * 17 + columns)
    table, lens, counts = batch(rng, b, columns, page, spread, spare)
    kept = [n if rng.random() < 0.5 else 0 for n in lens]
    table, counts = po.free(table, lens, kept, counts, page)
    for pairs in (1, 2, 37, len(counts)):
        t, refs = guarded(table, columns + 1), guarded(counts)
        out = t if in_place else Guarded((b, columns), columns + 2)
        refs_out = refs if in_place else Guarded((len(counts),))
        src, dst = Guarded((pairs,)), Guarded((pairs,))
        where = {} if in_place else dict(page_table_out=out.t, ref_counts_out=refs_out.t)
        m.sdpa_cache_compact(t.t, words(kept), refs.t, src.t, dst.t, page_size=page, **where)
        rows, cs, a, z = po.compact(table, kept, counts, pairs, page)
        assert src.check() == a and dst.check() == z and out.check() == rows and refs_out.check() == cs


@pytest.mark.parametrize("pages", [1, 7, 4096, 4097, 16385, 32769, 70000])
@pytest.mark.parametrize("used", [0.0, 0.03, 0.5, 0.97, 1.0])
def test_compact_of_any_number_of_pages(pages, used):
    """Shares of CTAs that the number of pages in use cuts in any place."""
    m, rng = lib(), np.random.default_rng(pages)
    counts = (rng.random(pages) < used).astype(np.int64) * rng.integers(1, 4, pages)
    movers = [p for p in range(pages) if counts[p]]
    lens, table = [16 * len(movers[:500])], [movers[:500] + [-1] * (501 - len(movers[:500]))]
    t, refs, src, dst = guarded(table), guarded(counts), Guarded((pages,)), Guarded((pages,))
    m.sdpa_cache_compact(t.t, words(lens), refs.t, src.t, dst.t, page_size=16)
    rows, cs, a, z = po.compact(table, lens, counts.tolist(), pages, 16)
    assert src.check() == a and dst.check() == z and t.check() == rows and refs.check() == cs


# ---- pages copied, rows kept -----------------------------------------------------------------

def raw(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


COPY = [
    # kind, h_kv, d, page, slot_major, pairs
    ("bf16", 8, 128, 64, True, 20), ("e4m3", 8, 128, 64, True, 20), ("f16", 3, 64, 16, False, 50), ("e4m3", 1, 256, 48, False, 3),
    ("e4m3", 12, 64, 16, True, 1), ("f16", 1, 128, 128, True, 7),
]


@pytest.mark.parametrize("kind,h,d,page,slot_major,pairs", COPY)
@pytest.mark.parametrize("padded", [False, True])
def test_copy(kind, h, d, page, slot_major, pairs, padded):
    m, rng = lib(), np.random.default_rng(pairs)
    c = make_cache((page * 2 * pairs + page,), h, d, page, kind, seed=5, slot_major=slot_major, spare=3, fill=1.0)
    k, v = c.k, c.v
    if padded:      # a cache inside a wider one: rows apart from each other
        wide = [torch.zeros(*x.shape[:-1], 2 * d, device="cuda").to(x.dtype) for x in (k, v)]
        for w, x in zip(wide, (k, v)):
            w[..., :d] = x
        k, v = (w[..., :d] for w in wide)
        rest = [raw(w[..., d:]) for w in wide]
    pages = k.shape[0]
    order = rng.permutation(pages)
    src, dst = order[:pairs].copy(), order[pairs:2 * pairs].copy()
    hide = rng.random(pairs) < 0.3
    bad = np.array([-1, -7, pages, 2 ** 31 - 1])[rng.integers(0, 4, pairs)]
    first = rng.random(pairs) < 0.5
    src, dst = np.where(hide & first, bad, src), np.where(hide & ~first, bad, dst)
    scales = [] if kind != "e4m3" else [c.k_scale, c.v_scale]
    want = [raw(x) for x in (k, v, *scales)]
    for w in want:
        for a, z, no in zip(src, dst, hide):
            if not no:
                w[z] = w[a]
    m.sdpa_cache_copy(k, v, words(src), words(dst), **c.scales())
    torch.cuda.synchronize()
    for x, w in zip((k, v, *scales), want):
        assert np.array_equal(raw(x), w)
    if padded:
        for w, r in zip(wide, rest):
            assert np.array_equal(raw(w[..., d:]), r)


def test_copy_with_a_list_that_is_mostly_empty():
    m = lib()
    c = make_cache((16 * 30,), 2, 64, 16, "f16", seed=6, fill=1.0)
    src, dst = np.full(50000, -1), np.full(50000, -1)
    src[[0, 33, 49999]], dst[[0, 33, 49999]] = (1, 2, 3), (10, 11, 12)
    want = raw(c.k), raw(c.v)
    for w in want:
        w[[10, 11, 12]] = w[[1, 2, 3]]
    m.sdpa_cache_copy(c.k, c.v, words(src), words(dst))
    assert np.array_equal(raw(c.k), want[0]) and np.array_equal(raw(c.v), want[1])


KEEP = [
    # lens_kv, lens_q, s, h, d, page, kind, slot_major
    ((100, 33, 64), None, 13, 2, 128, 16, "bf16", True), ((100, 33, 64), (13, 0, 20), 20, 3, 64, 16, "e4m3", False),
    ((500, 200), (150, 170), 170, 1, 256, 48, "e4m3", True), ((10, 3), (9, 7), 9, 12, 64, 16, "f16", True), ((1, 0), None, 1, 1, 128, 16, "f16", True),
]


@pytest.mark.parametrize("lens,lens_q,s,h,d,page,kind,slot_major", KEEP)
@pytest.mark.parametrize("path_kind", ["some", "all", "first", "bad"])
def test_keep(lens, lens_q, s, h, d, page, kind, slot_major, path_kind):
    m, rng, b = lib(), np.random.default_rng(s), len(lens)
    c = make_cache(lens, h, d, page, kind, seed=7, slot_major=slot_major, fill=1.0)
    table = c.page_table.cpu().numpy().copy()
    if path_kind == "bad":
        table[0, -1] = -1              # a missing page, and one outside
        table[-1, 0] = c.k.shape[0]
        c.page_table.copy_(torch.from_numpy(table))
    path, accepted = np.full((b, s), -1), np.zeros(b, np.int64)
    for i in range(b):
        n = s if lens_q is None else min(lens_q[i], s)
        keep = {"some": np.sort(rng.permutation(n)[: max(1, n // 2)]), "all": np.arange(n), "first": np.arange(min(n, 1)),
                "bad": np.sort(rng.permutation(n)[: max(1, 2 * n // 3)])}[path_kind][:n]
        path[i, : len(keep)] = keep
        accepted[i] = len(keep)
        if path_kind == "bad" and len(keep) > 2:
            path[i, len(keep) - 2:len(keep)] = (s, 2 ** 31 - 1)
            accepted[i] = s + 100 if i == 0 else len(keep)
    tensors = [c.k, c.v] + ([] if c.k_scale is None else [c.k_scale, c.v_scale])
    want = [raw(x) for x in tensors]

    def slots(i, pos):
        pg = table[i, pos // page]
        return (pg, pos % page) if 0 <= pg < c.k.shape[0] else None

    for w in want:
        w = w.reshape(c.k.shape[0], h, page, -1)
        for _, a, z in po.keep(slots, lens, lens_q, s, path, accepted):
            w[z[0], :, z[1]] = w[a[0], :, a[1]]
    lq = None if lens_q is None else words(lens_q)
    m.sdpa_cache_keep(*c.where(), words(path), words(accepted), seq_lens_q=lq, **c.scales())
    for x, w in zip(tensors, want):
        assert np.array_equal(raw(x), w)


@pytest.mark.parametrize("slot_major", [True, False])
def test_offsets_beyond_32_bits(slot_major):
    """A cache of 4.6 GB each of K and V: pages and rows at its far end."""
    m, page, h, d, pages = lib(), 64, 8, 128, 70000
    k, v = (torch.empty(pages, *((page, h) if slot_major else (h, page)), d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty(pages, h, page, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(1)
    far = [0, 3, 5, 32768, 65536, 69998, 69999]
    for x in (k, v):
        x[far] = torch.randint(0, 120, (len(far), *x.shape[1:]), generator=g, device="cuda", dtype=torch.uint8)
    for x in (ks, vs):
        x[far] = torch.rand(len(far), h, page, generator=g, device="cuda")
    view = lambda x: (x.view(torch.float8_e4m3fn).transpose(1, 2) if slot_major else x.view(torch.float8_e4m3fn))    # noqa: E731
    was = [x[far].clone() for x in (k, v, ks, vs)]
    m.sdpa_cache_copy(view(k), view(v), words([69999, 0, 65536]), words([3, 69998, 32768]), k_scale=ks, v_scale=vs)
    for x, w in zip((k, v, ks, vs), was):
        assert torch.equal(x[far], w[[0, 6, 2, 4, 4, 0, 6]])
    was = [x[far].clone() for x in (k, v, ks, vs)]
    # 10 new rows over the border of pages 69999 and 69998
    m.sdpa_cache_keep(view(k), view(v), words([[69999, 69998]]), words([70]), words([[0, 3, 7, 9] + [-1] * 6]), words([4]), k_scale=ks, v_scale=vs)
    for x, w, slot in zip((k, v, ks, vs), was, (1 if slot_major else 2,) * 2 + (2, 2)):
        w = w.transpose(1, slot).contiguous()           # slots second
        w[6, 61], w[6, 62], w[6, 63] = w[6, 63].clone(), w[5, 3].clone(), w[5, 5].clone()
        assert torch.equal(x[far].transpose(1, slot), w)


def test_pages_on_streams_and_captured():
    """Captured once, replayed on other lengths and tables; the calls follow each other without a wait."""
    m, page, b, columns = lib(), 16, 6, 40
    rng = np.random.default_rng(3)
    table, lens, counts = batch(rng, b, columns, page, 1, 200, missing=0.0)
    t, ln, new, refs, par = words(table), words(lens), words(lens), words(counts), words(range(b))
    out, refs_out, lens_out = torch.empty_like(t), torch.empty_like(refs), torch.empty_like(ln)
    src, dst, missing = torch.empty_like(ln), torch.empty_like(ln), words([0])
    moved = [torch.empty(64, dtype=torch.int32, device="cuda") for _ in range(2)]
    kept = torch.empty_like(ln)

    def step():
        m.sdpa_cache_fork(t, ln, par, refs, out, lens_out, refs_out, page_size=page)
        m.sdpa_cache_grow(out, lens_out, new, refs_out, src, dst, missing, page_size=page)
        m.sdpa_cache_free(out, new, kept, refs_out, page_size=page)
        m.sdpa_cache_compact(out, kept, refs_out, *moved, page_size=page)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(4):
        rng = np.random.default_rng(100 + seed)
        table, lens, counts = batch(rng, b, columns, page, 1, 200, missing=0.0)
        counts = (counts + [1] * refs.numel())[: refs.numel()]
        table = [[p if p < refs.numel() else -1 for p in row] for row in table]
        counts = [1 if rng.random() < 0.2 else 0 for _ in range(refs.numel())]
        for row, n in zip(table, lens):
            for p in row[: -(-n // page)]:
                if p >= 0:
                    counts[p] += 1
        parents = rng.integers(0, b, b)
        want = [lens[j] for j in parents]
        more = [min(n + int(rng.integers(0, 40)), columns * page) for n in want]
        less = [int(rng.integers(0, n + 1)) for n in more]
        for x, y in ((t, table), (ln, lens), (refs, counts), (par, parents), (new, more), (kept, less)):
            x.copy_(words(y))
        graph.replay()
        torch.cuda.synchronize()
        rows, ns, cs = po.fork(table, lens, parents, counts, page)
        got_rows, got_cs, a, z, lacked = po.grow(rows, ns, more, cs, page)
        rows, cs = (rows, cs) if lacked else (got_rows, got_cs)
        assert missing.tolist() == [lacked] and src.tolist() == a and dst.tolist() == z
        rows, cs = po.free(rows, more, less, cs, page)
        rows, cs, a, z = po.compact(rows, less, cs, 64, page)
        assert out.tolist() == rows and refs_out.tolist() == cs and moved[0].tolist() == a and moved[1].tolist() == z
