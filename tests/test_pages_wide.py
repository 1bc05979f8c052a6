"""Page calls of tables that go over the whole GPU, with counts kept apart: behind each other without a wait, and captured (GPU)."""
import numpy as np
import pytest
import torch

from oracle import pages_oracle as po
from sdpa_testlib import lib
from test_pages_parity import batch, words

pytestmark = pytest.mark.gpu

PAGE = 16


class Step:
    """fork, grow, free and compact in a row; `apart`: each call's table and counts go elsewhere, so that one launch or copy follows another."""

    def __init__(self, b, columns, pages, apart):
        empty = lambda *n: torch.full(n, -7, dtype=torch.int32, device="cuda")    # noqa: E731
        self.apart, self.b, self.columns, self.pages = apart, b, columns, pages
        self.tables, self.counts = [empty(b, columns) for _ in range(5)], [empty(pages) for _ in range(5)]
        self.lens, self.parents, self.forked, self.more, self.less = (empty(b) for _ in range(5))
        self.src, self.dst, self.missing = empty(b), empty(b), empty(1)
        self.moved = empty(pages // 2), empty(pages // 2)

    def run(self):
        m, t, c, z = lib(), self.tables, self.counts, dict(page_size=PAGE)
        if self.apart:
            out = [dict(page_table_out=t[i], ref_counts_out=c[i]) for i in (2, 3, 4)]
        else:
            t, c, out = [t[0], t[1], t[1], t[1], t[1]], [c[0]] * 5, [{}] * 3
        m.sdpa_cache_fork(t[0], self.lens, self.parents, c[0], t[1], self.forked, c[1] if self.apart else None, **z)
        m.sdpa_cache_grow(t[1], self.forked, self.more, c[1], self.src, self.dst, self.missing, **z, **out[0])
        m.sdpa_cache_free(t[2], self.more, self.less, c[2], **z, **out[1])
        m.sdpa_cache_compact(t[3], self.less, c[3], *self.moved, **z, **out[2])
        self.last = t[4], c[4]

    def fill(self, seed):
        rng = np.random.default_rng(seed)
        table, lens, counts = batch(rng, self.b, self.columns, PAGE, 1, 40, missing=0.02)
        n = len(counts)
        assert n <= self.pages
        counts = counts + [0 if rng.random() < 0.9 else 1 for _ in range(self.pages - n)]
        parents = rng.integers(-1, self.b + 1, self.b)
        kept = [lens[j] if 0 <= j < self.b else 0 for j in parents]
        more = [min(n + int(rng.integers(0, 60)), self.columns * PAGE) for n in kept]
        less = [int(rng.integers(0, n + 1)) for n in more]
        for x, y in ((self.tables[0], table), (self.lens, lens), (self.counts[0], counts), (self.parents, parents), (self.more, more), (self.less, less)):
            x.copy_(words(y))
        rows, ns, cs = po.fork(table, lens, parents, counts, PAGE)
        grown, more_cs, a, z, lacked = po.grow(rows, ns, more, cs, PAGE)
        rows, cs = (rows, cs) if lacked else (grown, more_cs)
        rows, cs = po.free(rows, more, less, cs, PAGE)
        rows, cs, x, y = po.compact(rows, less, cs, self.pages // 2, PAGE)
        return rows, cs, a, z, lacked, x, y

    def check(self, want):
        rows, cs, a, z, lacked, x, y = want
        assert self.missing.tolist() == [lacked] and self.src.tolist() == a and self.dst.tolist() == z
        assert self.last[0].tolist() == rows and self.last[1].tolist() == cs
        assert self.moved[0].tolist() == x and self.moved[1].tolist() == y


@pytest.mark.parametrize("apart", [True, False])
@pytest.mark.parametrize("b,columns,pages", [(64, 600, 40000), (300, 40, 14000), (20, 128, 4000)])
def test_wide_tables_in_a_row_and_captured(b, columns, pages, apart):
    step = Step(b, columns, pages, apart)
    for seed in range(2):
        want = step.fill(seed)
        torch.cuda.synchronize()
        step.run()
        torch.cuda.synchronize()
        step.check(want)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step.run()
    for seed in range(2, 5):
        want = step.fill(seed)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        step.check(want)


def test_captured_twice_and_replayed_in_turn():
    """Two graphs of calls of several sizes, with nothing of their own but their operands."""
    steps = [Step(64, 600, 40000, True), Step(20, 128, 4000, True)]
    graphs = []
    for s in steps:
        s.fill(9)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    wants = [s.fill(20 + i) for i, s in enumerate(steps)]
    torch.cuda.synchronize()
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for s, w in zip(steps, wants):
        s.check(w)
