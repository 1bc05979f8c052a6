"""The serving operators in a row, as a program that drafts trees uses them: beams forked and grown (with the copies of shared pages),
drafted rows rotated on several axes and written, attention of the tree, verification, accepted rows kept, the rest freed, the cache
compacted (GPU)."""
import numpy as np
import pytest
import torch

from oracle import pages_oracle as po
from oracle import serving_oracle as so
from sdpa_testlib import f64, lib
from serving_testlib import assert_attend_close, kv_rounding, make_cache, pack_tree, randn

pytestmark = pytest.mark.gpu

H_Q, H_KV, D, PAGE, S, VOCAB = 8, 2, 128, 16, 11, 997
PARENTS = np.array([-1, 0, 0, 1, 1, 2, 3, 3, 6, 8, 8])


def int32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def seen(parents):
    see = np.eye(len(parents), dtype=bool)
    for j in range(1, len(parents)):
        see[j] |= see[parents[j]]
    return see


class Server:
    """What a program holds: a cache, tables and counts, and the buffers of a step for `b` sequences (2 before the first step)."""

    def __init__(self, kind, b, seed):
        m, g = lib(), torch.Generator().manual_seed(seed)
        self.m, self.kind, self.b = m, kind, b
        self.cache = make_cache((37, 90), H_KV, D, PAGE, kind, seed=seed, spare=40, wide=12, fill=0.5)
        self.table, self.lens = self.cache.page_table, self.cache.lens
        pages = self.cache.k.shape[0]
        self.refs = int32(np.bincount(self.table[self.table >= 0].cpu().numpy(), minlength=pages))
        self.new_table = torch.full((b, 12), -7, dtype=torch.int32, device="cuda")
        empty = lambda *n: torch.empty(*n, dtype=torch.int32, device="cuda")    # noqa: E731
        self.fork_lens, self.grown, self.src, self.dst, self.missing = empty(b), empty(b), empty(b), empty(b), empty(1)
        self.moved = empty(pages), empty(pages)
        self.accepted, self.path, self.new_tokens, self.kept = empty(b), empty(b, S), empty(b, S), empty(b)
        self.rope, _ = m.sdpa_rope_table(D)
        self.axes = m.sdpa_rope_axes((16, 24, 24), order="interleaved")
        bf = lambda *n: randn(g, *n).bfloat16().cuda()    # noqa: E731
        self.q, self.k, self.v = (bf(b, S, h, D).permute(0, 2, 1, 3) for h in (H_Q, H_KV, H_KV))
        self.o, self.lse = torch.empty_like(self.q), torch.empty(b, H_Q, S, device="cuda")
        self.head = randn(g, H_Q * D, VOCAB).cuda() * 0.3
        self.parents = int32(np.tile(PARENTS, (b, 1)))
        self.tokens, self.uniform = torch.zeros(b, S, dtype=torch.int32, device="cuda"), torch.rand(b, S, generator=g).cuda()
        self.depth = int32([seen(PARENTS)[j].sum() - 1 for j in range(S)])
        self.tree = pack_tree(np.stack([seen(PARENTS)] * b)).cuda()
        self.work = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")

    def where(self):
        return self.cache.k, self.cache.v, self.new_table, self.grown

    def step(self, chosen, check=None):
        m, c, z = self.m, self.cache, dict(page_size=PAGE)
        scales = c.scales()
        m.sdpa_cache_fork(self.table, self.lens, chosen, self.refs, self.new_table, self.fork_lens, **z)
        torch.add(self.fork_lens, S, out=self.grown)
        m.sdpa_cache_grow(self.new_table, self.fork_lens, self.grown, self.refs, self.src, self.dst, self.missing, **z)
        m.sdpa_cache_copy(c.k, c.v, self.src, self.dst, **scales)
        # Drafted tokens stand on the time axis by their depth, and in a grid of their own.
        time = self.fork_lens[:, None] + self.depth
        self.pos = torch.stack((time, self.depth.expand_as(time), (2 * self.depth).expand_as(time))).contiguous()
        qr = torch.empty_like(self.q)
        m.sdpa_rope_fwd(self.q, None, qr, None, self.rope, self.pos, axes=self.axes)
        m.sdpa_cache_write(self.k, self.v, *self.where(), **scales, rope_table=self.rope, positions=self.pos, axes=self.axes)
        m.sdpa_decode(qr, *self.where(), self.o, self.lse, workspace=self.work, tree_mask=self.tree, **scales)
        self.qr = qr
        self.probs = torch.softmax(self.o.permute(0, 2, 1, 3).reshape(self.b, S, -1).float() @ self.head, -1)
        # The draft: the target's likeliest tokens behind each row's parent, by rank among its siblings.
        top = torch.topk(self.probs, 4, -1).indices
        rank = [sum(PARENTS[i] == PARENTS[j] for i in range(1, j)) for j in range(S)]
        for j in range(1, S):
            self.tokens[:, j] = top[:, PARENTS[j], rank[j]].to(torch.int32)
        m.sdpa_verify(self.tokens, self.probs, self.uniform, self.accepted, self.path, self.new_tokens, parents=self.parents)
        if check:
            check()
        m.sdpa_cache_keep(*self.where(), self.path, self.accepted, **scales)
        torch.add(self.fork_lens, self.accepted, out=self.kept)
        m.sdpa_cache_free(self.new_table, self.grown, self.kept, self.refs, **z)
        m.sdpa_cache_compact(self.new_table, self.kept, self.refs, *self.moved, **z)
        m.sdpa_cache_copy(c.k, c.v, *self.moved, **scales)

    def read(self, table, lens):
        n, out = 12 * PAGE, []
        for _ in range(2):
            out.append(torch.empty(table.shape[0], H_KV, n, D, dtype=torch.bfloat16, device="cuda"))
        self.m.sdpa_cache_read(self.cache.k, self.cache.v, table, lens, *out, **self.cache.scales())
        torch.cuda.synchronize()
        return [x.view(torch.int16).cpu().numpy() for x in out]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_steps(kind):
    sv = Server(kind, 4, 30)
    history = sv.read(sv.table, sv.lens)
    lens = sv.lens.tolist()
    for turn, chosen in enumerate(([0, 1, 0, 0], [2, 2, 1, 3], [3, 0, 0, 1])):
        before = [[x[j, :, : lens[j]] for j in chosen] for x in history]
        lens = [lens[j] for j in chosen]
        drafted = []

        def check():
            """The drafted rows stand behind what each beam took over, whoever else holds those pages."""
            assert sv.missing.item() == 0 and sv.fork_lens.tolist() == lens
            now = sv.read(sv.new_table, sv.grown)
            for x, was in zip(now, before):
                for i, n in enumerate(lens):
                    assert np.array_equal(x[i, :, :n], was[i]) and (x[i, :, n + S:] == 0).all()
            drafted.extend(now)
            c = sv.cache
            c.page_table, c.lens = sv.new_table, sv.grown
            freqs, _ = so.inv_freq(D)
            turned, reach = po.rotate_axes(f64(sv.q), sv.pos.cpu().numpy(), sv.axes, freqs)
            assert (np.abs(f64(sv.qr) - turned) <= 2.0 ** -8 * np.abs(turned) * 1.01 + 2.0 ** -20 * reach).all()
            kv, vv, ks, vs, tb = c.np()
            ref = so.attend(f64(sv.qr), kv, vv, ks, vs, tb, [n + S for n in lens], None, D ** -0.5, False, np.stack([seen(PARENTS)] * 4))
            assert_attend_close(sv.o, sv.lse, ref, "bf16", "f16" if kind == "e4m3" else "bf16", f"turn {turn}", kv_rounding(kind, S * H_Q // H_KV, D, "bf16"))
            want = po.verify(sv.tokens.cpu().numpy(), sv.probs.cpu().numpy(), sv.uniform.cpu().numpy(), sv.parents.cpu().numpy())
            assert all(np.array_equal(x.cpu().numpy(), w) for x, w in zip((sv.accepted, sv.path, sv.new_tokens), want))

        sv.step(int32(chosen), check)
        # Each sequence is what it was, and its accepted rows; pages in use are the first ones.
        accepted, path = sv.accepted.tolist(), sv.path.tolist()
        history = sv.read(sv.new_table, sv.kept)
        for x, was, draft in zip(history, before, drafted):
            for i, n in enumerate(lens):
                rows = draft[i][:, [n + r for r in path[i][: accepted[i]]]]
                assert np.array_equal(x[i, :, :n], was[i]) and np.array_equal(x[i, :, n: n + accepted[i]], rows)
                assert (x[i, :, n + accepted[i]:] == 0).all()
        lens = [n + a for n, a in zip(lens, accepted)]
        counts = sv.refs.tolist()
        table = sv.new_table.tolist()
        want = np.zeros(len(counts), np.int64)
        for row, n in zip(table, lens):
            for page in row[: -(-n // PAGE)]:
                want[page] += 1
        assert counts == want.tolist() and all(x > 0 for x in counts[: int((want > 0).sum())])
        # The next step's old table is this one's new one.
        sv.table, sv.lens = sv.new_table.clone(), int32(lens)


def test_a_captured_step_gives_what_an_eager_one_gives():
    chosen = int32([1, 0, 0, 1])
    eager, other = Server("e4m3", 4, 31), Server("e4m3", 4, 31)
    eager.step(chosen)
    state = [other.refs, other.cache.k, other.cache.v, other.cache.k_scale,
             other.cache.v_scale]
    saved = [x.clone() for x in state]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other.step(chosen)
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip(state, saved):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        other.step(chosen)
    for _ in range(2):
        for x, y in zip(state, saved):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        for name in ("refs", "new_table", "kept", "accepted", "path", "new_tokens"):
            assert torch.equal(getattr(eager, name), getattr(other, name)), name
        for x, y in zip(eager.read(eager.new_table, eager.kept), other.read(other.new_table, other.kept)):
            assert np.array_equal(x, y)
