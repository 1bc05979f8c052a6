"""Verified drafts against the oracle: whole numbers, so results are equal (GPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import pages_oracle as po
from sdpa_testlib import lib

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
MARK = 0x5A5A5A5A


def distributions(rng, b, s, vocab, sharp=2.5):
    x = rng.normal(size=(b, s, vocab)) * sharp
    x = np.exp(x - x.max(-1, keepdims=True))
    return (x / x.sum(-1, keepdims=True)).astype(np.float32)


def values(t):
    return t.float().cpu().numpy()


def view(x, dtype, row_pad=0, offset=0, batch_pad=0):
    """A [b, s, vocab] tensor of these values whose rows lie row_pad elements apart and start `offset` elements into an allocation."""
    b, s, vocab = x.shape
    t = torch.from_numpy(np.ascontiguousarray(x)).to(DT[dtype])
    row = vocab + row_pad
    buf = torch.full((offset + b * (s * row + batch_pad),), float("nan"), dtype=DT[dtype], device="cuda")
    out = buf.as_strided((b, s, vocab), (s * row + batch_pad, row, 1), offset)
    out.copy_(t)
    return out


def run(tokens, probs, uniform, parents=None, draft=None, lens=None, stream=None):
    b, s = tokens.shape
    dev = lambda x: None if x is None else torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")    # noqa: E731
    outs = [torch.full((n + 64,), MARK, dtype=torch.int32, device="cuda") for n in (b, b * s, b * s)]
    a, path, new = outs[0][32:32 + b], outs[1][32:32 + b * s].view(b, s), outs[2][32:32 + b * s].view(b, s)
    lib().sdpa_verify(dev(tokens), probs, torch.tensor(np.asarray(uniform, dtype=np.float32), device="cuda"), a, path, new, parents=dev(parents),
                      draft_probs=draft, seq_lens_q=dev(lens), stream=stream)
    torch.cuda.synchronize()
    for o in outs:
        assert (o[:32] == MARK).all() and (o[-32:] == MARK).all(), "written outside the tensor"
    return a.cpu().numpy(), path.cpu().numpy(), new.cpu().numpy()


def check(tokens, probs, uniform, parents=None, draft=None, lens=None):
    got = run(tokens, probs, uniform, parents, draft, lens)
    want = po.verify(tokens, values(probs), np.asarray(uniform, dtype=np.float32), parents, None if draft is None else values(draft), lens)
    for g, w, name in zip(got, want, ("accepted", "path", "new_tokens")):
        assert np.array_equal(g, w), (name, np.argwhere(g != w)[:5], g[g != w][:5], w[g != w][:5])
    return got


def random_parents(rng, b, s, reach=6):
    p = np.full((b, s), -1)
    for j in range(1, s):
        p[:, j] = rng.integers(max(0, j - reach), j, b)
    return p


CASES = [
    # b, s, vocab, dtype, mode, row_pad, offset
    (1, 1, 1, "f32", "chain", 0, 0), (3, 2, 7, "f32", "draft", 0, 0), (2, 5, 33, "bf16", "draft", 3, 1), (4, 5, 1000, "f32", "draft", 0, 0),
    (2, 6, 32000, "f16", "draft", 0, 0), (3, 4, 50257, "f32", "draft", 0, 0), (3, 4, 50257, "bf16", "draft", 0, 3), (2, 8, 4099, "f16", "chain", 5, 7),
    (5, 13, 1003, "f32", "tree", 0, 1), (2, 64, 5000, "bf16", "tree", 2, 0), (1, 300, 200, "f16", "tree", 0, 0), (2, 3, 131072, "f32", "draft", 0, 0),
    (20, 3, 65, "f32", "tree", 1, 2), (1, 2, 1 << 20, "bf16", "chain", 0, 0), (1, 2, (1 << 20) - 3, "f32", "draft", 0, 0), (400, 2, 130, "bf16", "draft", 6, 0),
]


@pytest.mark.parametrize("b,s,vocab,dtype,mode,row_pad,offset", CASES)
def test_verify(b, s, vocab, dtype, mode, row_pad, offset):
    rng = np.random.default_rng(vocab + s)
    p = distributions(rng, b, s, vocab)
    probs = view(p, dtype, row_pad, offset, batch_pad=offset)
    uniform = rng.random((b, s), dtype=np.float32)
    parents = draft = None
    if mode == "tree":
        parents = random_parents(rng, b, s)
        top = np.argsort(-p, -1, kind="stable")[..., :4]
        tokens = np.zeros((b, s), np.int64)
        for i in range(b):
            for j in range(1, s):
                tokens[i, j] = top[i, parents[i, j], min(rng.integers(0, 4), vocab - 1)]      # (siblings with one token among them)
    else:
        near = np.roll(p, 1, 1) ** 0.9 * np.exp(0.3 * rng.normal(size=p.shape))
        q = (near / near.sum(-1, keepdims=True)).astype(np.float32)
        tokens = np.array([[min(vocab - 1, int(np.searchsorted(np.cumsum(q[i, j]), rng.random()))) for j in range(s)] for i in range(b)])
        if mode == "draft":
            draft = view(q, dtype, 0, offset)
    check(tokens, probs, uniform, parents, draft)
    a, _, _ = check(tokens, probs, np.zeros_like(uniform), parents, draft)
    assert s == 1 or a.max() > 1                     # (0 accepts whatever the target has any of)
    check(tokens, probs, np.full_like(uniform, np.nextafter(np.float32(1), np.float32(0))), parents, draft)
    lens = rng.integers(-1, s + 2, b)
    check(tokens, probs, uniform, parents, draft, lens)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_split_and_alignment_do_not_matter(dtype):
    """The same rows at every offset from 16 bytes, the draft's at another."""
    rng = np.random.default_rng(1)
    p, q = distributions(rng, 2, 3, 777), distributions(rng, 2, 3, 777)
    tokens, uniform = rng.integers(0, 777, (2, 3)), rng.random((2, 3), dtype=np.float32)
    first = None
    for offset in range(9):
        got = run(tokens, view(p, dtype, 0, offset), uniform, draft=view(q, dtype, offset % 4, (5 * offset) % 8))
        first = first or got
        assert all(np.array_equal(x, y) for x, y in zip(got, first))


def test_draws_of_every_token():
    """One sequence a random number: the drawn token steps through the vocabulary as the running sum says, at the borders too."""
    vocab, n = 129, 600
    p = distributions(np.random.default_rng(2), 1, 1, vocab, 1.0)
    sums = np.cumsum(p[0, 0].astype(np.float64))
    u = np.concatenate([np.linspace(0, 1, n - vocab, endpoint=False), sums / sums[-1] * (1 - 2.0 ** -24)]).astype(np.float32)[:, None]
    a, _, new = check(np.zeros((n, 1), np.int64), view(np.repeat(p, n, 0), "f32"), u)
    assert (a == 1).all() and set(new[:, 0]) == set(range(vocab))


def test_values_that_are_no_probabilities():
    """NaN, infinities, negative values, sums far from one, rows of zeros."""
    vocab = 5000
    rng = np.random.default_rng(3)
    p = distributions(rng, 8, 3, vocab)
    p[0, :, 10] = np.nan
    p[1, :, 20], p[1, :, 21] = np.inf, -np.inf
    p[2, :, ::2] = -1.0
    p[3] = 1.0                               # a total of 5000
    p[4] = 0.0
    p[5, 1:] = np.nan
    p[6] *= 2.0 ** -30
    p[7, 0], p[7, 0, 1234] = 0.0, 1.0
    q = distributions(rng, 8, 3, vocab)
    q[1, :, 20] = np.inf
    q[2, 1, 4] = np.nan
    tokens = np.array([[0, 10, 10], [0, 20, 21], [0, 4, 5], [0, 1, 2], [0, 3, 4], [0, 7, 8], [0, 9, 9], [0, 1234, 1]])
    for u in (rng.random((8, 3), dtype=np.float32), np.zeros((8, 3)), np.full((8, 3), 0.999)):
        for kw in ({}, dict(draft=view(q, "f32")), dict(parents=np.array([[-1, 0, 0]] * 8))):
            a, _, new = check(tokens, view(p, "f32"), u, **kw)
            assert new[4, a[4] - 1] == -1
    for u in ((np.nan, 0.5, 0.5), (1.0, 2.0, 1.0), (-1.0, -0.5, 0.5), (np.inf, np.inf, -np.inf), (0.25, np.nan, np.nan)):
        for kw in ({}, dict(draft=view(q, "f32")), dict(parents=np.array([[-1, 0, 0]] * 8))):
            check(tokens, view(p, "f32"), np.array([u] * 8), **kw)


def test_a_large_total():
    """2^20 tokens of one each: a total of 2^62, drawn from without a loss."""
    vocab = 1 << 20
    probs = torch.ones(1, 1, vocab, device="cuda", dtype=torch.bfloat16)
    for u, want in ((0.0, 0), (0.5, vocab // 2), (1 - 2.0 ** -24, vocab - 1), (2.0 ** -20, 1), (0.3, math.floor(float(np.float32(0.3)) * vocab))):
        _, _, new = run(np.zeros((1, 1)), probs, [[u]])
        assert new[0, 0] == want


def test_what_is_left_of_equal_distributions():
    """The draft is the target: a refused token (only where the target has none of it) leaves nothing, and the target itself is drawn from."""
    rng = np.random.default_rng(4)
    p = distributions(rng, 6, 2, 300)
    p[:, 0, 7] = 0.0
    q = p[:, [1, 0]]
    tokens, uniform = np.full((6, 2), 7), rng.random((6, 2), dtype=np.float32)
    a, _, new = check(tokens, view(p, "f32"), uniform, draft=view(q, "f32"))
    assert (a == 1).all() and (new[:, 0] >= 0).all()
    # all of the target's mass on the tokens of the refused children
    p = np.zeros((1, 3, 4), np.float32)
    p[0, 0, :2] = 0.25
    a, _, new = check(np.array([[0, 0, 1]]), view(p, "f32"), [[0.9, 0.9, 0.9]], parents=np.array([[-1, 0, 0]]))
    assert a[0] == 1 and new[0, 0] == 1


def test_tokens_and_parents_out_of_range():
    rng = np.random.default_rng(5)
    b, s, vocab = 8, 6, 90
    p = distributions(rng, b, s, vocab, 0.5)
    tokens = rng.integers(0, vocab, (b, s))
    tokens[0, 1], tokens[1, 2], tokens[2, 1], tokens[3, 3] = -1, vocab, 2 ** 31 - 1, -2 ** 31
    tokens[:, 0] = -12345                                    # row 0's is not read
    parents = np.array([[77, 0, 1, 2, 3, 4]] * b)
    parents[4] = (0, 1, 2, 3, 4, 5)                          # every row its own
    parents[5] = (0, 0, 5, 1, -1, 3)
    parents[6] = (0, 3, 0, 2, 2 ** 31 - 1, -2 ** 31)
    for u in (np.zeros((b, s)), rng.random((b, s)) * 0.02):
        check(tokens, view(p, "f32"), u)
        check(tokens, view(p, "f32"), u, draft=view(distributions(rng, b, s, vocab, 0.5), "f32"))
        check(tokens, view(p, "f32"), u, parents)


@pytest.mark.parametrize("shape", ["star", "path", "random"])
def test_the_largest_trees(shape):
    rng = np.random.default_rng(6)
    s, vocab = 1024, 1500
    parents = {"star": np.zeros((1, s), np.int64), "path": np.arange(-1, s - 1)[None], "random": random_parents(rng, 1, s, 40)}[shape]
    parents[0, 0] = -1
    p = distributions(rng, 1, s, vocab, 0.3)
    tokens = rng.integers(0, vocab, (1, s))
    if shape == "path":
        p[:] = 0.0
        for j in range(1, s):
            p[0, j - 1, tokens[0, j]] = 1.0
        p[0, s - 1, 3] = 1.0
    uniform = rng.random((1, s), dtype=np.float32)
    a, _, new = check(tokens, view(p, "f32"), uniform, parents)
    if shape == "path":
        assert a[0] == s and new[0, -1] == 3
    check(tokens, view(p, "f32"), np.zeros_like(uniform), parents)


def test_tokens_are_distributed_as_the_targets():
    """20000 sequences of one drafted token: the first new token's frequencies are the target's within five standard deviations,
    with the draft's probabilities and without."""
    rng, n, vocab = np.random.default_rng(7), 20000, 8
    p, q = distributions(rng, 1, 2, vocab, 1.0), distributions(rng, 1, 1, vocab, 1.0)
    tokens = np.zeros((n, 2), np.int64)
    tokens[:, 1] = rng.choice(vocab, n, p=q[0, 0].astype(np.float64) / q[0, 0].astype(np.float64).sum())
    uniform = rng.random((n, 2), dtype=np.float32)
    probs, draft = view(p, "f32").expand(n, 2, vocab), view(np.repeat(q, 2, 1), "f32").expand(n, 2, vocab)
    for kw in ({}, dict(draft=draft), dict(parents=np.array([[-1, 0]] * n))):
        _, _, new = run(tokens, probs, uniform, **kw)
        share = np.bincount(new[:, 0], minlength=vocab) / n
        assert (np.abs(share - p[0, 0]) <= 5 * np.sqrt(p[0, 0] * (1 - p[0, 0]) / n)).all()


def test_offsets_beyond_32_bits():
    """Sequences 2^31 + 9 elements apart."""
    rng = np.random.default_rng(9)
    b, s, vocab, apart = 3, 3, 501, (1 << 31) + 9
    p, q = distributions(rng, b, s, vocab), distributions(rng, b, s, vocab)
    big = [torch.empty((b - 1) * apart + s * vocab, dtype=torch.bfloat16, device="cuda").as_strided((b, s, vocab), (apart, vocab, 1)) for _ in range(2)]
    for t, x in zip(big, (p, q)):
        t.copy_(torch.from_numpy(x).bfloat16())
    tokens = rng.integers(0, vocab, (b, s))
    for u in (rng.random((b, s), dtype=np.float32), np.full((b, s), 0.9), np.zeros((b, s))):
        check(tokens, big[0], u, draft=big[1])
        check(tokens, big[0], u, np.array([[-1, 0, 0]] * b))


def test_verify_on_streams_and_captured():
    rng = np.random.default_rng(8)
    b, s, vocab = 5, 4, 3001
    m = lib()
    sets = []
    for _ in range(3):
        p, q = distributions(rng, b, s, vocab), distributions(rng, b, s, vocab)
        sets.append((rng.integers(0, vocab, (b, s)), view(p, "f32"), rng.random((b, s), dtype=np.float32) * 0.3, view(q, "f32")))
    want = [po.verify(t, values(p), u, draft=values(q)) for t, p, u, q in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    held = []
    torch.cuda.synchronize()
    for (t, p, u, q), st in zip(sets, streams):
        x = torch.tensor(t, dtype=torch.int32, device="cuda"), torch.tensor(u, device="cuda")
        held.append((x, torch.empty(b, dtype=torch.int32, device="cuda"), *(torch.empty(b, s, dtype=torch.int32, device="cuda") for _ in range(2))))
    torch.cuda.synchronize()
    for _ in range(8):
        for (t, p, u, q), st, (x, a, path, new) in zip(sets, streams, held):
            with torch.cuda.stream(st):
                m.sdpa_verify(x[0], p, x[1], a, path, new, draft_probs=q)
    torch.cuda.synchronize()
    for w, (_, *got) in zip(want, held):
        assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(got, w))
    (tok, uni), a, path, new = held[0]
    p, q = sets[0][1].clone(), sets[0][3].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.sdpa_verify(tok, p, uni, a, path, new, draft_probs=q)
    for (t, p1, u, q1), w in zip(sets, want):
        tok.copy_(torch.tensor(t, dtype=torch.int32))
        uni.copy_(torch.tensor(u))
        p.copy_(p1)
        q.copy_(q1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip((a, path, new), w))
