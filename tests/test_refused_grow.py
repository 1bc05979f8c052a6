"""The step of drafted trees as the package's front page shows it, with pages enough and with too few (GPU): a step that finds no room
for its rows writes none, reads nothing back to the host, and leaves what the sequences hold as it is."""
import os
import re

import numpy as np
import pytest
import torch

from oracle import pages_oracle as po
from sdpa_testlib import lib
from serving_testlib import make_cache, pack_tree, randn

pytestmark = pytest.mark.gpu

H_Q, H_KV, D, PAGE, S, VOCAB, B = 8, 2, 128, 16, 11, 997, 4
PARENTS = np.array([-1, 0, 0, 1, 1, 2, 3, 3, 6, 8, 8])
CHOSEN, LENS = [0, 1, 0, 0], [37, 90]


def readme_step():
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    step, = [x for x in blocks if "sdpa_cache_grow" in x]
    return compile(step, "step", "exec")


def state(kind, spare):
    m, g = lib(), torch.Generator().manual_seed(12)
    c = make_cache(LENS, H_KV, D, PAGE, kind, seed=13, spare=spare, wide=8, fill=0.5)
    int32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")    # noqa: E731
    empty = lambda *n: torch.full(n, -7, dtype=torch.int32, device="cuda")    # noqa: E731
    see = np.eye(S, dtype=bool)
    for j in range(1, S):
        see[j] |= see[PARENTS[j]]
    bf = lambda h: randn(g, B, S, h, D).bfloat16().cuda().permute(0, 2, 1, 3)    # noqa: E731
    q = bf(H_Q)
    probs = torch.softmax(randn(g, B, S, VOCAB) * 2, -1)
    tokens = np.zeros((B, S), np.int64)
    top = probs.argsort(-1, descending=True).numpy()
    for j in range(1, S):
        tokens[:, j] = top[:, PARENTS[j], sum(PARENTS[1:j] == PARENTS[j])]
    return dict(torch=torch, sdpa=m, b=B, h_q=H_Q, h_kv=H_KV, d=D, page=PAGE, s=S, k_cache=c.k, v_cache=c.v, scales=c.scales(),
                page_table=c.page_table, lens=c.lens, parents=int32(CHOSEN), new_table=empty(B, 8), new_lens=empty(B), src=empty(B), dst=empty(B),
                missing=empty(1), ref_counts=int32(np.bincount(c.page_table[c.page_table >= 0].cpu().numpy(), minlength=c.k.shape[0])),
                table=m.sdpa_rope_table(D)[0], positions=torch.randint(0, 500, (3, B, S), generator=g, dtype=torch.int32).cuda(), q=q, k=bf(H_KV),
                v=bf(H_KV), o=torch.empty_like(q), ws=torch.empty(1 << 24, dtype=torch.uint8, device="cuda"), tree_mask=pack_tree(np.stack([see] * B)).cuda(),
                tokens=int32(tokens), probs=probs.cuda(), uniform=torch.rand(B, S, generator=g).cuda() * 0.3, accepted=empty(B), path=empty(B, S),
                new_tokens=empty(B, S), tree_parents=int32(np.tile(PARENTS, (B, 1))))


def held(st):
    """Every byte that a program keeps: the cache, its scales, and the owners of its pages."""
    return [x.contiguous().view(torch.uint8).clone() for x in (st["k_cache"], st["v_cache"], *(x for x in st["scales"].values() if x is not None))]


def read(st, table, lens):
    out = [torch.empty(len(lens), H_KV, 8 * PAGE, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    st["sdpa"].sdpa_cache_read(st["k_cache"], st["v_cache"], table, lens, *out, **st["scales"])
    return [x.view(torch.int16).cpu().numpy() for x in out]


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("spare", [0, 2, 3, 9])
def test_readme_step(kind, spare, captured):
    st, step = state(kind, spare), readme_step()
    was, table, counts = held(st), st["page_table"].tolist(), st["ref_counts"].clone()
    history = read(st, st["page_table"], st["lens"])
    rows, lens, owners = po.fork(table, LENS, CHOSEN, counts.tolist(), PAGE)
    lacked = po.grow(rows, lens, [n + S for n in lens], owners, PAGE)[4]
    assert lacked == max(0, 3 - spare)
    if captured:
        exec(step, st)                   # (what a first call does once)
        st["ref_counts"].copy_(counts)
        for x, w in zip((st["k_cache"], st["v_cache"], *(x for x in st["scales"].values() if x is not None)), was):
            x.copy_(w.view(x.dtype))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            exec(step, st)
        graph.replay()
    else:
        exec(step, st)
    torch.cuda.synchronize()
    accepted = st["accepted"].tolist()
    assert st["missing"].tolist() == [lacked] and st["new_lens"].tolist() == lens
    now = read(st, st["new_table"], st["new_lens"])
    for x, y in zip(history, now):
        for i, j in enumerate(CHOSEN):
            assert np.array_equal(x[j, :, : lens[i]], y[i, :, : lens[i]]), "a sequence's rows changed"
    if lacked:
        assert accepted == [0] * B and st["ref_counts"].tolist() == owners and st["new_table"].tolist() == rows
        assert all(torch.equal(x, y) for x, y in zip(held(st), was))
        assert (st["path"] == -1).all() and (st["new_tokens"] == -1).all()
    else:
        want = po.verify(st["tokens"].cpu().numpy(), st["probs"].cpu().numpy(), st["uniform"].cpu().numpy(), st["tree_parents"].cpu().numpy())
        assert accepted == want[0].tolist() and max(accepted) > 1 and np.array_equal(st["new_tokens"].cpu().numpy(), want[2])
        counts = np.zeros(len(owners), np.int64)
        for row, n, a in zip(st["new_table"].tolist(), lens, accepted):
            for page in row[: -(-(n + a) // PAGE)]:
                counts[page] += 1
        assert st["ref_counts"].tolist() == counts.tolist()
