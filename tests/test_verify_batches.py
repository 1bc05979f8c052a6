"""Verification of batches in which four and two CTAs share a sequence, and of the longest rows that two of them share (GPU)."""
import numpy as np
import pytest
import torch

from sdpa_testlib import lib
from test_verify_parity import DT, check, distributions, random_parents, view

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b", [77, 100, 153, 160, 310])
@pytest.mark.parametrize("dtype,vocab,offset", [("f32", 1003, 0), ("bf16", 260, 3)])
def test_batches(b, dtype, vocab, offset):
    rng, s = np.random.default_rng(b + vocab), 4
    p = distributions(rng, b, s, vocab)
    probs = view(p, dtype, 1, offset)
    near = np.roll(p, 1, 1) ** 0.9 * np.exp(0.3 * rng.normal(size=p.shape))
    q = (near / near.sum(-1, keepdims=True)).astype(np.float32)
    tokens = np.minimum(vocab - 1, (np.cumsum(q, -1) < rng.random((b, s, 1))).sum(-1))
    uniform, lens = rng.random((b, s), dtype=np.float32), rng.integers(-1, s + 2, b)
    check(tokens, probs, uniform, draft=view(q, dtype, 0, offset), lens=lens)
    check(tokens, probs, uniform, lens=lens)
    parents = random_parents(rng, b, s)
    top = np.argsort(-p, -1, kind="stable")[..., :3]
    for i in range(b):
        for j in range(1, s):
            tokens[i, j] = top[i, parents[i, j], rng.integers(0, 3)]
    a, _, _ = check(tokens, probs, uniform, parents)
    assert a.max() > 1


def drawn(row, u):
    """The definition in whole numbers of 2^-42, which 64 bits hold (a total of 2^62 at most)."""
    mass = torch.round(row.double().clamp(0, 1) * 2.0 ** 42).long()
    sums = torch.cumsum(mass, 0)
    total = int(sums[-1])
    at = [total * min(int(float(x) * 2 ** 31), 2 ** 31 - 1) >> 31 for x in u]
    return torch.searchsorted(sums, torch.tensor(at, device=row.device), right=True).tolist()


@pytest.mark.parametrize("b", [1, 100, 160, 200])
@pytest.mark.parametrize("dtype,vocab,offset", [("f32", 1 << 20, 3), ("f32", 1 << 20, 0), ("bf16", 1 << 20, 7), ("f16", (1 << 20) - 5, 1), ("f32", 131072, 2), ("f32", 3, 1)])
def test_long_rows(b, dtype, vocab, offset):
    """One row for all sequences, drawn from at random numbers that end in every part of it."""
    m, g = lib(), torch.Generator(device="cuda").manual_seed(vocab + offset)
    row = torch.full((offset + vocab + 9,), float("nan"), dtype=DT[dtype], device="cuda")[offset:offset + vocab]
    row.copy_(torch.rand(vocab, generator=g, device="cuda") * (1.0 if dtype == "f16" else 2.0 / vocab))
    u = torch.cat((torch.linspace(0, 1, b, device="cuda", dtype=torch.float64)[:-1].float(), torch.tensor([1 - 2.0 ** -24], device="cuda")))
    a, path, new = (torch.full((b, n), -9, dtype=torch.int32, device="cuda") for n in (1, 1, 1))
    zeros = torch.zeros(b, 1, dtype=torch.int32, device="cuda")
    m.sdpa_verify(zeros, row.expand(b, 1, vocab), u[:, None].contiguous(), a[:, 0].contiguous(), path, new)
    assert new[:, 0].tolist() == drawn(row, u.tolist())
    assert (path == 0).all()
