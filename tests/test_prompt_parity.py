"""Rotations and cache writes of prompts, where a thread walks several heads (GPU): against the fp64 oracle on sampled tokens.

How many heads a thread walks goes by the size of the call: with the sizes here 1 (the last few), 2, 4 and 8 of them, of numbers of
heads that they divide and do not divide."""
import numpy as np
import pytest
import torch

from oracle import pages_oracle as po
from oracle import serving_oracle as so
from sdpa_testlib import f64, lib
from serving_testlib import DT, HALF_STEP, TINY

pytestmark = pytest.mark.gpu


def rows(g, dtype, b, h, s, d):
    return torch.randn(b, s, h, d, generator=g, device="cuda").to(DT[dtype]).permute(0, 2, 1, 3)


def positions(rng, several, b, s):
    """Positions [axes, b, s] as numpy, and as the call takes them (None: each row's own)."""
    if not several:
        return None, None
    pos = rng.integers(0, 3000, (several, b, s)).astype(np.int32)
    return pos, torch.from_numpy(pos).cuda()


def sections(pairs, n):
    """`pairs` pairs dealt to n axes, unevenly."""
    cut = [pairs * (i + 1) // (n + 1) for i in range(n - 1)]
    return [b - a for a, b in zip([0] + cut, cut + [pairs])]


ROPE = [
    # b, s, h_q, h_k, d, rot, dtype, interleaved, axes
    (1, 4001, 32, 8, 128, 128, "bf16", False, 0), (1, 4001, 32, 8, 128, 128, "bf16", False, 3), (2, 2500, 9, 4, 128, 64, "f16", True, 2),
    (1, 9803, 13, 0, 128, 128, "bf16", True, 4), (1, 2001, 30, 9, 128, 128, "f16", False, 3), (2, 900, 16, 16, 256, 256, "bf16", False, 2),
    (2, 3001, 11, 5, 72, 72, "bf16", False, 0), (2, 3001, 11, 5, 72, 72, "bf16", True, 2), (1, 6001, 14, 3, 128, 120, "f16", False, 3),
    (1, 6001, 14, 3, 128, 40, "f16", True, 0), (1, 1999, 9, 4, 128, 122, "bf16", False, 3), (1, 1999, 9, 4, 128, 58, "bf16", True, 2),
    (3, 1301, 5, 1, 64, 26, "f16", False, 0), (1, 777, 8, 2, 128, 128, "bf16", False, 3),
]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("b,s,h_q,h_k,d,rot,dtype,inter,several", ROPE)
def test_rope_of_prompts(b, s, h_q, h_k, d, rot, dtype, inter, several, backward):
    m, g, rng = lib(), torch.Generator(device="cuda").manual_seed(3), np.random.default_rng(s + rot)
    q, k = rows(g, dtype, b, h_q, s, d), rows(g, dtype, b, h_k, s, d) if h_k else None
    table, _ = m.sdpa_rope_table(rot)
    freqs, _ = so.inv_freq(rot)
    pos_np, pos = positions(rng, several, b, s)
    kw = dict(interleaved=inter, attn_factor=1.5)
    axis = [0] * (rot // 2)
    if several:
        axis = kw["axes"] = m.sdpa_rope_axes(sections(rot // 2, several), order="interleaved" if several == 2 else "blocks")
    else:
        pos_np = np.broadcast_to(np.arange(s, dtype=np.int32), (1, b, s))
    out = [None if x is None else torch.full_like(x, float("nan")) for x in (q, k)]
    call = m.sdpa_rope_bwd if backward else m.sdpa_rope_fwd
    call(q, k, *out, table, pos, **kw)
    at = np.unique(np.concatenate([rng.integers(0, s, 60), [0, 1, s - 2, s - 1]]))
    pick = torch.from_numpy(at).cuda()
    for x, y in zip((q, k), out):
        if x is None:
            continue
        assert torch.equal(y[..., rot:], x[..., rot:]) and torch.isfinite(y).all()
        want, reach = po.rotate_axes(f64(x[:, :, pick]), pos_np[:, :, at], axis, freqs, inter, 1.5, backward)
        # cos and sin: 2^-22 (the angle's 2^-24 of a half turn, the series, the factor); two products, one sum
        tol = HALF_STEP[dtype] * np.abs(want) * 1.01 + 2.0 ** -20 * reach + TINY[dtype]
        assert (np.abs(f64(y[:, :, pick]) - want) <= tol).all()
    there = [None if x is None else x.clone() for x in (q, k)]        # in place
    call(*there, *there, table, pos, **kw)
    assert all(x is None or torch.equal(x, y) for x, y in zip(there, out))


WRITE = [
    # lens_kv, lens_q, s, h, d, page, cache, rows, rot, interleaved, axes
    ((5001, 6200), (5001, 4900), 5001, 8, 128, 64, "e4m3", "bf16", 128, False, 0), ((5001, 6200), (5001, 4900), 5001, 8, 128, 64, "e4m3", "bf16", 128, False, 3),
    ((5001, 6200), None, 5001, 5, 128, 16, "bf16", "bf16", 128, True, 0), ((4999,), None, 4999, 8, 128, 48, "e4m3", "f16", 128, True, 2),
    ((4999,), None, 4999, 7, 128, 64, "f16", "f16", 128, False, 3), ((5300, 17, 5000), (5300, 0, 4000), 5300, 3, 128, 128, "e4m3", "bf16", 128, False, 4),
    ((5300, 5000), None, 5000, 12, 128, 64, "e4m3", "bf16", 128, True, 0), ((5000, 5300), None, 5000, 12, 128, 64, "bf16", "bf16", 128, False, 3),
    ((2600, 2601), None, 2600, 8, 256, 64, "e4m3", "f16", 256, False, 0), ((2600, 2601), None, 2600, 6, 256, 32, "bf16", "bf16", 256, True, 3),
    ((9900, 9000), None, 9900, 12, 64, 64, "e4m3", "bf16", 64, False, 2), ((9900, 9001, 1000), None, 9900, 8, 64, 64, "f16", "f16", 64, True, 0),
    ((9801, 9800), None, 9800, 8, 128, 64, "e4m3", "bf16", 64, False, 0), ((9801, 9800), None, 9800, 5, 128, 64, "bf16", "bf16", 64, True, 3),
    ((5001, 6200), None, 5001, 8, 128, 64, "e4m3", "bf16", 32, True, 0), ((5001, 6200), None, 5001, 4, 128, 64, "e4m3", "f16", 96, False, 2),
    ((9801, 9800), None, 9800, 8, 128, 64, "e4m3", "bf16", 0, False, 0), ((9801, 9800), None, 9800, 12, 128, 64, "bf16", "bf16", 0, False, 0),
    ((5001, 6200), None, 5001, 3, 128, 64, "f16", "f16", 0, False, 0), ((9900, 9000), None, 9900, 2, 64, 64, "e4m3", "f16", 0, False, 0),
    ((5001, 6200), None, 5001, 8, 128, 64, "e4m3", "bf16", 122, False, 0), ((5001, 6200), None, 5001, 8, 128, 64, "e4m3", "bf16", 122, True, 3),
    ((5001, 6200), None, 5001, 5, 128, 64, "bf16", "bf16", 122, False, 2), ((5001, 6200), None, 5001, 12, 128, 64, "f16", "f16", 58, True, 0),
    ((4999,), None, 4999, 8, 128, 64, "e4m3", "f16", 58, False, 3), ((4999,), None, 4999, 8, 128, 64, "e4m3", "f16", 58, True, 0),
    ((2500,), None, 2500, 8, 128, 64, "bf16", "bf16", 122, True, 2), ((2500,), None, 2500, 8, 128, 64, "bf16", "bf16", 122, False, 0),
    ((2500,), None, 2500, 8, 128, 64, "e4m3", "bf16", 122, True, 0), ((1500, 20), (1000, 20), 1000, 4, 256, 16, "e4m3", "f16", 250, False, 2),
    ((300, 20), (33, 20), 33, 4, 64, 16, "e4m3", "f16", 26, True, 0), ((300, 20), (33, 20), 33, 4, 64, 16, "f16", "f16", 26, False, 2),
]


@pytest.mark.parametrize("lens,lens_q,s,h,d,page,kind,row,rot,inter,several", WRITE)
def test_cache_write_of_prompts(lens, lens_q, s, h, d, page, kind, row, rot, inter, several):
    m, g, rng, b = lib(), torch.Generator(device="cuda").manual_seed(5), np.random.default_rng(s + h + rot), len(lens)
    k, v = (rows(g, row, b, h, s, d) for _ in range(2))
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((b, max(need)), -1, np.int32)
    for i, n in enumerate(need):
        table[i, :n] = order[sum(need[:i]): sum(need[:i]) + n]
    size = 1 if kind == "e4m3" else 2
    raw = [torch.full((pages, page, h, d * size), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(2)]
    caches = [x.view(DT[kind]).permute(0, 2, 1, 3) for x in raw]
    scales = [torch.full((pages, h, page), -7.0, device="cuda") for _ in range(2)] if kind == "e4m3" else [None, None]
    kw = {}
    axis, pos_np = [0] * (rot // 2), None
    if rot:
        kw = dict(rope_table=m.sdpa_rope_table(rot)[0], interleaved=inter, attn_factor=1.25)
        pos_np, kw["positions"] = positions(rng, several, b, s)
        if several:
            axis = kw["axes"] = m.sdpa_rope_axes(sections(rot // 2, several), order="interleaved" if several == 2 else "blocks")
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")    # noqa: E731
    m.sdpa_cache_write(k, v, *caches, torch.from_numpy(table).cuda(), dev(lens), seq_lens_q=None if lens_q is None else dev(lens_q), k_scale=scales[0],
                       v_scale=scales[1], **kw)
    where = so.slots(table, page, pages, lens, lens_q, s)
    touched = np.zeros((pages, page), dtype=bool)
    touched[[x[2] for x in where], [x[3] for x in where]] = True
    left = torch.from_numpy(~touched).cuda()
    for x, sc in zip(raw, scales):
        assert (x[left] == 0x5A).all() and (sc is None or (sc.transpose(1, 2)[left] == -7.0).all()), "written elsewhere"
        assert sc is None or (sc.transpose(1, 2)[~left] > 0).all()
    for j in np.unique(np.concatenate([rng.integers(0, len(where), 90), [0, len(where) - 1]])):
        i, r, pg, sl = where[j]
        n = lens_q[i] if lens_q is not None else s
        x = f64(k[i, :, r])[None, :, None]
        reach = np.zeros_like(x)
        if rot:
            at = np.array([[[lens[i] - n + r]]]) if pos_np is None else pos_np[:, i, r][:, None, None]
            x, reach = po.rotate_axes(x, at, axis, so.inv_freq(rot)[0], inter, 1.25)
        for want, rc, cache, sc in ((x[0, :, 0], reach[0, :, 0], caches[0], scales[0]), (f64(v[i, :, r]), np.zeros((h, d)), caches[1], scales[1])):
            got, slack = f64(cache[pg, :, sl].float()), 2.0 ** -20 * rc
            if sc is None:
                assert (np.abs(got - want) <= HALF_STEP[kind] * np.abs(want) * 1.01 + slack + TINY[kind]).all()
                continue
            ref, scale = so.row_scale(want), f64(sc[pg, :, sl])
            # the largest element carries the slack of a rotation; two fp32 divisions
            assert (np.abs(scale - ref) <= 2.0 ** -22 * ref + slack.max(-1) / 448).all()
            y = got * scale[:, None]
            half = np.maximum(HALF_STEP["e4m3"] * np.abs(want), TINY["e4m3"] * scale[:, None])
            assert (np.abs(y - want) <= half * (1 + 2.0 ** -10) + 2 * slack + 2.0 ** -21 * np.abs(want)).all()
