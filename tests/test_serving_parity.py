"""Rotary positions, the paged cache and the attention over it against the fp64 oracle (GPU)."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as so
from sdpa_testlib import check_guard, f64, guarded_empty_like, lib
from serving_testlib import (DT, HALF_STEP, TINY, assert_attend_close, kv_rounding, make_cache, random_tree, randn,
                             run_decode, values_of)

pytestmark = pytest.mark.gpu


def bshd(g, dtype, b, h, s, d, token_major=True):
    x = randn(g, b, s, h, d).to(DT[dtype]).cuda()
    return x.permute(0, 2, 1, 3) if token_major else x.permute(0, 2, 1, 3).contiguous()


# ---- rotary positions ------------------------------------------------------------------------

ROPE = [
    # b, h_q, h_k, s, d, rot, dtype, interleaved, token_major, positions
    (2, 4, 2, 37, 128, 128, "bf16", False, True, "far"),
    (1, 1, 1, 1, 64, 64, "f16", False, True, "far"),
    (2, 3, 0, 5, 64, 32, "bf16", True, True, None),
    (1, 16, 2, 130, 256, 64, "f16", True, False, "shared"),
    (3, 2, 1, 9, 128, 122, "bf16", False, True, "far"),      # rot/2 odd: the element-wise path
    (1, 2, 2, 7, 72, 18, "f16", True, True, "negative"),     # d not a multiple of 16
    (1, 2, 1, 3, 8, 2, "bf16", False, False, None),
    (1, 5, 3, 300, 512, 512, "f16", False, True, "far"),
]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("b,h_q,h_k,s,d,rot,dtype,inter,token_major,where", ROPE)
def test_rope(b, h_q, h_k, s, d, rot, dtype, inter, token_major, where, backward):
    m, g = lib(), torch.Generator().manual_seed(3)
    q = bshd(g, dtype, b, h_q, s, d, token_major)
    k = bshd(g, dtype, b, h_k, s, d, token_major) if h_k else None
    table, att = m.sdpa_rope_table(rot, scaling="yarn", factor=4.0, original_context=4096)
    freqs, att_ref = so.inv_freq(rot, scaling="yarn", factor=4.0, original_context=4096)
    assert abs(att - att_ref) < 1e-6
    pos_np = np.broadcast_to(np.arange(s), (b, s)).copy()
    pos = None
    if where is not None:
        lo, hi = {"far": (0, 2_000_000_000), "negative": (-70000, 0), "shared": (0, 1 << 20)}[where]
        pos_np = np.random.default_rng(5).integers(lo, hi, (1 if where == "shared" else b, s))
        pos = torch.tensor(pos_np, dtype=torch.int32, device="cuda")
        pos_np = np.broadcast_to(pos_np, (b, s))
    qo, qb = guarded_empty_like(q)
    ko, kb = guarded_empty_like(k) if k is not None else (None, None)
    call = m.sdpa_rope_bwd if backward else m.sdpa_rope_fwd
    call(q, k, qo, ko, table, pos, interleaved=inter, attn_factor=att)
    torch.cuda.synchronize()
    for x, y, buf in ((q, qo, qb), (k, ko, kb)):
        if x is None:
            continue
        check_guard(buf, "rope")
        want, reach = so.rotate(f64(x), pos_np, freqs, inter, att, backward)
        # cos and sin: 2^-22 (the angle's 2^-24 of a half turn, sincospi, the factor); two products, one sum
        tol = HALF_STEP[dtype] * np.abs(want) * 1.01 + 2.0 ** -20 * reach + TINY[dtype]
        if rot < d:
            assert torch.equal(y[..., rot:], x[..., rot:])
        assert (np.abs(f64(y) - want) <= tol).all()
    # in place
    q2, k2 = q.clone(), None if k is None else k.clone()
    call(q2, k2, q2, k2, table, pos, interleaved=inter, attn_factor=att)
    assert torch.equal(q2, qo) and (k is None or torch.equal(k2, ko))


def test_rope_backward_is_the_gradient():
    """<dy, R dx> = <R^T dy, x> in fp64 sums over the rounded outputs, and by differences: the map is linear."""
    m, g = lib(), torch.Generator().manual_seed(8)
    x, dy = (bshd(g, "f16", 1, 2, 33, 64) for _ in range(2))
    table, _ = m.sdpa_rope_table(64)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    m.sdpa_rope_fwd(x, None, y, None, table)
    m.sdpa_rope_bwd(dy, None, dx, None, table)
    left, right = (f64(y) * f64(dy)).sum(), (f64(x) * f64(dx)).sum()
    # every product is off by at most 2^-11 + 2^-20 of |y dy| (and |x dx|) each
    tol = 2.0 ** -10 * (np.abs(f64(y) * f64(dy)).sum() + np.abs(f64(x) * f64(dx)).sum())
    assert abs(left - right) <= tol
    e = torch.zeros_like(x)
    e[0, 1, 20, 5] = 0.5                     # a difference along one input, exact in the inputs' type
    x1 = (x.double() + e.double()).half()
    y1 = torch.empty_like(x)
    m.sdpa_rope_fwd(x1, None, y1, None, table)
    slope = ((f64(y1) - f64(y)) * f64(dy)).sum()
    step = f64(x1)[0, 1, 20, 5] - f64(x)[0, 1, 20, 5]
    row = np.abs(f64(dy)[0, 1, 20]) @ (np.abs(f64(y1)[0, 1, 20]) + np.abs(f64(y)[0, 1, 20]))
    assert abs(slope - step * f64(dx)[0, 1, 20, 5]) <= 2.0 ** -10 * row


# ---- cache -----------------------------------------------------------------------------------

WRITE = [
    # lens_kv, lens_q, s, h_kv, d, page, cache, rows, rot, interleaved, slot_major, positions
    ((40, 1, 17), (40, 1, 3), 40, 2, 128, 16, "e4m3", "bf16", 128, False, True, False),
    ((5, 0, 33), None, 1, 8, 128, 32, "e4m3", "f16", 64, True, False, False),
    ((200, 64), (200, 0), 200, 1, 64, 48, "f16", "f16", 0, False, True, False),
    ((70, 71, 2), (9, 12, 12), 12, 3, 256, 64, "e4m3", "bf16", 250, False, True, True),   # 12 new rows, 2 tokens
    ((130,), (130,), 131, 4, 64, 128, "bf16", "bf16", 58, True, True, False),
    ((31, 16), (5, 1), 5, 16, 256, 16, "bf16", "bf16", 128, False, False, True),
]


@pytest.mark.parametrize("lens,lens_q,s,h,d,page,kind,rows,rot,inter,slot_major,own_pos", WRITE)
def test_cache_write(lens, lens_q, s, h, d, page, kind, rows, rot, inter, slot_major, own_pos):
    m, g, b = lib(), torch.Generator().manual_seed(2), len(lens)
    c = make_cache(lens, h, d, page, kind, seed=4, slot_major=slot_major, fill=2.0)
    before = (values_of(c.k), values_of(c.v), None if c.k_scale is None else f64(c.k_scale),
              None if c.v_scale is None else f64(c.v_scale))
    k, v = (bshd(g, rows, b, h, s, d, token_major=i == 0) for i in range(2))
    lq = None if lens_q is None else torch.tensor(lens_q, dtype=torch.int32, device="cuda")
    rope, pos_np = {}, np.zeros((b, s))
    n_of = lambda i: min(max(lens_q[i], 0), s) if lens_q is not None else s
    for i in range(b):
        pos_np[i] = lens[i] - n_of(i) + np.arange(s)
    if rot:
        table, att = m.sdpa_rope_table(rot, scaling="linear", factor=2.0)
        rope = dict(rope_table=table, interleaved=inter, attn_factor=1.25)
        if own_pos:
            pos_np = np.random.default_rng(1).integers(0, 100000, (b, s))
            rope["positions"] = torch.tensor(pos_np, dtype=torch.int32, device="cuda")
    m.sdpa_cache_write(k, v, *c.where(), seq_lens_q=lq, **c.scales(), **rope)
    torch.cuda.synchronize()
    freqs, _ = so.inv_freq(rot, scaling="linear", factor=2.0) if rot else (np.zeros(0), 1)
    want_k, reach = so.rotate(f64(k), pos_np, freqs, inter, 1.25) if rot else (f64(k), np.zeros(k.shape))
    touched = np.zeros((c.k.shape[0], page), dtype=bool)
    for cache, scale, want, rc, old, old_scale in ((c.k, c.k_scale, want_k, reach, before[0], before[2]),
                                                   (c.v, c.v_scale, f64(v), np.zeros(v.shape), before[1], before[3])):
        got = values_of(cache)
        sc = None if scale is None else f64(scale)
        for i, r, pg, sl in so.slots(c.page_table.cpu().numpy(), page, c.k.shape[0], lens, lens_q, s):
            touched[pg, sl] = True
            x, slack = want[i, :, r], 2.0 ** -20 * rc[i, :, r]
            if sc is None:
                assert (np.abs(got[pg, :, sl] - x) <= HALF_STEP[kind] * np.abs(x) * 1.01 + slack + TINY[kind]).all()
                continue
            ref = so.row_scale(x)
            # the largest element carries the slack of a rotation; two fp32 divisions
            assert (np.abs(sc[pg, :, sl] - ref) <= 2.0 ** -22 * ref + slack.max(-1) / 448).all()
            y = got[pg, :, sl] * sc[pg, :, sl, None]
            half = np.maximum(HALF_STEP["e4m3"] * np.abs(x), TINY["e4m3"] * sc[pg, :, sl, None])
            assert (np.abs(y - x) <= half * (1 + 2.0 ** -10) + 2 * slack + 2.0 ** -21 * np.abs(x)).all()
        rest = ~touched
        assert np.array_equal(got.transpose(0, 2, 1, 3)[rest], old.transpose(0, 2, 1, 3)[rest], equal_nan=True)
        if sc is not None:
            assert np.array_equal(sc.transpose(0, 2, 1)[rest], old_scale.transpose(0, 2, 1)[rest], equal_nan=True)


def test_cache_write_extremes():
    """Rows of zeros, of the smallest and largest values, with an infinity, with a NaN."""
    m = lib()
    c = make_cache((8,), 1, 64, 16, "e4m3", fill=0.0)
    x = torch.randn(1, 1, 8, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    x[0, 0, 0] = 0
    x[0, 0, 1] = 2.0 ** -130
    x[0, 0, 2, 5] = 3.0e38
    x[0, 0, 3, 5] = float("inf")
    x[0, 0, 4, 5] = float("nan")
    x[0, 0, 5, 5] = -float("inf")
    x = x.cuda()
    m.sdpa_cache_write(x, x, *c.where(), **c.scales())
    k, v = torch.empty_like(x), torch.empty_like(x)
    m.sdpa_cache_read(*c.where(), k, v, **c.scales())
    for y in (k, v):
        y = f64(y)[0, 0]
        assert (y[0] == 0).all() and (y[1] == 0).all()
        assert np.isnan(y[3:6]).all()
        for r in (2, 6, 7):
            ref = f64(x)[0, 0, r]
            sc = so.row_scale(ref[None])[0]
            assert (np.abs(y[r] - ref) <= np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * sc) * 1.01 + 2.0 ** -8 * np.abs(ref)).all()


READ = [((40, 0, 17, 1), 40, 2, 128, 16, "e4m3", "bf16", True), ((5, 64), 70, 3, 64, 32, "f16", "f16", False),
        ((130, 7), 100, 1, 256, 48, "e4m3", "f16", False), ((1,), 1, 8, 128, 64, "bf16", "bf16", True)]


@pytest.mark.parametrize("lens,s,h,d,page,kind,rows,slot_major", READ)
def test_cache_read(lens, s, h, d, page, kind, rows, slot_major):
    m, b = lib(), len(lens)
    c = make_cache(lens, h, d, page, kind, seed=6, slot_major=slot_major)
    k, kb = guarded_empty_like(torch.empty(b, s, h, d).permute(0, 2, 1, 3), DT[rows])
    v, vb = guarded_empty_like(torch.empty(b, h, s, d), DT[rows])
    m.sdpa_cache_read(*c.where(), k, v, **c.scales())
    torch.cuda.synchronize()
    check_guard(kb, "k")
    check_guard(vb, "v")
    kv, vv, ks, vs, table = c.np()
    for got, val, sc in ((f64(k), kv, ks), (f64(v), vv, vs)):
        for i, n in enumerate(lens):
            want, _ = so.dense(val, sc, table, i, min(n, s))
            x = got[i, :, : min(n, s)]
            half = HALF_STEP[rows] if kind == "e4m3" else 0.0
            assert (np.abs(x - want) <= half * np.abs(want) * 1.01 + TINY[rows] * (half > 0)).all()
            assert (got[i, :, n:] == 0).all()


def test_pages_outside_the_cache_hold_nothing():
    """Entries of the page table outside [0, pages): skipped by a write, zeros in a read, hidden from attention."""
    m, g = lib(), torch.Generator().manual_seed(9)
    c = make_cache((64, 40), 2, 128, 16, "bf16", seed=1, fill=0.0)
    c.page_table[0, 1] = c.k.shape[0]
    c.page_table[0, 3] = -7
    c.page_table[1, 2] = 2 ** 31 - 1
    old = c.k.clone()
    x = bshd(g, "bf16", 2, 2, 16, 128)
    m.sdpa_cache_write(x, x, *c.where())
    torch.cuda.synchronize()
    assert torch.equal(old[c.page_table[0, 0].item()], c.k[c.page_table[0, 0].item()])
    k, v = torch.empty(2, 2, 64, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 2, 64, 128, dtype=torch.bfloat16, device="cuda")
    m.sdpa_cache_read(*c.where(), k, v)
    assert (k[0, :, 16:32] == 0).all() and (k[0, :, 48:] == 0).all() and (k[0, :, 32:48] != 0).any()
    for s in (3, 20):
        q = bshd(g, "bf16", 2, 4, s, 128)
        o, lse = run_decode(c, q)
        kv, vv, _, _, table = c.np()
        ref = so.attend(f64(q), kv, vv, None, None, table, (64, 40), None, 128 ** -0.5)
        assert_attend_close(o, lse, ref, "bf16", "bf16")


# ---- attention -------------------------------------------------------------------------------

ATTEND = [
    # lens_kv, lens_q, s, h_q, h_kv, d, page, cache, q dtype, mask, slot_major
    ((100, 1, 0, 64, 65, 1000), None, 1, 8, 2, 128, 16, "bf16", "bf16", None, True),
    ((100, 1, 0, 63, 129, 777), None, 1, 8, 1, 128, 64, "e4m3", "bf16", None, True),
    ((300, 17), None, 1, 3, 3, 64, 32, "f16", "f16", None, False),
    ((513, 48), None, 1, 16, 1, 64, 16, "e4m3", "f16", None, False),
    ((200, 31), None, 1, 4, 4, 256, 48, "bf16", "bf16", None, True),
    ((129, 16, 15), None, 1, 20, 2, 256, 128, "e4m3", "bf16", None, True),
    ((90, 20, 7), (7, 3, 0), 7, 8, 2, 128, 16, "bf16", "bf16", "causal", True),
    ((64, 5, 12), None, 12, 4, 2, 64, 16, "e4m3", "f16", "causal", True),      # more new rows than keys
    ((100, 40), None, 13, 6, 6, 64, 16, "f16", "f16", "tree", True),
    ((150, 33, 64), (33, 33, 20), 33, 8, 2, 128, 64, "e4m3", "bf16", "tree", False),
    ((70,), None, 64, 16, 2, 128, 32, "bf16", "bf16", "tree", True),
    ((400, 130), None, 40, 4, 1, 256, 16, "e4m3", "f16", "tree", True),
    ((260,), None, 5, 12, 12, 256, 16, "f16", "f16", None, True),
    # more than 16 rows a KV head
    ((300, 0, 128, 1), (20, 20, 3, 20), 20, 2, 1, 128, 48, "e4m3", "bf16", "causal", True),
    ((129, 500), None, 70, 12, 3, 128, 16, "f16", "f16", "tree", True),          # 280 rows: a block and 24 rows
    ((257, 64, 33), (9, 0, 33), 33, 8, 1, 64, 64, "e4m3", "bf16", "tree", False),
    ((1025, 40), None, 17, 1, 1, 64, 80, "bf16", "bf16", None, True),
    ((384,), None, 3, 48, 2, 128, 128, "e4m3", "f16", None, True),
    ((1500, 700, 0, 300), (70, 9, 70, 70), 70, 8, 2, 128, 64, "e4m3", "f16", "tree", True),
    ((1030, 77), None, 12, 12, 1, 64, 16, "e4m3", "f16", "causal", False),
    ((900, 500), None, 10, 8, 1, 128, 16, "e4m3", "f16", "tree", True),
    ((700, 690), None, 257, 1, 1, 128, 32, "bf16", "bf16", "causal", True),
]


@pytest.mark.parametrize("lens,lens_q,s,h_q,h_kv,d,page,kind,dtype,mask,slot_major", ATTEND)
def test_decode(lens, lens_q, s, h_q, h_kv, d, page, kind, dtype, mask, slot_major):
    g, b = torch.Generator().manual_seed(11), len(lens)
    c = make_cache(lens, h_kv, d, page, kind, seed=12, slot_major=slot_major, v_spread=1000.0 if kind == "e4m3" else 1.0)
    q = bshd(g, dtype, b, h_q, s, d)
    tree = np.stack([random_tree(s, 20 + i) for i in range(b)]) if mask == "tree" else None
    o, lse = run_decode(c, q, lens_q=lens_q, causal="bottom_right" if mask == "causal" else False, tree=tree)
    kv, vv, ks, vs, table = c.np()
    ref = so.attend(f64(q), kv, vv, ks, vs, table, lens, lens_q, d ** -0.5, mask == "causal", tree)
    assert_attend_close(o, lse, ref, dtype, "bf16" if kind == "bf16" else "f16", kv_rounding=kv_rounding(kind, s * h_q // h_kv, d, dtype))


@pytest.mark.parametrize("kind,d,h_q,s", [("bf16", 128, 8, 1), ("e4m3", 128, 8, 1), ("f16", 64, 4, 3), ("e4m3", 256, 2, 2),
                                          ("e4m3", 128, 4, 5), ("bf16", 128, 1, 18), ("f16", 64, 2, 140)])
def test_decode_long_ragged(kind, d, h_q, s):
    """Long and short sequences in one batch: blocks of rows split over many CTAs, and CTAs that hold several."""
    g = torch.Generator().manual_seed(13)
    lens = (20011, 3, 0, 4096, 1, 777, 64)
    dtype = "f16" if kind == "f16" else "bf16"
    c = make_cache(lens, 1, d, 64, kind, seed=14)
    q = bshd(g, dtype, len(lens), h_q, s, d)
    o, lse = run_decode(c, q, causal="bottom_right" if s > 1 else False)
    kv, vv, ks, vs, table = c.np()
    ref = so.attend(f64(q), kv, vv, ks, vs, table, lens, None, d ** -0.5, s > 1)
    assert_attend_close(o, lse, ref, dtype, "bf16" if kind == "bf16" else "f16", kv_rounding=kv_rounding(kind, s * h_q, d, dtype))


@pytest.mark.parametrize("kind,s,h_q,dtype", [("bf16", 1, 8, "bf16"), ("bf16", 17, 8, "bf16"), ("e4m3", 17, 8, "bf16"), ("e4m3", 3, 64, "bf16"),
                                              ("e4m3", 5, 64, "bf16"), ("e4m3", 5, 64, "f16"), ("e4m3", 17, 64, "f16")])
def test_decode_many_tiles_a_cta(kind, s, h_q, dtype):
    """Runs of many tiles, so that every ring wraps often; what lies behind each sequence is NaN."""
    g, d, h_kv = torch.Generator().manual_seed(31), 128, 8
    lens = tuple(2500 + 61 * i for i in range(12))
    c = make_cache(lens, h_kv, d, 48, kind, seed=32)
    q = bshd(g, dtype, len(lens), h_q, s, d)
    o, lse = run_decode(c, q, causal="bottom_right")
    again, _ = run_decode(c, q, causal="bottom_right")
    assert torch.equal(o, again)
    kv, vv, ks, vs, table = c.np()
    ref = so.attend(f64(q), kv, vv, ks, vs, table, lens, None, d ** -0.5, True)
    assert_attend_close(o, lse, ref, dtype, "bf16" if kind == "bf16" else "f16", kv_rounding=kv_rounding(kind, s * h_q // h_kv, d, dtype))


@pytest.mark.parametrize("kind,d,s,h_q,h_kv", [("bf16", 128, 1, 2, 1), ("e4m3", 128, 18, 1, 1), ("bf16", 64, 20, 2, 1), ("f16", 128, 150, 1, 1),
                                               ("e4m3", 64, 70, 40, 10), ("e4m3", 256, 2, 4, 4)])
def test_decode_many_short_sequences(kind, d, s, h_q, h_kv):
    """More sequences than CTAs, so that a run holds several whole ones, some empty and some of one token."""
    g = torch.Generator().manual_seed(33)
    b = 400 if h_kv == 1 else 60
    lens = tuple((i * 37) % 150 if i % 7 else (i // 7) % 3 for i in range(b))
    dtype = "f16" if kind == "f16" else "bf16"
    c = make_cache(lens, h_kv, d, 16, kind, seed=34)
    q = bshd(g, dtype, b, h_q, s, d)
    o, lse = run_decode(c, q, causal="bottom_right")
    rows = [i for i in range(b) if b <= 60 or i % 9 == 0]
    kv, vv, ks, vs, table = c.np()
    ref = so.attend(f64(q)[rows], kv, vv, ks, vs, table[rows], [lens[i] for i in rows], None, d ** -0.5, True)
    assert_attend_close(o[rows], lse[rows], ref, dtype, "bf16" if kind == "bf16" else "f16", kv_rounding=kv_rounding(kind, s * h_q // h_kv, d, dtype))


@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
def test_decode_peaked_scores(kind):
    """One key far above the rest, late in a long context; scales that make scores large; a negative scale."""
    dtype = "f16" if kind == "f16" else "bf16"
    g = torch.Generator().manual_seed(15)
    q = bshd(g, dtype, 1, 4, 1, 128)
    c = make_cache((3001,), 1, 128, 16, kind, seed=16)
    kv, vv, ks, vs, table = c.np()
    for scale, rows in ((1.0, 1), (-0.7, 1), (0.0, 1), (1.0, 5), (-0.7, 5), (0.0, 5), (1.0, 40), (-0.7, 40), (0.0, 40)):
        if rows > 1:
            q = bshd(g, dtype, 1, 4, rows, 128)
        o, lse = run_decode(c, q, scale=scale)
        ref = so.attend(f64(q), kv, vv, ks, vs, table, (3001,), None, scale)
        # scores up to 2^6 now: their errors grow with the scale (eight times the default's bound)
        O, L, spread = ref[:3]
        tol = (HALF_STEP["bf16" if kind == "bf16" else "f16"] + 2.0 ** -10 + kv_rounding(kind, 4 * rows, 128, dtype)) * spread + HALF_STEP[dtype] * np.abs(O) * 1.01 + TINY[dtype]
        assert (np.abs(f64(o) - O) <= tol).all()
        assert (np.abs(f64(lse) - L) <= 2.0 ** -10 + 2.0 ** -20 * np.abs(L)).all()


@pytest.mark.parametrize("kind,d,rows,h_kv", [("bf16", 128, 1, 2), ("e4m3", 128, 2, 3), ("f16", 64, 13, 12), ("e4m3", 64, 1, 1), ("bf16", 256, 3, 1),
                                              ("e4m3", 256, 2, 2)])
@pytest.mark.parametrize("lens", [(0, 1, 64, 65), (1000,), (17,), (129, 1279, 700), (40, 0, 512) + (60,) * 70])
def test_decode_short_sequences(kind, d, rows, h_kv, lens):
    """One CTA to eight for a sequence, some of them without a tile; a table that could hold more."""
    dtype = "f16" if kind == "f16" else "bf16"
    g = torch.Generator().manual_seed(31)
    q = bshd(g, dtype, len(lens), 2 * h_kv, rows, d)
    c = make_cache(lens, h_kv, d, 64, kind, seed=32, v_spread=1000.0 if kind == "e4m3" else 1.0)
    kv, vv, ks, vs, table = c.np()
    o, lse = run_decode(c, q, causal="bottom_right")
    ref = so.attend(f64(q), kv, vv, ks, vs, table, lens, None, d ** -0.5, True)
    assert_attend_close(o, lse, ref, dtype, "bf16" if kind == "bf16" else "f16")
    again, lse2 = run_decode(c, q, causal="bottom_right")
    assert torch.equal(o, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("rows", [1, 12, 40])
def test_decode_few_keys_lse(kind, rows):
    """With a handful of keys the LSE is the scores: products of the stored elements, exact but for fp32 sums.

    Each of the d / 16 steps of a tensor core's sum is off by at most 2^-21 of the absolute sum (its terms are
    cut to 2^-22 of the largest, and it is rounded), d = 128: 2^-18 sum |q k| |scale| in all; the factor on the
    scores, the key's scale, ex2 and log2 add 2^-20 (1 + |LSE|)."""
    dtype = "f16" if kind == "f16" else "bf16"
    g = torch.Generator().manual_seed(rows)
    q = bshd(g, dtype, 3, 4, rows, 128)
    c = make_cache((1, 2, 5), 1, 128, 16, kind, seed=29)
    kv, vv, ks, vs, table = c.np()
    lens_q = [min(n, rows) for n in (1, 2, 5)]
    _, lse = run_decode(c, q, lens_q=lens_q)
    L, _, reach = so.attend(f64(q), kv, vv, ks, vs, table, (1, 2, 5), lens_q, 128 ** -0.5)[1:]
    for b, n in enumerate(lens_q):
        err = np.abs(f64(lse)[b, :, :n] - L[b, :, :n])
        assert (err <= 2.0 ** -18 * reach[b, :, :n] + 2.0 ** -20 * (1 + np.abs(L[b, :, :n]))).all(), err.max()


@pytest.mark.parametrize("s,h_q", [(5, 2), (20, 8)])
@pytest.mark.parametrize("spoil", [float("nan"), float("inf")])
def test_hidden_tokens_may_have_any_scale(s, h_q, spoil):
    """A drafted token written as NaN or infinity (its scale is one then) reaches exactly the rows that see it."""
    g = torch.Generator().manual_seed(23)
    n, bad = 50, s // 2
    c = make_cache((n,), 1, 128, 16, "e4m3", seed=24)
    q = bshd(g, "bf16", 1, h_q, s, 128)
    tree = random_tree(s, 4)[None]
    tree[0, :, bad] = False
    tree[0, bad, bad] = True
    clean, clean_lse = run_decode(c, q, tree=tree)
    pos = n - s + bad
    pg, sl = c.page_table[0, pos // 16].item(), pos % 16
    seen = torch.zeros(s, dtype=torch.bool)
    seen[bad] = True
    for scales in ((c.v_scale,), (c.k_scale,), (c.k_scale, c.v_scale)):
        kept = [t[pg, 0, sl].clone() for t in scales]
        for t in scales:
            t[pg, 0, sl] = spoil
        o, lse = run_decode(c, q, tree=tree)
        assert torch.equal(o[0, :, ~seen], clean[0, :, ~seen]) and torch.equal(lse[0, :, ~seen], clean_lse[0, :, ~seen])
        if spoil != spoil or scales[-1] is c.v_scale:      # (a score of -inf is a weight of zero)
            assert not torch.isfinite(o[0, :, seen]).any()
        for t, x in zip(scales, kept):
            t[pg, 0, sl] = x


@pytest.mark.parametrize("rows", [1, 40])
def test_decode_zero_scales(rows):
    """Rows of zeros whose scale is zero count in the sums and add nothing."""
    g = torch.Generator().manual_seed(25)
    c = make_cache((300, 40), 2, 128, 16, "e4m3", seed=26)
    q = bshd(g, "bf16", 2, 4, rows, 128)
    for t, sc in ((c.k, c.k_scale), (c.v, c.v_scale)):
        zero = torch.rand(sc.shape, generator=g).cuda() < 0.6
        sc[zero] = 0.0
        t.view(torch.uint8)[zero] = 0
    kv, vv, ks, vs, table = c.np()
    o, lse = run_decode(c, q)
    ref = so.attend(f64(q), kv, vv, ks, vs, table, (300, 40), None, 128 ** -0.5)
    assert_attend_close(o, lse, ref, "bf16", "f16", kv_rounding=kv_rounding("e4m3", rows * 2, 128, "bf16"))


@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("s,h_q", [(5, 2), (20, 8)])
def test_hidden_tokens_may_hold_anything(kind, s, h_q):
    """Infinities and NaNs in drafted tokens reach exactly the rows that see them."""
    m, g = lib(), torch.Generator().manual_seed(17)
    dtype = "f16" if kind == "f16" else "bf16"
    n, bad = 50, s // 2                    # drafted token `bad` is spoilt
    c = make_cache((n,), 1, 128, 16, kind, seed=18)
    q = bshd(g, dtype, 1, h_q, s, 128)
    tree = random_tree(s, 3)[None]
    tree[0, :, bad] = False
    tree[0, bad, bad] = True
    tree[0, s - 1, bad] = True
    clean, clean_lse = run_decode(c, q, tree=tree)
    pos = n - s + bad
    pg, sl = c.page_table[0, pos // 16].item(), pos % 16
    spoil = {"f16": float("inf"), "bf16": float("-inf"), "e4m3": float("nan")}[kind]
    c.v[pg, 0, sl, 7] = spoil
    c.k[pg, 0, sl, 9] = float("nan")
    o, lse = run_decode(c, q, tree=tree)
    hit = tree[0, :, bad]
    assert torch.isnan(o[0, :, hit]).all()
    assert torch.equal(o[0, :, ~hit], clean[0, :, ~hit]) and torch.equal(lse[0, :, ~hit], clean_lse[0, :, ~hit])
    # a spoilt value alone: only its column, in the rows that see it
    c.k[pg, 0, sl, 9] = 0.5
    o, lse = run_decode(c, q, tree=tree)
    assert torch.isfinite(lse).all()
    assert not torch.isfinite(o[0, :, hit][..., 7]).any()
    if kind != "e4m3":
        assert (o[0, :, hit][..., 7] == spoil).all()
    keep = [i for i in range(128) if i != 7]
    assert torch.isfinite(o[..., keep]).all() and torch.equal(o[0, :, ~hit], clean[0, :, ~hit])


def test_infinite_value_in_the_prefix_reaches_every_row():
    """A non-finite value before the drafted tokens, in their first 16-key slice, is seen by all."""
    g = torch.Generator().manual_seed(19)
    c = make_cache((40,), 1, 64, 16, "bf16", seed=20)
    q = bshd(g, "bf16", 1, 2, 3, 64)
    c.v[c.page_table[0, 2].item(), 0, 2, 3] = float("inf")      # position 34; drafts are 37..39
    o, _ = run_decode(c, q, tree=random_tree(3, 1)[None])
    assert (o[..., 3] == float("inf")).all() and torch.isfinite(o[..., 4:]).all()


# ---- together, as they are used ------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
def test_prompt_then_drafts(kind):
    """A ragged prompt is rotated and written, read back for the dense attention call over it, then three drafted
    tokens (a tree with two branches) are written and attend to the cache; against the oracle over the
    cache's own values."""
    m, g = lib(), torch.Generator().manual_seed(21)
    b, h_q, h_kv, d, page, s = 2, 8, 2, 128, 16, 70
    prompt = (70, 33)
    c = make_cache((73, 36), h_kv, d, page, kind, seed=22)
    table, att = m.sdpa_rope_table(d, scaling="yarn", factor=2.0, original_context=64)
    freqs, _ = so.inv_freq(d, scaling="yarn", factor=2.0, original_context=64)
    q, k, v = bshd(g, "bf16", b, h_q, s, d), bshd(g, "bf16", b, h_kv, s, d), bshd(g, "bf16", b, h_kv, s, d)
    lens = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    c.lens = lens
    m.sdpa_cache_write(k, v, *c.where(), seq_lens_q=lens, **c.scales(), rope_table=table, attn_factor=att)
    qr = torch.empty_like(q)
    m.sdpa_rope_fwd(q, None, qr, None, table, attn_factor=att)
    kd, vd = torch.empty(b, h_kv, s, d, dtype=torch.bfloat16, device="cuda"), torch.empty(b, h_kv, s, d, dtype=torch.bfloat16, device="cuda")
    m.sdpa_cache_read(*c.where(), kd, vd, **c.scales())
    o = torch.empty_like(q)
    m.sdpa_fwd(qr, kd, vd, o, causal="bottom_right", seq_lens_q=lens, seq_lens_kv=lens)
    want_k, _ = so.rotate(f64(k), np.broadcast_to(np.arange(s), (b, s)), freqs, False, att)
    for i, n in enumerate(prompt):
        err = np.linalg.norm(f64(kd)[i, :, :n] - want_k[i, :, :n]) / np.linalg.norm(want_k[i, :, :n])
        assert err <= (2.0 ** -4 if kind == "e4m3" else 2.0 ** -7)
        x = np.einsum("hgqd,hkd->hgqk", f64(qr)[i, :, :n].reshape(h_kv, h_q // h_kv, n, d), f64(kd)[i, :, :n]) * d ** -0.5
        x = np.where(np.arange(n)[None, :] <= np.arange(n)[:, None], x, -np.inf)
        p = np.exp(x - x.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        ref = np.einsum("hgqk,hkd->hgqd", p, f64(vd)[i, :, :n]).reshape(h_q, n, d)
        assert np.abs(f64(o)[i, :, :n] - ref).max() <= 2e-2
    # three drafts: token 1 follows 0; token 2 is another branch after the prompt
    see = np.array([[1, 0, 0], [1, 1, 0], [0, 0, 1]], dtype=bool)
    depth = np.array([0, 1, 0])
    q3, k3, v3 = bshd(g, "bf16", b, h_q, 3, d), bshd(g, "bf16", b, h_kv, 3, d), bshd(g, "bf16", b, h_kv, 3, d)
    pos = torch.tensor(np.array(prompt)[:, None] + depth, dtype=torch.int32, device="cuda")
    c.lens = lens + 3
    m.sdpa_cache_write(k3, v3, *c.where(), **c.scales(), rope_table=table, positions=pos, attn_factor=att)
    m.sdpa_rope_fwd(q3, None, q3, None, table, pos, attn_factor=att)
    o3, lse3 = run_decode(c, q3, tree=np.stack([see, see]))
    kv, vv, ks, vs, tb = c.np()
    ref = so.attend(f64(q3), kv, vv, ks, vs, tb, (73, 36), None, d ** -0.5, False, np.stack([see, see]))
    assert_attend_close(o3, lse3, ref, "bf16", "f16" if kind == "e4m3" else "bf16")


def test_streams_and_graphs():
    """On a side stream, and captured: a replay reads the lengths, pages and rows that are there then."""
    m, g = lib(), torch.Generator().manual_seed(23)
    c = make_cache((300, 120), 2, 128, 16, "e4m3", seed=24, wide=32)
    q = bshd(g, "bf16", 2, 8, 1, 128)
    k, v = (bshd(g, "bf16", 2, 2, 1, 128) for _ in range(2))
    table, _ = m.sdpa_rope_table(128)
    o, lse = torch.empty_like(q), torch.empty(2, 8, 1, device="cuda")
    ws = torch.empty(m.sdpa_decode_workspace_size(q, *c.where(), **c.scales()), dtype=torch.uint8, device="cuda")
    qr = torch.empty_like(q)

    def step():
        m.sdpa_cache_write(k, v, *c.where(), **c.scales(), rope_table=table)
        m.sdpa_rope_fwd(q, None, qr, None, table, pos)
        m.sdpa_decode(qr, *c.where(), o, lse, workspace=ws, **c.scales())

    pos = (c.lens - 1).view(2, 1).contiguous()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    kv, vv, ks, vs, tb = c.np()
    assert_attend_close(o, lse, so.attend(f64(qr), kv, vv, ks, vs, tb, (300, 120), None, 128 ** -0.5), "bf16", "f16")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    # other lengths and rows for the replay
    c.lens.copy_(torch.tensor([77, 9], dtype=torch.int32))
    pos.copy_((c.lens - 1).view(2, 1))
    q.copy_(bshd(g, "bf16", 2, 8, 1, 128))
    k.copy_(bshd(g, "bf16", 2, 2, 1, 128))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    kv, vv, ks, vs, tb = c.np()
    assert_attend_close(o, lse, so.attend(f64(qr), kv, vv, ks, vs, tb, (77, 9), None, 128 ** -0.5), "bf16", "f16")


def test_results_do_not_change_from_call_to_call():
    g = torch.Generator().manual_seed(25)
    c = make_cache((5000, 3, 700), 2, 128, 64, "e4m3", seed=26)
    q = bshd(g, "bf16", 3, 16, 4, 128)
    first = run_decode(c, q, causal="bottom_right")
    for _ in range(3):
        again = run_decode(c, q, causal="bottom_right")
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("kind,h_q,s,columns", [("bf16", 8, 1, 16), ("e4m3", 8, 1, 400), ("bf16", 8, 12, 60), ("e4m3", 8, 40, 60)])
def test_calls_at_once_and_captured_lengths(kind, h_q, s, columns):
    """Two streams at once give what they give one after the other; one captured call serves every length."""
    m, g = lib(), torch.Generator().manual_seed(41)
    page = 16
    lens = (columns * page, 37)
    c = make_cache(lens, 2, 128, page, kind, seed=42, wide=columns)
    qs = [bshd(g, "bf16", 2, h_q, s, 128) for _ in range(2)]
    alone = [run_decode(c, q, causal="bottom_right") for q in qs]
    n = m.sdpa_decode_workspace_size(qs[0], *c.where(), **c.scales())
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in qs]
    outs = [(torch.empty_like(q), torch.empty(2, h_q, s, device="cuda")) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(8):
        for st, q, w, (o, lse) in zip(streams, qs, ws, outs):
            with torch.cuda.stream(st):
                m.sdpa_decode(q, *c.where(), o, lse, workspace=w, causal="bottom_right", **c.scales())
    torch.cuda.synchronize()
    for (o, lse), (o1, lse1) in zip(outs, alone):
        assert torch.equal(o, o1) and torch.equal(lse, lse1)
    graph, (o, lse) = torch.cuda.CUDAGraph(), outs[0]
    with torch.cuda.graph(graph):
        m.sdpa_decode(qs[0], *c.where(), o, lse, workspace=ws[0], causal="bottom_right", **c.scales())
    for now in ((1, 1), (0, 20), (columns * page // 2 + 3, 37), (columns * page, 0)):
        c.lens.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = o.clone(), lse.clone()
        want = run_decode(c, qs[0], causal="bottom_right")
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        if now[1] == 0:
            assert not got[0][1].any() and torch.isneginf(got[1][1]).all()
