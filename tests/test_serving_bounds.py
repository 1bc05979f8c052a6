"""Serving calls with lengths outside their ranges, and what they write beside their outputs and workspace (GPU)."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as so
from sdpa_testlib import check_guard, f64, guarded_empty_like, lib
from serving_testlib import (DT, HALF_STEP, TINY, assert_attend_close, kv_rounding, make_cache, random_tree, randn, run_decode,
                             values_of)

pytestmark = pytest.mark.gpu

PAGE, COLUMNS = 16, 6                 # room for 96 tokens
FILLED = (96, 30, 75, 50, 96)
LENS_KV = (101, -3, 75, 50, 2 ** 31 - 1)        # taken as 96, 0, 75, 50, 96


def bshd(seed, dtype, b, h, s, d):
    return randn(torch.Generator().manual_seed(seed), b, s, h, d).to(DT[dtype]).cuda().permute(0, 2, 1, 3)


def cache_of(h_kv, d, kind, seed, **kw):
    c = make_cache(FILLED, h_kv, d, PAGE, kind, seed=seed, wide=COLUMNS, **kw)
    c.lens = torch.tensor(LENS_KV, dtype=torch.int32, device="cuda")
    return c


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
def test_write_clamps_lengths(kind):
    s, h, d = 12, 2, 128
    lens_q = (16, 3, -1, 2 ** 31 - 1, -2 ** 31)         # taken as 12, 3, 0, 12, 0
    c = cache_of(h, d, kind, 70, fill=2.0)
    old_k, old_v = values_of(c.k), values_of(c.v)
    k, v = bshd(71, "bf16", 5, h, s, d), bshd(72, "bf16", 5, h, s, d)
    lib().sdpa_cache_write(k, v, *c.where(), **c.scales(),
                           seq_lens_q=torch.tensor(lens_q, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    written = so.slots(c.page_table.cpu().numpy(), PAGE, c.k.shape[0], LENS_KV, lens_q, s)
    assert len(written) == 12 + 0 + 0 + 12 + 0          # (sequence 1 has no tokens: its rows lie before position 0)
    touched = np.zeros((c.k.shape[0], PAGE), dtype=bool)
    for cache, scale, x, old in ((c.k, c.k_scale, k, old_k), (c.v, c.v_scale, v, old_v)):
        got = values_of(cache)
        for i, r, pg, sl in written:
            touched[pg, sl] = True
            want = f64(x)[i, :, r]
            if scale is None:
                assert np.array_equal(got[pg, :, sl], want)
            else:
                sc = f64(scale)[pg, :, sl][:, None]
                half = np.maximum(HALF_STEP["e4m3"] * np.abs(want), TINY["e4m3"] * sc)
                assert (np.abs(got[pg, :, sl] * sc - want) <= half * (1 + 2.0 ** -10) + 2.0 ** -21 * np.abs(want)).all()
        assert np.array_equal(got.transpose(0, 2, 1, 3)[~touched], old.transpose(0, 2, 1, 3)[~touched], equal_nan=True)


@pytest.mark.parametrize("kind", ["e4m3", "f16"])
def test_read_clamps_lengths(kind):
    h, d, s = 2, 64, 110                  # more rows than the table has room for
    c = cache_of(h, d, kind, 73)
    k, kb = guarded_empty_like(torch.empty(5, h, s, d), torch.float16)
    v, vb = guarded_empty_like(torch.empty(5, h, s, d), torch.float16)
    lib().sdpa_cache_read(*c.where(), k, v, **c.scales())
    torch.cuda.synchronize()
    check_guard(kb, "k")
    check_guard(vb, "v")
    kv, vv, ks, vs, table = c.np()
    for got, val, sc in ((f64(k), kv, ks), (f64(v), vv, vs)):
        for i, n in enumerate(LENS_KV):
            n = min(max(n, 0), PAGE * COLUMNS)
            want, _ = so.dense(val, sc, table, i, n)
            half = HALF_STEP["f16"] if kind == "e4m3" else 0.0
            assert (np.abs(got[i, :, :n] - want) <= half * np.abs(want) * 1.01 + TINY["f16"] * (half > 0)).all()
            assert (got[i, :, n:] == 0).all()


# One row or three (a cluster a sequence), 12 rows, 40 and 280 rows a KV head.
@pytest.mark.parametrize("kind,d", [("bf16", 128), ("e4m3", 128), ("e4m3", 64), ("f16", 256)])
@pytest.mark.parametrize("s,h_q", [(3, 2), (6, 4), (20, 4), (70, 8)])
@pytest.mark.parametrize("mask", ["tree", "causal", None])
def test_decode_clamps_lengths(mask, s, h_q, kind, d):
    lens_q = (s + 4, s, -1, 2 ** 31 - 1, s - 1)
    dtype = "f16" if kind == "f16" else "bf16"
    c = cache_of(2, d, kind, 74)
    q = bshd(75, dtype, 5, h_q, s, d)
    tree = np.stack([random_tree(s, 80 + i) for i in range(5)]) if mask == "tree" else None
    o, lse = run_decode(c, q, lens_q=lens_q, causal="bottom_right" if mask == "causal" else False, tree=tree)
    kv, vv, ks, vs, table = c.np()
    ref = so.attend(f64(q), kv, vv, ks, vs, table, LENS_KV, lens_q, d ** -0.5, mask == "causal", tree)
    assert_attend_close(o, lse, ref, dtype, "bf16" if kind == "bf16" else "f16", kv_rounding=kv_rounding(kind, s * h_q // 2, d, dtype))


def test_decode_clamps_lengths_of_runs():
    """The same lengths where a table of many columns has runs of tiles walked by teams of CTAs."""
    c = make_cache((20000, 30, 75, 50, 96), 2, 128, PAGE, "e4m3", seed=76, wide=1250)
    lens = (20007, -3, 75, 50, 96)
    c.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = bshd(77, "bf16", 5, 8, 1, 128)
    o, lse = run_decode(c, q, lens_q=(2, 1, 0, -1, 1))
    kv, vv, ks, vs, table = c.np()
    ref = so.attend(f64(q), kv, vv, ks, vs, table, lens, (2, 1, 0, -1, 1), 128 ** -0.5)
    assert_attend_close(o, lse, ref, "bf16", "f16")


PLANS = [
    # lens, columns of the table, s, h_q, h_kv, d, cache
    ((1000, 30), 64, 1, 8, 2, 128, "bf16"),               # a cluster a sequence: no parts
    ((20000, 300), 1250, 1, 8, 2, 128, "e4m3"),           # teams, blocks of 8 rows
    ((20000, 300), 1250, 4, 4, 1, 128, "bf16"),           # blocks of 16
    ((9000, 300), 600, 3, 4, 1, 256, "e4m3"),
    ((900, 40), 57, 128, 64, 64, 256, "f16"),             # more blocks of rows than CTAs at once: one team
    ((3000, 300), 188, 12, 8, 2, 128, "bf16"),            # tcgen05 tiles: 48 rows
    ((3000, 300), 188, 12, 8, 2, 64, "e4m3"),
    ((3000, 300), 188, 70, 16, 2, 128, "e4m3"),           # 560 rows: two blocks and 48 rows
    ((700, 40), 44, 128, 320, 40, 128, "bf16"),           # 160 blocks: one team
]


@pytest.mark.parametrize("lens,columns,s,h_q,h_kv,d,kind", PLANS)
def test_workspace_is_as_large_as_said(lens, columns, s, h_q, h_kv, d, kind):
    """Nothing is written around the workspace's bytes, whatever split of the work the sizes give."""
    m, dtype = lib(), "f16" if kind == "f16" else "bf16"
    c = make_cache(lens, h_kv, d, PAGE, kind, seed=78, wide=columns)
    q = bshd(79, dtype, len(lens), h_q, s, d)
    n = m.sdpa_decode_workspace_size(q, *c.where(), **c.scales())
    assert n % 256 == 0
    buf = torch.full((n + 2 * 65536,), 0x5A, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    m.sdpa_decode(q, *c.where(), o, lse, workspace=buf[65536:65536 + n], **c.scales(), causal="bottom_right")
    torch.cuda.synchronize()
    assert (buf[:65536] == 0x5A).all() and (buf[65536 + n:] == 0x5A).all()
    o2, lse2 = run_decode(c, q, causal="bottom_right")
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.isfinite(o).all()


@pytest.mark.parametrize("kind,s,h_q", [("e4m3", 1, 8), ("bf16", 1, 8), ("e4m3", 20, 8)])
def test_a_view_of_the_page_table(kind, s, h_q):
    """The first columns of a wide table, with the workspace of all of them."""
    m, lens = lib(), (300, 17, 0)
    c = make_cache(lens, 2, 128, PAGE, kind, seed=90, wide=2000)
    q = bshd(91, "bf16", 3, h_q, s, 128)
    ws = torch.empty(m.sdpa_decode_workspace_size(q, *c.where(), **c.scales()), dtype=torch.uint8, device="cuda")
    c.page_table = c.page_table[:, :19]
    assert c.page_table.stride(0) == 2000
    o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    m.sdpa_decode(q, *c.where(), o, lse, workspace=ws, **c.scales(), causal="bottom_right")
    kv, vv, ks, vs, table = c.np()
    ref = so.attend(f64(q), kv, vv, ks, vs, table, lens, None, 128 ** -0.5, True)
    assert_attend_close(o, lse, ref, "bf16", "bf16" if kind == "bf16" else "f16", kv_rounding=kv_rounding(kind, s * h_q // 2, 128, "bf16"))
