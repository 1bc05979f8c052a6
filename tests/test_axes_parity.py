"""Rotary positions with several axes against the fp64 oracle: forward, backward, on the way into a cache (GPU)."""
import numpy as np
import pytest
import torch

from oracle import pages_oracle as po
from oracle import serving_oracle as so
from sdpa_testlib import check_guard, f64, guarded_empty_like, lib
from serving_testlib import DT, HALF_STEP, TINY, make_cache, randn, values_of

pytestmark = pytest.mark.gpu


def bshd(g, dtype, b, h, s, d, token_major=True):
    x = randn(g, b, s, h, d).to(DT[dtype]).cuda()
    return x.permute(0, 2, 1, 3) if token_major else x.permute(0, 2, 1, 3).contiguous()


AXES = [
    # b, h_q, h_k, s, d, dtype, interleaved, token_major, sections, order, positions
    (2, 4, 2, 37, 128, "bf16", False, True, (16, 24, 24), "blocks", "far"),
    (1, 1, 1, 1, 64, "f16", False, True, (16, 16), "blocks", "far"),
    (2, 3, 0, 5, 64, "bf16", True, True, (5, 1, 10), "interleaved", "shared"),       # half of each head, axes mixed in a thread
    (1, 16, 2, 130, 256, "f16", True, False, (7, 9, 5, 11), "interleaved", "near"),
    (3, 2, 1, 9, 128, "bf16", False, True, (31, 30), "blocks", "far"),               # rot/2 odd: element by element
    (1, 2, 2, 7, 72, "f16", True, True, (4, 3, 2), "interleaved", "negative"),       # d not a multiple of 16
    (1, 2, 1, 3, 8, "bf16", False, False, (1,), "blocks", "near"),
    (1, 5, 3, 300, 512, "f16", False, True, (200, 50, 5, 1), "blocks", "far"),
    (2, 12, 12, 33, 64, "f16", True, True, (16, 16), "blocks", "one row"),
    (2, 5, 2, 19, 72, "bf16", False, True, (12, 24), "blocks", "far"),               # multiples of 8, not of 16
    (1, 9, 9, 40, 72, "f16", True, True, (18, 18), "interleaved", "near"),
    (1, 3, 1, 11, 128, "bf16", True, False, (5, 6, 9), "interleaved", "far"),        # rot 40
    (2, 2, 0, 6, 64, "f16", False, True, (3, 1), "blocks", "negative"),              # rot 8
]


def where(kind, n, b, s, seed):
    rng = np.random.default_rng(seed)
    lo, hi = {"far": (0, 2_000_000_000), "near": (0, 40), "negative": (-70000, 0), "shared": (0, 1 << 20), "one row": (0, 5000)}[kind]
    pos = rng.integers(lo, hi, (n, 1 if kind in ("shared", "one row") else b, s)).astype(np.int32)
    dev = torch.tensor(pos, device="cuda")
    if kind == "one row":
        dev = dev[:, 0]
    return np.broadcast_to(pos, (n, b, s)), dev


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("b,h_q,h_k,s,d,dtype,inter,token_major,sections,order,kind", AXES)
def test_axes(b, h_q, h_k, s, d, dtype, inter, token_major, sections, order, kind, backward):
    m, g = lib(), torch.Generator().manual_seed(3)
    q = bshd(g, dtype, b, h_q, s, d, token_major)
    k = bshd(g, dtype, b, h_k, s, d, token_major) if h_k else None
    rot, axes = 2 * sum(sections), m.sdpa_rope_axes(sections, order=order)
    scaling = dict(scaling="yarn", factor=4.0, original_context=4096) if rot > 2 else {}
    table, att = m.sdpa_rope_table(rot, **scaling)
    freqs, att_ref = so.inv_freq(rot, **scaling)
    assert abs(att - att_ref) < 1e-6
    pos_np, pos = where(kind, len(sections), b, s, 5)
    qo, qb = guarded_empty_like(q)
    ko, kb = guarded_empty_like(k) if k is not None else (None, None)
    call = m.sdpa_rope_bwd if backward else m.sdpa_rope_fwd
    call(q, k, qo, ko, table, pos, interleaved=inter, attn_factor=att, axes=axes)
    torch.cuda.synchronize()
    for x, y, buf in ((q, qo, qb), (k, ko, kb)):
        if x is None:
            continue
        check_guard(buf, "rope")
        want, reach = po.rotate_axes(f64(x), pos_np, axes, freqs, inter, att, backward)
        # cos and sin: 2^-22 (the angle's 2^-24 of a half turn, the series, the factor); two products, one sum
        tol = HALF_STEP[dtype] * np.abs(want) * 1.01 + 2.0 ** -20 * reach + TINY[dtype]
        if rot < d:
            assert torch.equal(y[..., rot:], x[..., rot:])
        assert (np.abs(f64(y) - want) <= tol).all()
    q2, k2 = q.clone(), None if k is None else k.clone()        # in place
    call(q2, k2, q2, k2, table, pos, interleaved=inter, attn_factor=att, axes=axes)
    assert torch.equal(q2, qo) and (k is None or torch.equal(k2, ko))


@pytest.mark.parametrize("rot,inter", [(64, False), (64, True), (26, False), (26, True), (40, False), (40, True)])
def test_one_position_on_all_axes_is_the_plain_rotation(rot, inter):
    m, g = lib(), torch.Generator().manual_seed(4)
    q = bshd(g, "bf16", 2, 3, 21, 64)
    table, _ = m.sdpa_rope_table(rot)
    pos = torch.randint(0, 1 << 30, (2, 21), generator=g, dtype=torch.int32).cuda()
    want, got = torch.empty_like(q), torch.empty_like(q)
    m.sdpa_rope_fwd(q, None, want, None, table, pos, interleaved=inter)
    m.sdpa_rope_fwd(q, None, got, None, table, pos.expand(3, 2, 21), interleaved=inter, axes=m.sdpa_rope_axes((rot // 2 - 6, 5, 1), order="interleaved"))
    assert torch.equal(got, want)
    m.sdpa_rope_fwd(q, None, got, None, table, pos[None], interleaved=inter, axes=bytes(rot // 2))
    assert torch.equal(got, want)


def test_axes_with_frequencies_of_their_own():
    """Rows and columns of an image with the same frequencies each: two tables, one behind the other; each axis's pairs turn as a
    head of half the size by that axis alone."""
    m, g = lib(), torch.Generator().manual_seed(6)
    x = bshd(g, "f16", 1, 2, 30, 64)
    half, _ = m.sdpa_rope_table(32)
    table, axes = torch.cat((half, half)), m.sdpa_rope_axes((16, 16))
    i = torch.arange(30, dtype=torch.int32, device="cuda")
    pos = torch.stack((i // 6, i % 6))
    y = torch.empty_like(x)
    m.sdpa_rope_fwd(x, None, y, None, table, pos, interleaved=True, axes=axes)
    for a in range(2):
        part = x[..., 32 * a: 32 * a + 32].contiguous()
        want = torch.empty_like(part)
        m.sdpa_rope_fwd(part, None, want, None, half, pos[a].contiguous(), interleaved=True)
        assert torch.equal(y[..., 32 * a: 32 * a + 32], want)


def test_axes_backward_is_the_gradient():
    """<dy, R x> = <R^T dy, x>, and a difference along one input: the map is linear."""
    m, g = lib(), torch.Generator().manual_seed(8)
    x, dy = (bshd(g, "f16", 1, 2, 33, 64) for _ in range(2))
    table, _ = m.sdpa_rope_table(64)
    axes = m.sdpa_rope_axes((8, 12, 12), order="interleaved")
    _, pos = where("near", 3, 1, 33, 9)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    m.sdpa_rope_fwd(x, None, y, None, table, pos, axes=axes)
    m.sdpa_rope_bwd(dy, None, dx, None, table, pos, axes=axes)
    left, right = (f64(y) * f64(dy)).sum(), (f64(x) * f64(dx)).sum()
    # every product is off by at most 2^-11 + 2^-20 of |y dy| (and |x dx|) each
    assert abs(left - right) <= 2.0 ** -10 * (np.abs(f64(y) * f64(dy)).sum() + np.abs(f64(x) * f64(dx)).sum())
    for e in (5, 37):
        x1 = x.clone()
        x1[0, 1, 20, e] += 0.5
        y1 = torch.empty_like(x)
        m.sdpa_rope_fwd(x1, None, y1, None, table, pos, axes=axes)
        slope = ((f64(y1) - f64(y)) * f64(dy)).sum()
        step = f64(x1)[0, 1, 20, e] - f64(x)[0, 1, 20, e]
        row = np.abs(f64(dy)[0, 1, 20]) @ (np.abs(f64(y1)[0, 1, 20]) + np.abs(f64(y)[0, 1, 20]))
        assert abs(slope - step * f64(dx)[0, 1, 20, e]) <= 2.0 ** -10 * row


WRITE = [
    # lens_kv, lens_q, s, h_kv, d, page, cache, rows, sections, order, interleaved, slot_major
    ((40, 1, 17), (40, 1, 3), 40, 2, 128, 16, "e4m3", "bf16", (16, 24, 24), "blocks", False, True),
    ((5, 0, 33), None, 1, 8, 128, 32, "e4m3", "f16", (11, 21), "interleaved", True, False),
    ((70, 71, 2), (9, 12, 12), 12, 3, 256, 64, "e4m3", "bf16", (25, 50, 50), "blocks", False, True),       # rot 250
    ((130,), (130,), 131, 4, 64, 128, "bf16", "bf16", (9, 20), "interleaved", True, True),                  # rot 58
    ((31, 16), (5, 1), 5, 16, 256, 16, "f16", "f16", (10, 20, 4, 30), "interleaved", False, False),
]


@pytest.mark.parametrize("lens,lens_q,s,h,d,page,kind,rows,sections,order,inter,slot_major", WRITE)
def test_cache_write_with_axes(lens, lens_q, s, h, d, page, kind, rows, sections, order, inter, slot_major):
    m, g, b = lib(), torch.Generator().manual_seed(2), len(lens)
    c = make_cache(lens, h, d, page, kind, seed=4, slot_major=slot_major, fill=2.0)
    k, v = (bshd(g, rows, b, h, s, d, token_major=i == 0) for i in range(2))
    rot, axes = 2 * sum(sections), m.sdpa_rope_axes(sections, order=order)
    table, _ = m.sdpa_rope_table(rot, scaling="linear", factor=2.0)
    freqs, _ = so.inv_freq(rot, scaling="linear", factor=2.0)
    pos_np, pos = where("near", len(sections), b, s, 11)
    old = values_of(c.k), values_of(c.v)
    lq = None if lens_q is None else torch.tensor(lens_q, dtype=torch.int32, device="cuda")
    m.sdpa_cache_write(k, v, *c.where(), seq_lens_q=lq, **c.scales(), rope_table=table, positions=pos, interleaved=inter, attn_factor=1.25, axes=axes)
    torch.cuda.synchronize()
    want_k, reach = po.rotate_axes(f64(k), pos_np, axes, freqs, inter, 1.25)
    touched = np.zeros((c.k.shape[0], page), dtype=bool)
    for cache, scale, want, rc, before in ((c.k, c.k_scale, want_k, reach, old[0]), (c.v, c.v_scale, f64(v), np.zeros(v.shape), old[1])):
        got, sc = values_of(cache), None if scale is None else f64(scale)
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
        assert np.array_equal(got.transpose(0, 2, 1, 3)[~touched], before.transpose(0, 2, 1, 3)[~touched], equal_nan=True)
