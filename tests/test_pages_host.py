"""Host-side checks of the axes of rotary positions, of the pages of a cache and of verified drafts: what is refused before any launch,
and the oracle itself (no GPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import pages_oracle as po
from oracle import serving_oracle as so

FAKE = 0x7F0000000000   # 16-byte aligned, never dereferenced: every call below fails validation


@pytest.fixture(scope="module")
def m():
    import attention_flashattention_sdpa_gb300 as mod
    return mod


_held = []      # the structures whose addresses are out


def addr(x):
    _held.append(x)
    return ctypes.addressof(x)


def test_structs_match_the_library(m):
    for i, cls in ((5, m.RopeAxes), (6, m.Pages), (7, m.Verify)):
        assert m.lib.sdpa_serving_struct_size(i) == ctypes.sizeof(cls)
    assert m.lib.sdpa_serving_struct_size(8) == 0


# ---- axes ---------------------------------------------------------------------------------

def test_axes_of_sections(m):
    assert m.sdpa_rope_axes((2, 3, 1)) == bytes([0, 0, 1, 1, 1, 2])
    assert m.sdpa_rope_axes([2, 3, 1], order="interleaved") == bytes([0, 1, 2, 0, 1, 1])
    assert m.sdpa_rope_axes([4]) == bytes(4)
    for bad in ([], [1, 0], [1, 1, 1, 1, 1], [-1, 2]):
        with pytest.raises(ValueError, match="sections"):
            m.sdpa_rope_axes(bad)
    with pytest.raises(ValueError, match="order"):
        m.sdpa_rope_axes([1, 1], order="rows")


def _rope(m, **over):
    st = m.Strides(4 * 10 * 128, 10 * 128, 128, 1)
    p = m.Rope(b=1, h_q=4, h_k=4, s=10, d=128, rot=64, dtype=m.DTYPE_BF16, interleaved=0, attn_factor=1.0, table=FAKE,
               positions=FAKE, positions_stride=10, q=st, k=st, q_out=st, k_out=st)
    for k, v in over.items():
        setattr(p, k, v)
    return p


def _axes(m, axes=2, axis=None, stride=10):
    a = m.RopeAxes(axes=axes, axis_stride=stride)
    for i, x in enumerate([0] * 16 + [1] * 16 if axis is None else axis):
        a.axis[i] = x
    return a


def _cache(m, **over):
    st = m.Strides(2 * 16 * 128, 16 * 128, 128, 1)
    c = m.Cache(num_pages=8, page_size=16, h_kv=2, d=128, dtype=m.DTYPE_BF16, b=2, max_pages=4, k=FAKE, v=FAKE, k_strides=st,
                v_strides=st, k_scale=0, v_scale=0, page_table=FAKE, page_table_stride=4, seq_lens_kv=FAKE)
    for k, v in over.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("rope,axes,status,msg", [
    ({}, None, 1, "axes descriptor"), ({}, dict(axes=0), 2, "axes"), ({}, dict(axes=5), 2, "axes"), ({}, dict(stride=-1), 1, "axis_stride"),
    ({}, dict(axis=[0] * 31 + [2]), 1, "axis[31]"), (dict(positions=0), {}, 1, "positions"), (dict(rot=63), {}, 1, "rot"),
    (dict(positions=FAKE + 2), {}, 3, "positions"), (dict(d=12), {}, 2, "head dim"),
])
def test_axes_refusals(m, rope, axes, status, msg):
    p, a = _rope(m, **rope), None if axes is None else _axes(m, **axes)
    for f in (m.lib.sdpa_rope_axes_fwd, m.lib.sdpa_rope_axes_bwd):
        assert f(addr(p), None if a is None else addr(a), FAKE, FAKE, FAKE, FAKE, None) == status
        assert msg in m.sdpa_last_error_string()
    if "d" not in rope:      # (the write's d is the cache's)
        st = m.Strides(2 * 5 * 128, 5 * 128, 128, 1)
        r = m.CacheRows(s=5, dtype=m.DTYPE_BF16, k=st, v=st, seq_lens_q=0, rope=addr(p))
        c = _cache(m)
        assert m.lib.sdpa_cache_write_axes(addr(c), addr(r), None if a is None else addr(a), FAKE, FAKE, None) == status
        assert msg in m.sdpa_last_error_string()


def test_axes_of_a_write_need_a_rope(m):
    st, c, a = m.Strides(2 * 5 * 128, 5 * 128, 128, 1), _cache(m), _axes(m)
    r = m.CacheRows(s=5, dtype=m.DTYPE_BF16, k=st, v=st, seq_lens_q=0, rope=0)
    assert m.lib.sdpa_cache_write_axes(addr(c), addr(r), addr(a), FAKE, FAKE, None) == 1 and "rope" in m.sdpa_last_error_string()


def test_binding_axes(m):
    q, table = torch.zeros(2, 2, 3, 64, dtype=torch.bfloat16), torch.zeros(32, dtype=torch.int64)
    axes, pos = m.sdpa_rope_axes((10, 22)), torch.zeros(2, 2, 3, dtype=torch.int32)
    for bad in (axes[:-1], list(axes), "0" * 32):
        with pytest.raises(ValueError, match="axes must be bytes"):
            m.sdpa_rope_fwd(q, None, q, None, table, pos, axes=bad)
    for bad in (None, pos.long(), torch.zeros(2, 3, 3, dtype=torch.int32), torch.zeros(2, 2, 4, dtype=torch.int32),
                torch.zeros(3, dtype=torch.int32), torch.zeros(2, 3, 2, dtype=torch.int32).transpose(1, 2)):
        with pytest.raises(ValueError, match="positions"):
            m.sdpa_rope_fwd(q, None, q, None, table, bad, axes=axes)
    with pytest.raises(ValueError, match="CUDA"):
        m.sdpa_rope_bwd(q, None, q, None, table, pos, axes=axes)
    with pytest.raises(ValueError, match="rope_table"):
        c = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
        m.sdpa_cache_write(q, q, c, c, torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), axes=axes)


def test_oracle_one_axis_is_the_plain_rotation():
    rng = np.random.default_rng(0)
    x, pos = rng.normal(size=(2, 3, 5, 16)), rng.integers(-50, 50, (3, 2, 5))
    freqs, _ = so.inv_freq(12)
    for inter in (False, True):
        a, ra = po.rotate_axes(x, pos, [1] * 6, freqs, inter, 1.5)
        b, rb = so.rotate(x, pos[1], freqs, inter, 1.5)
        assert np.allclose(a, b) and np.allclose(ra, rb)


# ---- pages --------------------------------------------------------------------------------

def _pages(m, **over):
    p = m.Pages(num_pages=100, page_size=16, b=3, max_pages=4, page_table=FAKE, page_table_stride=4, seq_lens=FAKE + 0x1000,
                ref_counts=FAKE + 0x2000, page_table_out=FAKE + 0x3000, page_table_out_stride=4, ref_counts_out=FAKE + 0x4000)
    for k, v in over.items():
        setattr(p, k, v)
    return p


A, B, C = FAKE + 0x10000, FAKE + 0x20000, FAKE + 0x30000

BAD_PAGES = [
    (dict(num_pages=0), 1, "sizes"), (dict(page_size=0), 1, "sizes"), (dict(b=0), 1, "sizes"), (dict(max_pages=0), 1, "sizes"),
    (dict(page_size=24), 2, "page_size"), (dict(page_table=0), 1, "page_table"), (dict(seq_lens=0), 1, "seq_lens"),
    (dict(ref_counts=0), 1, "ref_counts"), (dict(page_table_out=0), 1, "page_table_out"), (dict(ref_counts_out=0), 1, "ref_counts_out"),
    (dict(ref_counts=FAKE + 0x2002), 3, "4-byte"), (dict(page_table_stride=3), 3, "stride"), (dict(page_table_out_stride=3), 3, "stride"),
    (dict(page_table_out=FAKE + 16), 3, "apart"), (dict(ref_counts_out=FAKE + 0x2000 + 4), 3, "apart"),
    (dict(b=(1 << 24) + 1), 2, "too large"), (dict(num_pages=(1 << 30) + 1), 2, "too large"), (dict(max_pages=(1 << 30) + 1), 2, "too large"), (dict(max_pages=1 << 30, page_table_stride=1 << 30, page_table_out_stride=1 << 30, b=300), 2, "too large"),
]


@pytest.mark.parametrize("over,status,msg", BAD_PAGES)
def test_pages_refusals(m, over, status, msg):
    p = addr(_pages(m, **over))
    for got in (m.lib.sdpa_cache_fork(p, A, 3, B, None), m.lib.sdpa_cache_grow(p, A, B, C, C + 64, None),
                m.lib.sdpa_cache_free(p, A, None), m.lib.sdpa_cache_compact(p, A, B, 5, None)):
        assert got == status and msg in m.sdpa_last_error_string()


def test_pages_refusals_of_each_call(m):
    p, same = addr(_pages(m)), _pages(m, page_table_out=FAKE, page_table_out_stride=5)
    L = m.lib
    for call, status, msg in (
            (lambda: L.sdpa_cache_fork(None, A, 3, B, None), 1, "descriptor"),
            (lambda: L.sdpa_cache_grow(None, A, B, C, C + 64, None), 1, "descriptor"),
            (lambda: L.sdpa_cache_free(None, A, None), 1, "descriptor"),
            (lambda: L.sdpa_cache_compact(None, A, B, 5, None), 1, "descriptor"),
            (lambda: L.sdpa_cache_fork(p, None, 3, B, None), 1, "parents"), (lambda: L.sdpa_cache_fork(p, A, 0, B, None), 1, "sizes"),
            (lambda: L.sdpa_cache_fork(p, A, 3, B + 2, None), 3, "seq_lens_out"),
            (lambda: L.sdpa_cache_fork(p, A, 3, FAKE + 0x1008, None), 3, "seq_lens_out"),
            (lambda: L.sdpa_cache_fork(p, A, 3, A + 8, None), 3, "seq_lens_out"),
            (lambda: L.sdpa_cache_fork(addr(_pages(m, page_table_out=FAKE)), A, 3, B, None), 3, "apart"),
            (lambda: L.sdpa_cache_free(addr(same), A, None), 3, "stride"),
            (lambda: L.sdpa_cache_grow(addr(_pages(m, b=4097, page_table_out=FAKE)), A, B, C, C + 64, None), 2, "4097"),
            (lambda: L.sdpa_cache_grow(addr(_pages(m, b=2048, max_pages=1 << 20, page_table_stride=1 << 20, page_table_out=FAKE, page_table_out_stride=1 << 20)),
                                       A, B, C, C + 8192, None), 2, "2^31"),
            (lambda: L.sdpa_cache_grow(p, None, B, C, C + 64, None), 1, "new_lens"), (lambda: L.sdpa_cache_grow(p, A, None, C, C + 64, None), 1, "src"),
            (lambda: L.sdpa_cache_grow(p, A, B, C + 1, C + 64, None), 3, "dst"), (lambda: L.sdpa_cache_grow(p, A, B, C, None, None), 1, "missing"),
            (lambda: L.sdpa_cache_grow(p, A, B, B + 8, C, None), 3, "apart"), (lambda: L.sdpa_cache_free(p, None, None), 1, "keep_lens"),
            (lambda: L.sdpa_cache_compact(p, A, B, 0, None), 1, "pairs"), (lambda: L.sdpa_cache_compact(p, None, B, 5, None), 1, "src"),
            (lambda: L.sdpa_cache_compact(p, A, A + 16, 5, None), 3, "apart")):
        assert call() == status and msg in m.sdpa_last_error_string(), (status, msg, m.sdpa_last_error_string())


BAD_STORED = [
    (dict(num_pages=0), 1, "cache sizes"), (dict(page_size=24), 2, "page_size"), (dict(d=96), 2, "head dim"), (dict(dtype=3), 2, "E4M3"),
    (dict(dtype=2), 1, "k_scale"), (dict(k_scale=FAKE), 1, "takes no"), (dict(k=0), 1, "k cache"), (dict(v=FAKE + 8), 3, "v cache"),
]


@pytest.mark.parametrize("over,status,msg", BAD_STORED)
def test_copy_and_keep_refuse_a_cache(m, over, status, msg):
    c = addr(_cache(m, **over))
    assert m.lib.sdpa_cache_copy(c, A, B, 5, None) == status and msg in m.sdpa_last_error_string()
    assert m.lib.sdpa_cache_keep(c, A, B, 5, None, None) == status and msg in m.sdpa_last_error_string()


def test_copy_and_keep_refusals(m):
    c, bare = addr(_cache(m)), addr(_cache(m, b=0, max_pages=0, page_table=0, seq_lens_kv=0))
    L = m.lib
    for call, status, msg in (
            (lambda: L.sdpa_cache_copy(None, A, B, 5, None), 1, "descriptor"), (lambda: L.sdpa_cache_copy(bare, A, B, 0, None), 1, "pairs"),
            (lambda: L.sdpa_cache_copy(bare, None, B, 5, None), 1, "src"), (lambda: L.sdpa_cache_copy(c, A, B + 2, 5, None), 3, "dst"),
            (lambda: L.sdpa_cache_keep(None, A, B, 5, None, None), 1, "descriptor"), (lambda: L.sdpa_cache_keep(bare, A, B, 5, None, None), 1, "cache sizes"),
            (lambda: L.sdpa_cache_keep(c, A, B, 0, None, None), 1, "s=0"), (lambda: L.sdpa_cache_keep(c, None, B, 5, None, None), 1, "path"),
            (lambda: L.sdpa_cache_keep(c, A, None, 5, None, None), 1, "accepted"), (lambda: L.sdpa_cache_keep(c, A, B, 5, C + 1, None), 3, "seq_lens_q")):
        assert call() == status and msg in m.sdpa_last_error_string()


def test_binding_pages(m):
    i32 = dict(dtype=torch.int32)
    t, lens, refs, out = torch.zeros(2, 3, **i32), torch.zeros(2, **i32), torch.zeros(9, **i32), torch.zeros(2, 3, **i32)
    two, one, z = torch.zeros(2, **i32), torch.zeros(1, **i32), dict(page_size=16)
    with pytest.raises(ValueError, match="CUDA"):
        m.sdpa_cache_fork(t, lens, two, refs, out, two, **z)
    with pytest.raises(ValueError, match="CUDA"):
        m.sdpa_cache_grow(t, lens, two, refs, two, two, one, **z)
    with pytest.raises(ValueError, match="CUDA"):
        m.sdpa_cache_free(t, lens, two, refs, **z)
    with pytest.raises(ValueError, match="CUDA"):
        m.sdpa_cache_compact(t, lens, refs, two, two, **z)
    for call in (lambda: m.sdpa_cache_fork(t.long(), lens, two, refs, out, two, **z), lambda: m.sdpa_cache_fork(t, lens, two, refs, out[:1], two, **z),
                 lambda: m.sdpa_cache_fork(t, lens, two, refs, out.T, two, **z), lambda: m.sdpa_cache_fork(t, lens, t, refs, out, two, **z),
                 lambda: m.sdpa_cache_fork(t, lens, two, refs, out, one, **z), lambda: m.sdpa_cache_grow(t, one, two, refs, two, two, one, **z),
                 lambda: m.sdpa_cache_grow(t, lens, two, refs, one, one, one, **z), lambda: m.sdpa_cache_grow(t, lens, two, refs, two, two, two, **z),
                 lambda: m.sdpa_cache_grow(t, lens, two, refs, two, one, one, **z), lambda: m.sdpa_cache_free(t, lens, two.long(), refs, **z),
                 lambda: m.sdpa_cache_free(t, lens, two, refs.float(), **z), lambda: m.sdpa_cache_free(t, lens, two, refs, ref_counts_out=one, **z),
                 lambda: m.sdpa_cache_free(t, lens, two, refs, page_table_out=out[:, :2], **z), lambda: m.sdpa_cache_compact(t, lens, t, two, two, **z),
                 lambda: m.sdpa_cache_compact(t, lens, refs, t, two, **z)):
        with pytest.raises(ValueError):
            call()


def test_binding_copy_and_keep(m):
    c = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32)
    pairs, t, lens = torch.zeros(3, **i32), torch.zeros(2, 3, **i32), torch.zeros(2, **i32)
    with pytest.raises(ValueError, match="CUDA"):
        m.sdpa_cache_copy(c, c, pairs, pairs)
    with pytest.raises(ValueError, match="CUDA"):
        m.sdpa_cache_keep(c, c, t, lens, torch.zeros(2, 5, **i32), lens)
    for call in (lambda: m.sdpa_cache_copy(c, c[:3], pairs, pairs), lambda: m.sdpa_cache_copy(c, c, pairs, pairs[:2]),
                 lambda: m.sdpa_cache_copy(c, c, pairs.long(), pairs), lambda: m.sdpa_cache_copy(c, c, t, t),
                 lambda: m.sdpa_cache_copy(c, c, pairs, pairs, k_scale=torch.zeros(4, 16, 2), v_scale=torch.zeros(4, 2, 16)),
                 lambda: m.sdpa_cache_keep(c, c, t, lens, lens, lens), lambda: m.sdpa_cache_keep(c, c, t, lens, torch.zeros(3, 5, **i32), lens),
                 lambda: m.sdpa_cache_keep(c, c, t, lens, torch.zeros(2, 5, **i32), lens[:1]),
                 lambda: m.sdpa_cache_keep(c, c, t, lens, torch.zeros(2, 5, **i32), lens, seq_lens_q=lens.long())):
        with pytest.raises(ValueError):
            call()


def test_oracle_pages_by_hand():
    """Two sequences of 20 and 16 tokens in pages of 16; the first is taken over twice, and both grow in its last page."""
    rows, lens, counts = po.fork([[3, 1, -1], [5, 0, -1]], [20, 16], [0, 0, -1], [0, 1, 0, 1, 0, 1], 16)
    assert rows == [[3, 1, -1], [3, 1, -1], [-1, -1, -1]] and lens == [20, 20, 0] and counts == [0, 2, 0, 2, 0, 0]
    rows, counts, src, dst, missing = po.grow(rows, lens, [21, 33, 1], counts, 16)
    assert rows == [[3, 0, -1], [3, 1, 2], [4, -1, -1]] and (src, dst, missing) == ([1, -1, -1], [0, -1, -1], 0)
    assert counts == [1, 1, 1, 2, 1, 0]
    assert po.grow(rows, [21, 33, 1], [48, 48, 33], counts, 16)[2:] == ([-1] * 3, [-1] * 3, 2)
    rows, counts = po.free(rows, [21, 33, 1], [0, 17, 1], counts, 16)
    assert rows == [[-1, -1, -1], [3, 1, -1], [4, -1, -1]] and counts == [0, 1, 0, 1, 1, 0]
    rows, counts, src, dst = po.compact(rows, [0, 17, 1], counts, 3, 16)
    assert rows == [[-1, -1, -1], [0, 1, -1], [2, -1, -1]] and counts == [1, 1, 1, 0, 0, 0]
    assert (src, dst) == ([3, 4, -1], [0, 2, -1])


# ---- verification -------------------------------------------------------------------------

def _verify(m, **over):
    p = m.Verify(b=2, s=4, vocab=100, dtype=m.DTYPE_F32, tokens=FAKE, parents=0, seq_lens_q=0, uniform=FAKE, probs=FAKE, probs_b=400,
                 probs_s=100, draft_probs=0, draft_b=0, draft_s=0, accepted=FAKE, path=FAKE, new_tokens=FAKE)
    for k, v in over.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("over,status,msg", [
    (dict(b=0), 1, "sizes"), (dict(s=0), 1, "sizes"), (dict(vocab=0), 1, "sizes"), (dict(s=1025), 2, "rows"), (dict(vocab=(1 << 20) + 1), 2, "vocabulary"),
    (dict(b=(1 << 24) + 1), 2, "too large"), (dict(dtype=2), 2, "F16, BF16 or F32"), (dict(parents=FAKE, draft_probs=FAKE), 2, "chain"),
    (dict(tokens=0), 1, "tokens"), (dict(uniform=FAKE + 2), 3, "uniform"), (dict(accepted=0), 1, "accepted"), (dict(path=0), 1, "path"),
    (dict(new_tokens=FAKE + 1), 3, "new_tokens"), (dict(parents=FAKE + 2), 3, "parents"), (dict(seq_lens_q=FAKE + 2), 3, "seq_lens_q"),
    (dict(probs=0), 1, "probs"), (dict(probs=FAKE + 2), 3, "probs"), (dict(draft_probs=FAKE + 2), 3, "draft_probs"),
    (dict(probs_s=-1), 3, "strides"), (dict(draft_b=-1), 3, "strides"),
])
def test_verify_refusals(m, over, status, msg):
    p = _verify(m, **over)
    assert m.lib.sdpa_verify(addr(p), None) == status and msg in m.sdpa_last_error_string()


def test_verify_without_a_descriptor(m):
    assert m.lib.sdpa_verify(None, None) == 1 and "descriptor" in m.sdpa_last_error_string()


def test_binding_verify(m):
    i = torch.zeros(2, 3, dtype=torch.int32)
    n, u, p = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3), torch.zeros(2, 3, 7)
    with pytest.raises(ValueError, match="CUDA"):
        m.sdpa_verify(i, p, u, n, i, i)
    for call in (lambda: m.sdpa_verify(i, p.double(), u, n, i, i), lambda: m.sdpa_verify(i, p[0], u, n, i, i),
                 lambda: m.sdpa_verify(i, p.transpose(1, 2), u, n, i, i), lambda: m.sdpa_verify(i.long(), p, u, n, i, i),
                 lambda: m.sdpa_verify(i, p, u.double(), n, i, i), lambda: m.sdpa_verify(i, p, u, i, i, i), lambda: m.sdpa_verify(i, p, u, n, n, i),
                 lambda: m.sdpa_verify(i, p, u, n, i, n), lambda: m.sdpa_verify(i, p, u, n, i, i, parents=n),
                 lambda: m.sdpa_verify(i, p, u, n, i, i, draft_probs=p.half()), lambda: m.sdpa_verify(i, p, u, n, i, i, draft_probs=p[:, :, :6]),
                 lambda: m.sdpa_verify(i, p, u, n, i, i, seq_lens_q=u[0])):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("draft", [False, True])
def test_oracle_verification_keeps_the_distribution(draft):
    """Summed over a grid of random numbers (and over what the draft draws), one drafted token and the token that replaces a refused
    one are distributed as the target's own."""
    p, q = np.array([0.5, 0.25, 0.25, 0.0]), np.array([0.25, 0.25, 0.125, 0.375])
    probs = np.stack([p, np.array([0.0, 0.0, 0.0, 1.0])])[None].astype(np.float32)
    grid = (np.arange(16) + 0.5) / 16
    got = np.zeros(4)
    for x, weight in enumerate(q):
        for u in grid:
            for v in grid:
                a, _, new = po.verify(np.array([[0, x]]), probs, np.array([[v, u]]), draft=np.stack([q, q])[None].astype(np.float32) if draft else None)
                got[new[0, 0]] += weight / 256
                assert a[0] == 1 or new[0, 1] == 3
    # A cell of the grid is 1/16: sums over it are exact but where a border cuts a cell, one border a token and draw.
    assert np.abs(got - p).max() <= 1 / 16


def test_oracle_masses():
    assert po.mass(0.5) == 1 << 41 and po.mass(math.nan) == 0 and po.mass(2.0) == 1 << 42 and po.mass(-1.0) == 0
    assert po.mass(1.5 * 2.0 ** -42) == 2 and po.mass(2.5 * 2.0 ** -42) == 2
