"""Host-side checks of the serving entry points: the rotary table, and what is refused before any launch (no GPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import serving_oracle as so

FAKE = 0x7F0000000000   # 16-byte aligned, never dereferenced: every call below fails validation


@pytest.fixture(scope="module")
def m():
    import attention_flashattention_sdpa_gb300 as mod
    return mod


def _as_fraction(table):
    return [(int(t) % (1 << 64)) / 2.0 ** 64 for t in table]


@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                dict(scaling="yarn", factor=16.0, original_context=4096.0),
                                dict(scaling="yarn", factor=2.0, original_context=100.0, beta_fast=4.0, beta_slow=0.5)])
@pytest.mark.parametrize("rot,base", [(64, 10000.0), (128, 500000.0), (6, 100.0)])
def test_rope_table(m, rot, base, kw):
    table, att = m.sdpa_rope_table(rot, base, device="cpu", **kw)
    freqs, att_ref = so.inv_freq(rot, base, **kw)
    want = freqs / (2 * math.pi)
    got = np.array(_as_fraction(table))
    assert table.dtype == torch.int64 and table.shape == (rot // 2,)
    # fp64 functions on both sides, and an entry is a whole number of 2^-64 turns: half of one is lost
    assert np.abs(got - want).max() <= 2.0 ** -48 and (np.abs(got - want) <= 2.0 ** -45 * want + 2.0 ** -65).all()
    assert abs(att - att_ref) <= 2.0 ** -22


def test_rope_table_of_own_frequencies(m):
    table, att = m.sdpa_rope_table(6, inv_freq=[1.0, 2 * math.pi + 1.0, -1.0], device="cpu")
    f = _as_fraction(table)
    assert att == 1.0 and abs(f[0] - f[1]) < 2.0 ** -50 and abs(f[0] + f[2] - 1.0) < 2.0 ** -50


@pytest.mark.parametrize("kw", [dict(rot=7), dict(rot=0), dict(rot=-2), dict(rot=8, base=0.0), dict(rot=8, base=math.inf),
                                dict(rot=8, scaling="linear", factor=0.5), dict(rot=2, scaling="ntk", factor=2.0),
                                dict(rot=8, scaling="yarn", factor=2.0),
                                dict(rot=8, scaling="yarn", factor=2.0, original_context=10, beta_fast=1, beta_slow=1),
                                dict(rot=4, inv_freq=[1.0, math.nan])])
def test_rope_table_refusals(m, kw):
    with pytest.raises(m.SdpaError):
        m.sdpa_rope_table(device="cpu", **kw)


def test_rope_table_argument_errors(m):
    with pytest.raises(ValueError):
        m.sdpa_rope_table(8, scaling="dynamic", device="cpu")
    with pytest.raises(ValueError):
        m.sdpa_rope_table(8, inv_freq=[1.0], device="cpu")
    assert m.lib.sdpa_rope_table(None, FAKE, None) == 1


def _rope(m, **over):
    st = m.Strides(4 * 10 * 128, 10 * 128, 128, 1)
    p = m.Rope(b=1, h_q=4, h_k=4, s=10, d=128, rot=64, dtype=m.DTYPE_BF16, interleaved=0, attn_factor=1.0, table=FAKE,
               positions=0, positions_stride=0, q=st, k=st, q_out=st, k_out=st)
    for k, v in over.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("over,status,msg", [
    (dict(b=0), 1, "sizes"), (dict(s=0), 1, "sizes"), (dict(h_k=-1), 1, "sizes"), (dict(d=12), 2, "head dim"),
    (dict(d=520), 2, "head dim"), (dict(dtype=2), 2, "F16 or BF16"), (dict(rot=63), 1, "rot"), (dict(rot=0), 1, "rot"),
    (dict(rot=130), 1, "rot"), (dict(interleaved=2), 1, "interleaved"), (dict(attn_factor=math.nan), 1, "attn_factor"),
    (dict(table=0), 1, "table"), (dict(table=FAKE + 4), 3, "table"), (dict(positions=FAKE + 2), 3, "positions"),
    (dict(positions_stride=-1), 1, "positions_stride"),
])
def test_rope_refusals(m, over, status, msg):
    for f in (m.lib.sdpa_rope_fwd, m.lib.sdpa_rope_bwd):
        assert f(ctypes.addressof(_rope(m, **over)), FAKE, FAKE, FAKE, FAKE, None) == status
        assert msg in m.sdpa_last_error_string()


def test_rope_view_refusals(m):
    f = m.lib.sdpa_rope_fwd
    p = _rope(m)
    at = ctypes.addressof(p)
    assert f(None, FAKE, FAKE, FAKE, FAKE, None) == 1
    assert f(at, None, FAKE, FAKE, FAKE, None) == 1 and "q: null" in m.sdpa_last_error_string()
    assert f(at, FAKE, FAKE, FAKE, FAKE + 8, None) == 3 and "k_out" in m.sdpa_last_error_string()
    q = _rope(m, q=m.Strides(4 * 10 * 128, 10 * 128, 256, 1))
    assert f(ctypes.addressof(q), FAKE, FAKE + 32, FAKE, FAKE + 64, None) == 3 and "its input" in m.sdpa_last_error_string()
    q = _rope(m, k=m.Strides(0, 10 * 128, 0, 1))
    assert f(ctypes.addressof(q), FAKE, FAKE, FAKE + 32, FAKE + 64, None) == 3 and "positive" in m.sdpa_last_error_string()


def _cache(m, **over):
    st = m.Strides(2 * 16 * 128, 16 * 128, 128, 1)
    c = m.Cache(num_pages=8, page_size=16, h_kv=2, d=128, dtype=m.DTYPE_BF16, b=2, max_pages=4, k=FAKE, v=FAKE, k_strides=st,
                v_strides=st, k_scale=0, v_scale=0, page_table=FAKE, page_table_stride=4, seq_lens_kv=FAKE)
    for k, v in over.items():
        setattr(c, k, v)
    return c


def _rows(m, **over):
    st = m.Strides(2 * 5 * 128, 5 * 128, 128, 1)
    r = m.CacheRows(s=5, dtype=m.DTYPE_BF16, k=st, v=st, seq_lens_q=0, rope=0)
    for k, v in over.items():
        setattr(r, k, v)
    return r


BAD_CACHE = [
    (dict(num_pages=0), 1, "cache sizes"), (dict(max_pages=0), 1, "cache sizes"), (dict(b=0), 1, "cache sizes"),
    (dict(page_size=24), 2, "page_size"), (dict(d=96), 2, "head dim"), (dict(dtype=3), 2, "E4M3"), (dict(dtype=2), 1, "k_scale"),
    (dict(dtype=2, k_scale=FAKE, v_scale=FAKE + 4), 3, "16-byte"), (dict(k_scale=FAKE), 1, "takes no"),
    (dict(page_table=0), 1, "page_table"), (dict(seq_lens_kv=0), 1, "seq_lens_kv"), (dict(page_table=FAKE + 2), 3, "4-byte"),
    (dict(page_table_stride=3), 3, "page_table_stride"), (dict(k=0), 1, "k cache"), (dict(v=FAKE + 8), 3, "v cache"),
]


@pytest.mark.parametrize("over,status,msg", BAD_CACHE)
def test_cache_refusals(m, over, status, msg):
    c, r, d, n = _cache(m, **over), _rows(m), _decode(m), ctypes.c_size_t(0)
    a, b, e = (ctypes.addressof(x) for x in (c, r, d))
    for f in (m.lib.sdpa_cache_write, m.lib.sdpa_cache_read):
        assert f(a, b, FAKE, FAKE, None) == status and msg in m.sdpa_last_error_string()
    assert m.lib.sdpa_decode(a, e, FAKE, FAKE, None, FAKE, 1 << 40, None) == status and msg in m.sdpa_last_error_string()
    assert m.lib.sdpa_decode_workspace_size(a, e, ctypes.byref(n)) == status


def test_rows_refusals(m):
    c = _cache(m)
    at = ctypes.addressof(c)
    for over, status, msg in ((dict(s=0), 1, "s=0"), (dict(dtype=2), 2, "F16 or BF16"), (dict(dtype=0), 2, "own dtype"),
                              (dict(seq_lens_q=FAKE + 1), 3, "seq_lens_q")):
        assert m.lib.sdpa_cache_write(at, ctypes.addressof(_rows(m, **over)), FAKE, FAKE, None) == status
        assert msg in m.sdpa_last_error_string()
    assert m.lib.sdpa_cache_write(at, None, FAKE, FAKE, None) == 1
    assert m.lib.sdpa_cache_read(None, None, FAKE, FAKE, None) == 1
    assert m.lib.sdpa_cache_read(at, ctypes.addressof(_rows(m)), FAKE, None, None) == 1 and "v: null" in m.sdpa_last_error_string()
    turn = _rope(m, rot=130)
    assert m.lib.sdpa_cache_write(at, ctypes.addressof(_rows(m, rope=ctypes.addressof(turn))), FAKE, FAKE, None) == 1
    assert "rot" in m.sdpa_last_error_string()


def _decode(m, **over):
    st = m.Strides(8 * 3 * 128, 3 * 128, 128, 1)
    d = m.Decode(h_q=8, s_q=3, dtype=m.DTYPE_BF16, causal=0, attn_scale=0.1, q=st, o=st, seq_lens_q=0, tree_mask=0,
                 tree_mask_stride=0)
    for k, v in over.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("over,status,msg", [
    (dict(h_q=0), 1, "sizes"), (dict(s_q=0), 1, "sizes"), (dict(h_q=7), 1, "multiple"), (dict(dtype=2), 2, "F16 or BF16"),
    (dict(dtype=0), 2, "its dtype"), (dict(causal=1), 2, "top-left"), (dict(causal=3), 1, "causal"),
    (dict(causal=2, tree_mask=FAKE), 2, "tree mask"), (dict(tree_mask=FAKE + 1), 3, "4-byte"),
    (dict(tree_mask=FAKE, tree_mask_stride=-1), 1, "tree_mask_stride"), (dict(attn_scale=math.inf), 1, "attn_scale"),
    (dict(s_q=1 << 28), 2, "too large"),
])
def test_decode_refusals(m, over, status, msg):
    c, d = _cache(m), _decode(m, **over)
    assert m.lib.sdpa_decode(ctypes.addressof(c), ctypes.addressof(d), FAKE, FAKE, None, FAKE, 1 << 40, None) == status
    assert msg in m.sdpa_last_error_string()


def test_decode_view_and_workspace_refusals(m):
    c, d, n = _cache(m), _decode(m), ctypes.c_size_t(0)
    a, e = ctypes.addressof(c), ctypes.addressof(d)
    f = m.lib.sdpa_decode
    assert m.lib.sdpa_decode_workspace_size(a, e, ctypes.byref(n)) == 0 and n.value > 0 and n.value % 256 == 0
    assert f(a, e, None, FAKE, None, FAKE, 1 << 40, None) == 1 and "q: null" in m.sdpa_last_error_string()
    assert f(a, e, FAKE, FAKE + 8, None, FAKE, 1 << 40, None) == 3
    assert f(a, e, FAKE, FAKE, FAKE + 2, FAKE, 1 << 40, None) == 3 and "lse" in m.sdpa_last_error_string()
    assert f(a, e, FAKE, FAKE, None, None, 1 << 40, None) == 4
    assert f(a, e, FAKE, FAKE, None, FAKE, n.value - 1, None) == 4 and str(n.value) in m.sdpa_last_error_string()
    assert f(a, e, FAKE, FAKE, None, FAKE + 16, 1 << 40, None) == 4


# ---- the Python binding refuses before it hands over a pointer --------------------------------------

def _py(m, **over):
    t = dict(q=torch.zeros(2, 8, 1, 128, dtype=torch.bfloat16), k_cache=torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16),
             v_cache=torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16), page_table=torch.zeros(2, 3, dtype=torch.int32),
             seq_lens_kv=torch.zeros(2, dtype=torch.int32))
    t.update(over)
    return t


def _py_decode(m, t, **kw):
    m.sdpa_decode(t["q"], t["k_cache"], t["v_cache"], t["page_table"], t["seq_lens_kv"], torch.empty_like(t["q"]),
                  workspace=torch.zeros(8), **kw)


def test_binding_refuses_cpu_tensors(m):
    with pytest.raises(ValueError, match="CUDA"):
        _py_decode(m, _py(m))
    q, table = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16), torch.zeros(32, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        m.sdpa_rope_fwd(q, None, q, None, table)


@pytest.mark.parametrize("over", [
    dict(page_table=torch.zeros(2, 3, dtype=torch.int64)), dict(seq_lens_kv=torch.zeros(3, dtype=torch.int32)),
    dict(seq_lens_kv=torch.zeros(2)), dict(v_cache=torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)),
    dict(page_table=torch.zeros(3, 2, dtype=torch.int32).T),
])
def test_binding_refuses_shapes(m, over):
    with pytest.raises(ValueError):
        _py_decode(m, _py(m, **over))


def test_binding_refuses_scales_of_another_shape(m):
    t = _py(m)
    with pytest.raises(ValueError, match="k_scale"):
        _py_decode(m, t, k_scale=torch.zeros(4, 16, 2), v_scale=torch.zeros(4, 2, 16))


def test_binding_rope_shapes(m):
    q, table = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16), torch.zeros(32, dtype=torch.int64)
    with pytest.raises(ValueError, match="go together"):
        m.sdpa_rope_fwd(q, q, q, None, table)
    with pytest.raises(ValueError, match="table"):
        m.sdpa_rope_fwd(q, None, q, None, table.float())
    with pytest.raises(ValueError, match="positions"):
        m.sdpa_rope_fwd(q, None, q, None, table, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="dtype"):
        m.sdpa_rope_fwd(q.float(), None, q.float(), None, table)


def test_binding_structs_match_the_library(m):
    for i, cls in enumerate((m.RopeTable, m.Rope, m.Cache, m.CacheRows, m.Decode)):
        assert m.lib.sdpa_serving_struct_size(i) == ctypes.sizeof(cls)
    assert m.lib.sdpa_serving_struct_size(9) == 0


# ---- the oracle itself -----------------------------------------------------------------------------

def test_oracle_rotation_preserves_scores_at_equal_distance():
    """q.k after rotation depends on the distance of their positions alone."""
    rng = np.random.default_rng(0)
    f, _ = so.inv_freq(16)
    q, k = rng.normal(size=(1, 1, 1, 16)), rng.normal(size=(1, 1, 1, 16))
    dots = []
    for p in (0, 5, 1000):
        a, _ = so.rotate(q, np.array([[p + 7]]), f, True)
        b, _ = so.rotate(k, np.array([[p]]), f, True)
        dots.append((a * b).sum())
    assert np.ptp(dots) < 1e-9


def test_oracle_attention_is_dense_attention():
    """One page of everything: the paged oracle equals softmax attention written out."""
    rng = np.random.default_rng(1)
    kv = rng.normal(size=(2, 2, 1, 16, 4))
    q = rng.normal(size=(1, 1, 2, 4))
    o, lse = so.attend(q, kv[0], kv[1], None, None, np.array([[1, 0]]), (20,), None, 0.5, True)[:2]
    k = np.concatenate([kv[0][1, 0], kv[0][0, 0][:4]])
    v = np.concatenate([kv[1][1, 0], kv[1][0, 0][:4]])
    for r in range(2):
        n = 19 + r
        p = np.exp(0.5 * k[:n] @ q[0, 0, r])
        assert np.allclose(o[0, 0, r], p @ v[:n] / p.sum()) and np.isclose(lse[0, 0, r], np.log(p.sum()))


def test_first_calls_from_two_threads(m, monkeypatch):
    """A call that comes while another thread's first one still looks up what it needs of torch finds all of it, too."""
    import threading
    q, table = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16), torch.zeros(32, dtype=torch.int64)
    monkeypatch.setattr(m._Lazy, "torch", None)
    monkeypatch.setattr(m, "_DTYPES", {})
    look_up, inside, go = m.dtype_code, threading.Event(), threading.Event()

    def slow(t):
        if threading.current_thread().name == "first":
            inside.set()
            assert go.wait(30)
        return look_up(t)

    monkeypatch.setattr(m, "dtype_code", slow)
    said = {}

    def call():
        try:
            m.sdpa_rope_fwd(q, None, q, None, table)
        except ValueError as e:
            said[threading.current_thread().name] = str(e)

    first = threading.Thread(target=call, name="first")
    first.start()
    assert inside.wait(30)
    second = threading.Thread(target=call, name="second")
    second.start()
    second.join(30)
    go.set()
    first.join(30)
    assert "CUDA" in said["second"] and "CUDA" in said["first"]      # the tensors are on the CPU; nothing else is wrong


@pytest.mark.parametrize("h_q,h_kv,s_q,d,dtype", [(8, 2, 1, 128, 1), (32, 8, 1, 128, 2), (64, 1, 4, 64, 1), (16, 16, 3, 256, 2),
                                                  (64, 8, 64, 128, 2), (320, 40, 128, 128, 1), (8, 2, 70, 256, 1)])
def test_a_workspace_for_more_columns_serves_fewer(m, h_q, h_kv, s_q, d, dtype):
    before, n = 0, ctypes.c_size_t(0)
    for columns in (1, 2, 3, 7, 16, 20, 21, 60, 100, 500, 2048, 40000):
        st = m.Strides(h_kv * 64 * d, 64 * d, d, 1)
        scales = dict(k_scale=FAKE, v_scale=FAKE) if dtype == 2 else {}
        c = _cache(m, page_size=64, h_kv=h_kv, d=d, dtype=dtype, b=3, max_pages=columns, page_table_stride=columns, k_strides=st,
                   v_strides=st, **scales)
        e = _decode(m, h_q=h_q, s_q=s_q, dtype=1)
        assert m.lib.sdpa_decode_workspace_size(ctypes.addressof(c), ctypes.addressof(e), ctypes.byref(n)) == 0
        assert n.value >= before
        before = n.value
