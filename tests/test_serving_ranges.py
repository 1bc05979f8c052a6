"""Attention over an E4M3 cache at the ends of the range of its scales (GPU)."""
import numpy as np
import pytest
import torch

from sdpa_testlib import f64
from serving_testlib import DT, HALF_STEP, TINY, make_cache, randn, run_decode, values_of

pytestmark = pytest.mark.gpu


def queries(seed, dtype, s, h_q, d):
    x = randn(torch.Generator().manual_seed(seed), 1, s, h_q, d).to(DT[dtype]).cuda()
    return x.permute(0, 2, 1, 3)


def definition(c, n, q, scale):
    """Of one sequence over one KV head, every key seen, in 64 bits: the weights [rows, n] (rows: [h_q, s]), LSE, V's
    codes [n, d] and scales [n], and reach [rows, n] = |scale| sum_d |q_d k_jd|."""
    pages = c.page_table.cpu().numpy()[0][np.arange(n) // c.k.shape[2]]
    slot = np.arange(n) % c.k.shape[2]
    k = values_of(c.k)[pages, 0, slot] * f64(c.k_scale)[pages, 0, slot][:, None]
    rows = f64(q)[0].reshape(-1, q.shape[-1])
    x = scale * (rows @ k.T)
    big = x.max(-1, keepdims=True)
    p = np.exp(x - big)
    total = p.sum(-1, keepdims=True)
    return p / total, (big + np.log(total))[:, 0], values_of(c.v)[pages, 0, slot], f64(c.v_scale)[pages, 0, slot], \
        abs(scale) * (np.abs(rows) @ np.abs(k).T)


def check(c, n, q, dtype, o, lse, scale):
    """The bounds of assert_attend_close with the scores' error written out (d / 16 steps of a tensor core's sum, each off
    by 2^-21 of reach; ex2, log2 and up to 32 moves of the reference: 2^-17), and what F16 weights add where the
    scales of V differ much: a weight times its scale over 2^v is off by half of F16's least step, 2^-25, where the
    row's largest weight is 2^5 or more (an offset of 2^6, an integer reference) and 2^v up to four times the largest
    scale, so by 2^-28 of the largest weight times the largest scale, times the code."""
    p, L, codes, vs, reach = definition(c, n, q, scale)
    v = codes * vs[:, None]
    want, spread = p @ v, p @ np.abs(v)
    score = q.shape[3] / 16 * 2.0 ** -21 * reach
    extra = vs.max() * 2.0 ** -28 * p.max(-1, keepdims=True) * np.abs(codes).sum(0)
    tol = (HALF_STEP["f16"] + 2.0 ** -17 + score.max(-1, keepdims=True)) * spread + extra + \
        HALF_STEP[dtype] * np.abs(want) * 1.01 + TINY[dtype]
    got = f64(o)[0].reshape(want.shape)
    assert np.isfinite(got).all(), "O is not finite"
    worst = (np.abs(got - want) / tol).max()
    assert worst <= 1, f"O: {worst:.2f} of the tolerance"
    err = np.abs(f64(lse).reshape(-1) - L)
    assert (err <= (p * score).sum(-1) + 2.0 ** -17 + 2.0 ** -20 * np.abs(L)).all(), f"LSE: max err {err.max():.3e}"


def scaled(pattern, c, g):
    """Puts a pattern into V's scales (of every slot; those behind the sequence do not count)."""
    vs = c.v_scale
    pick = torch.rand(vs.shape, generator=g).cuda()
    if pattern == "mixed":                   # next to ordinary ones, scales that count for nothing, one kind subnormal
        vs.copy_(torch.where(pick < 0.4, 1.0, torch.where(pick < 0.7, 1e-30, 1e-40)))
    elif pattern == "tiny":
        vs.copy_(1e-30 * (1 + pick))
    elif pattern == "subnormal":
        vs.copy_(1e-40 * (1 + pick))
    elif pattern == "zero":
        vs.zero_()
    elif pattern == "zero next to the largest":
        vs.copy_(torch.where(pick < 0.5, 0.0, torch.where(pick < 0.98, 0.01, 2.0 ** 118)))
    elif pattern == "large":                 # a few rows of up to 448 * 2^118, in BF16's range
        vs.copy_(torch.where(pick < 0.02, 2.0 ** 118, 0.01))
    elif pattern == "one largest":           # a scale beyond 2^126, of codes that leave the values in range
        vs.fill_(0.01)
        pg, sl = c.page_table[0, 1].item(), 3
        vs[pg, 0, sl] = 1.5 * 2.0 ** 126
        c.v[pg, 0, sl] = torch.where(torch.arange(c.v.shape[3], device="cuda") % 2 == 0, 1.0, -0.5).to(c.v.dtype)


PATTERNS = ["mixed", "tiny", "subnormal", "zero", "large", "zero next to the largest", "one largest"]


# One token (a cluster a sequence; with many columns of the page table, runs of tiles that are joined), 12 rows (blocks of
# 16), 40 rows (one tile of 128 for both softmax warpgroups), 280 rows (a tile for each, and 24 rows more).
@pytest.mark.parametrize("columns", [None, 4096])
@pytest.mark.parametrize("s,h_q,d", [(1, 4, 128), (3, 4, 64), (1, 4, 256), (10, 4, 128), (10, 4, 64), (70, 4, 128)])
@pytest.mark.parametrize("pattern", PATTERNS)
def test_scales_of_values(pattern, s, h_q, d, columns):
    g, n = torch.Generator().manual_seed(50), 1500
    c = make_cache((n,), 1, d, 16, "e4m3", seed=51, wide=columns)
    scaled(pattern, c, g)
    q = queries(52, "bf16", s, h_q, d)
    # scores of some +-20, so that the weights of single keys differ by many powers of two
    scale = 5 * d ** -0.5
    o, lse = run_decode(c, q, scale=scale)
    check(c, n, q, "bf16", o, lse, scale)
    if pattern == "zero":
        assert not o.any()


@pytest.mark.parametrize("columns", [None, 4096])
@pytest.mark.parametrize("spoil", [float("nan"), float("inf")])
@pytest.mark.parametrize("s", [1, 3, 40])
def test_lse_does_not_depend_on_the_scales_of_values(s, spoil, columns):
    """A value scale that is not finite spoils O, and leaves LSE as it is."""
    c = make_cache((700,), 1, 128, 16, "e4m3", seed=53, wide=columns)
    q = queries(54, "bf16", s, 4, 128)
    clean, clean_lse = run_decode(c, q)
    c.v_scale[c.page_table[0, 20].item(), 0, 5] = spoil
    o, lse = run_decode(c, q)
    assert torch.equal(lse, clean_lse) and torch.isfinite(lse).all()
    assert torch.isfinite(clean).all() and not torch.isfinite(o).any()


@pytest.mark.parametrize("others", ["ordinary", "zero"])
@pytest.mark.parametrize("s,h_q", [(5, 2), (20, 8), (70, 4)])
def test_hidden_tokens_may_have_the_largest_scales(s, h_q, others):
    """A drafted token whose V is 2^118 times the others' changes nothing for the rows that do not see it."""
    c = make_cache((90,), 1, 128, 16, "e4m3", seed=55)
    if others == "zero":
        c.v_scale.zero_()
    q = queries(56, "bf16", s, h_q, 128)
    bad = s // 2
    tree = np.tril(np.ones((s, s), dtype=bool))[None]
    tree[0, :, bad] = False
    tree[0, bad, bad] = True
    clean, clean_lse = run_decode(c, q, tree=tree)
    pos = 90 - s + bad
    c.v_scale[c.page_table[0, pos // 16].item(), 0, pos % 16] = 2.0 ** 118
    o, lse = run_decode(c, q, tree=tree)
    rest = [i for i in range(s) if i != bad]
    off, was = (o - clean)[:, :, rest].double().abs(), clean[:, :, rest].double().abs()
    if s * h_q <= 32:
        assert not off.any() and torch.equal(lse[:, :, rest], clean_lse[:, :, rest])
    # Blocks of many rows: the exponents of a tile's weights take the scale's 2^7 or less in, so that they are off by half of
    # a step of 2^-16, the weights by 2^-17; the values are below 2^3, results are rounded to the next step or the one
    # beside it.  The sum of the row that sees the token is brought down by 2^e, e < 32, so that O stays in range, and e
    # joins the reference m, |m| < 32 here: below 2^6, off by half a step of 2^-18.  LSE has a step of its own too.
    assert (off <= 2.0 ** -7 * was + 2.0 ** -14).all()
    assert (lse - clean_lse).abs().max() <= 2.0 ** -17 + 2.0 ** -19 + 2.0 ** -21
    assert torch.isfinite(o).all() and (o[:, :, bad].abs().amax(-1) > 2.0 ** 90).all()


@pytest.mark.parametrize("s,h_q", [(1, 4), (10, 4)])
def test_long_sequence_of_zero_scales(s, h_q):
    """Rows of V that are all zero count in the sums like any others, however many there are."""
    n = 131072
    c = make_cache((n,), 1, 64, 128, "e4m3", seed=57)
    c.v_scale.zero_()
    c.k_scale.zero_()              # every score 0: no key weighs less than the largest
    q = queries(58, "bf16", s, h_q, 64)
    o, lse = run_decode(c, q)
    check(c, n, q, "bf16", o, lse, 0.125)
    assert not o.any()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("s", [1, 10, 70])
def test_scales_of_values_grow(s, dtype):
    """Scales that grow by many powers of two along the sequence, and fall again; results in both types."""
    n = 3000
    c = make_cache((n,), 1, 128, 16, "e4m3", seed=59)
    at = torch.arange(n, device="cuda")
    size = 2.0 ** (-((at - n // 2).abs() // 100).float())        # 2^-15 .. 1 .. 2^-15
    c.v_scale[c.page_table[0].long()[at // 16], 0, at % 16] = 0.01 * size
    q = queries(60, dtype, s, 4, 128)
    o, lse = run_decode(c, q)
    check(c, n, q, dtype, o, lse, 128 ** -0.5)


@pytest.mark.parametrize("s", [1, 20])
@pytest.mark.parametrize("kind,q_size,k_size,scale", [("e4m3", 2.0 ** -60, 1.0, 0.0), ("e4m3", 2.0 ** -100, 1.0, 1e-38),
                                                      ("bf16", 1.0, 2.0 ** 110, 0.0), ("e4m3", 1.0, 2.0 ** 110, 0.0)])
def test_scores_of_zero(kind, q_size, k_size, scale, s):
    """A scale on the scores of zero, or so small that they are next to nothing: every visible key weighs the same, and those
    behind the sequence nothing."""
    n = 200
    c = make_cache((n,), 1, 128, 16, kind, seed=61)
    if kind == "e4m3":
        c.k_scale *= k_size
    else:
        c.k *= k_size
    q = queries(62, "bf16", s, 4, 128) * q_size
    o, lse = run_decode(c, q, scale=scale)
    pages, slot = c.page_table.cpu().numpy()[0][np.arange(n) // 16], np.arange(n) % 16
    v = values_of(c.v)[pages, 0, slot] * (f64(c.v_scale)[pages, 0, slot][:, None] if kind == "e4m3" else 1.0)
    weights = "f16" if kind == "e4m3" else "bf16"
    # no rounding of a weight but its own and the scale's it holds; results to BF16
    tol = (HALF_STEP[weights] + 2.0 ** -17) * np.abs(v).mean(0) + HALF_STEP["bf16"] * np.abs(v.mean(0)) * 1.01
    assert (np.abs(f64(o)[0] - v.mean(0)) <= tol).all()
    assert np.abs(f64(lse) - np.log(n)).max() <= 2.0 ** -17


@pytest.mark.parametrize("s", [1, 20])
def test_scores_of_zero_times_what_is_not_finite(s):
    """Zero times an infinity of Q is a NaN, and no zero."""
    c = make_cache((200,), 1, 128, 16, "bf16", seed=63)
    q = queries(64, "bf16", s, 4, 128)
    q[0, 1, s - 1, 5] = float("inf")
    o, lse = run_decode(c, q, scale=0.0)
    bad = torch.zeros(1, 4, s, dtype=torch.bool, device="cuda")
    bad[0, 1, s - 1] = True
    assert torch.isnan(lse[bad]).all() and torch.isnan(o[bad]).all()
    assert torch.isfinite(lse[~bad]).all() and torch.isfinite(o[~bad]).all()


@pytest.mark.parametrize("kind,dtype,s,h_q,d", [("bf16", "bf16", 1, 8, 128), ("bf16", "bf16", 2, 3, 64), ("bf16", "bf16", 1, 2, 256),
                                                ("f16", "f16", 1, 4, 128), ("f16", "f16", 2, 4, 256), ("e4m3", "f16", 1, 8, 128)])
@pytest.mark.parametrize("columns", [None, 4096])
def test_weights_of_few_rows_are_held_in_two_terms(kind, dtype, s, h_q, d, columns):
    """O within the rounding of its store and of weights to twice the bits of one term (half a step of half a step).

    The rest: scores as in check(); with |q k| scale below 2^5 a weight's exponent is off by under 2^-18, ex2 and sums by
    2^-20, F16's least step by 2^-25 of weights of 2^6 (all keys together: 2^-20)."""
    n = 1500
    c = make_cache((n,), 1, d, 16, kind, seed=65, wide=columns)
    q = queries(66, dtype, s, h_q, d)
    o, _ = run_decode(c, q)
    pages, slot = c.page_table.cpu().numpy()[0][np.arange(n) // 16], np.arange(n) % 16
    by = (lambda t: f64(t)[pages, 0, slot][:, None]) if kind == "e4m3" else (lambda t: 1.0)
    k, v = values_of(c.k)[pages, 0, slot] * by(c.k_scale), values_of(c.v)[pages, 0, slot] * by(c.v_scale)
    rows = f64(q)[0].reshape(-1, d)
    x = rows @ k.T * d ** -0.5
    assert np.abs(x).max() < 32
    p = np.exp(x - x.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    score = d / 16 * 2.0 ** -21 * (d ** -0.5 * (np.abs(rows) @ np.abs(k).T)).max(-1, keepdims=True)
    want, spread = p @ v, p @ np.abs(v)
    two = HALF_STEP["bf16" if kind == "bf16" else "f16"] ** 2
    tol = (two + score + 2.0 ** -17) * spread + HALF_STEP[dtype] * np.abs(want) * 1.01 + TINY[dtype]
    assert (np.abs(f64(o)[0].reshape(want.shape) - want) <= tol).all()
