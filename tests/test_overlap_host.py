"""What a call writes lies apart from what it reads: refused before any launch (no GPU)."""
import ctypes

import pytest

FAKE = 0x7F0000000000   # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def m():
    import torch

    import attention_flashattention_sdpa_gb300 as mod
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: a call that is not refused must find no GPU")
    return mod


# ---- verification: 3 sequences of 5 rows --------------------------------------------------------

READ = dict(tokens=FAKE, parents=FAKE + 0x1000, seq_lens_q=FAKE + 0x2000, uniform=FAKE + 0x3000)
WRITTEN = dict(accepted=FAKE + 0x4000, path=FAKE + 0x5000, new_tokens=FAKE + 0x6000)
ROWS = dict(tokens=15, parents=15, uniform=15, path=15, new_tokens=15, seq_lens_q=3, accepted=3)


def verify(m, **over):
    p = m.Verify(b=3, s=5, vocab=100, dtype=m.DTYPE_F32, probs=FAKE + 0x100000, probs_b=500, probs_s=100, **{**READ, **WRITTEN, **over})
    return m.lib.sdpa_verify(ctypes.addressof(p), None)


@pytest.mark.parametrize("out", WRITTEN)
@pytest.mark.parametrize("other", [*READ, *WRITTEN])
def test_verify_refuses_outputs_that_overlap(m, out, other):
    if out == other:
        pytest.skip("itself")
    at = {**READ, **WRITTEN}[other]
    for delta in (0, 4 * (ROWS[other] - 1), -4 * (ROWS[out] - 1)):
        assert verify(m, **{out: at + delta}) == 3 and "apart" in m.sdpa_last_error_string(), (out, other, delta)
    for delta in (4 * ROWS[other], -4 * ROWS[out]):      # next to each other: past the checks, and then there is no GPU
        assert verify(m, **{out: at + delta}) == 5, m.sdpa_last_error_string()


def test_verify_without_the_optional_inputs(m):
    assert verify(m, parents=0, seq_lens_q=0) == 5, m.sdpa_last_error_string()


# ---- pages: 3 rows of 4 columns (6 words apart), 100 pages ---------------------------------------

PAGES = dict(page_table=(FAKE, 16), seq_lens=(FAKE + 0x1000, 3), ref_counts=(FAKE + 0x2000, 100), page_table_out=(FAKE + 0x3000, 16),
             ref_counts_out=(FAKE + 0x4000, 100))
LISTS = dict(fork=dict(parents=(FAKE + 0x5000, 3), seq_lens_out=(FAKE + 0x6000, 3)),
             grow=dict(new_lens=(FAKE + 0x5000, 3), src=(FAKE + 0x6000, 3), dst=(FAKE + 0x7000, 3), missing=(FAKE + 0x8000, 1)),
             free=dict(keep_lens=(FAKE + 0x5000, 3)), compact=dict(src=(FAKE + 0x6000, 7), dst=(FAKE + 0x7000, 7)))
OUT = {"page_table_out", "ref_counts_out", "seq_lens_out", "src", "dst", "missing"}


def pages(m, call, in_place=(), **over):
    at = {name: a for name, (a, _) in {**PAGES, **LISTS[call]}.items()}
    at.update(over)
    for name in in_place:
        at[name + "_out"] = at[name]
    p = m.Pages(num_pages=100, page_size=16, b=3, max_pages=4, page_table_stride=6, page_table_out_stride=6, **{n: at[n] for n in PAGES})
    held, L = ctypes.addressof(p), m.lib
    if call == "fork":
        return L.sdpa_cache_fork(held, at["parents"], 3, at["seq_lens_out"], None)
    if call == "grow":
        return L.sdpa_cache_grow(held, at["new_lens"], at["src"], at["dst"], at["missing"], None)
    if call == "free":
        return L.sdpa_cache_free(held, at["keep_lens"], None)
    return L.sdpa_cache_compact(held, at["src"], at["dst"], 7, None)


@pytest.mark.parametrize("call", LISTS)
def test_pages_refuse_what_overlaps(m, call):
    """Every output on the first and the last word of every other operand, and right before and behind it."""
    where = {**PAGES, **LISTS[call]}
    for out in sorted(OUT & set(where)):
        n = where[out][1]
        for other, (at, words) in where.items():
            if other == out:
                continue
            same = out == other + "_out" and other in ("page_table", "ref_counts")
            for delta in (0, 4 * (words - 1), -4 * (n - 1)):
                if same and delta == 0 and not (call == "fork" and out == "page_table_out"):
                    continue             # in place
                got = pages(m, call, **{out: at + delta})
                assert got == 3 and "apart" in m.sdpa_last_error_string(), (out, other, delta, got)
            for delta in (4 * words, -4 * n):
                assert pages(m, call, **{out: at + delta}) == 5, (out, other, delta, m.sdpa_last_error_string())


@pytest.mark.parametrize("call", LISTS)
def test_pages_in_place(m, call):
    where = ("ref_counts",) if call == "fork" else ("page_table", "ref_counts")
    assert pages(m, call, in_place=where) == 5, m.sdpa_last_error_string()
    for name in sorted({"src", "dst", "missing", "seq_lens_out"} & set(LISTS[call])):
        for over in where:
            assert pages(m, call, in_place=where, **{name: PAGES[over][0] + 4}) == 3 and "apart" in m.sdpa_last_error_string()
    if "new_lens" in LISTS[call]:        # lengths that stay as they are
        assert pages(m, call, in_place=where, new_lens=PAGES["seq_lens"][0]) == 5, m.sdpa_last_error_string()
