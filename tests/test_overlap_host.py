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
