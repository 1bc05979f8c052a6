"""Oracle of rotary positions with several axes, of the pages of a cache and of verified drafts.

Plain numpy and Python's whole numbers, written from the definitions; it shares no code with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

UNIT = 1 << 42


def rotate_axes(x, positions, axis, freqs, interleaved=False, factor=1.0, inverse=False):
    """x [b, h, s, d] with positions [axes, b, s]: pair i turns by positions[axis[i]] * freqs[i].  Returns (y, reach) as
    serving_oracle.rotate does."""
    y, reach, n = x.copy(), np.zeros_like(x), len(freqs)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        t = positions[axis[i]].astype(np.float64)[:, None, :] * freqs[i] * (-1.0 if inverse else 1.0)
        c, s = factor * np.cos(t), factor * np.sin(t)
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
        reach[..., a] = reach[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(factor)
    return y, reach


def _clamped(lens, columns, page_size):
    return [min(max(int(n), 0), columns * page_size) for n in lens]


def _columns(n, page_size):
    return -(-n // page_size)


def fork(table, lens, parents, counts, page_size):
    """New rows, lengths and counts."""
    width = len(table[0])
    lens = _clamped(lens, width, page_size)
    counts, rows, out = list(counts), [], []
    for j in parents:
        n = lens[j] if 0 <= j < len(table) else 0
        row = [table[j][c] if c < _columns(n, page_size) else -1 for c in range(width)]
        rows.append(row)
        out.append(n)
        for page in row[: _columns(n, page_size)]:
            if 0 <= page < len(counts):
                counts[page] += 1
    for row, n in zip(table, lens):
        for page in row[: _columns(n, page_size)]:
            if 0 <= page < len(counts):
                counts[page] -= 1
    return rows, out, counts


def grow(table, lens, new_lens, counts, page_size):
    """Rows, counts, src, dst, missing."""
    width = len(table[0])
    lens, new_lens = _clamped(lens, width, page_size), _clamped(new_lens, width, page_size)
    rows, counts = [list(r) for r in table], list(counts)
    free = [page for page, c in enumerate(counts) if c == 0]
    src, dst = [-1] * len(lens), [-1] * len(lens)
    wanted = 0
    for i, (n, m) in enumerate(zip(lens, new_lens)):
        tail = rows[i][n // page_size] if n % page_size and m > n else -1
        if 0 <= tail < len(counts) and counts[tail] > 1:
            src[i] = tail
            if wanted < len(free):
                dst[i] = free[wanted]
                counts[dst[i]], rows[i][n // page_size] = 1, dst[i]
            counts[tail] -= 1
            wanted += 1
        for c in range(_columns(n, page_size), _columns(m, page_size)):
            if wanted < len(free):
                rows[i][c] = free[wanted]
                counts[free[wanted]] = 1
            wanted += 1
    if wanted > len(free):
        return None, None, [-1] * len(lens), [-1] * len(lens), wanted - len(free)
    return rows, counts, src, dst, 0


def free(table, lens, keep_lens, counts, page_size):
    """Rows and counts."""
    width = len(table[0])
    rows, counts = [list(r) for r in table], list(counts)
    for row, n, m in zip(rows, _clamped(lens, width, page_size), keep_lens):
        for c in range(_columns(min(n, max(int(m), 0)), page_size), _columns(n, page_size)):
            if 0 <= row[c] < len(counts):
                counts[row[c]] -= 1
            row[c] = -1
    return rows, counts


def compact(table, lens, counts, pairs, page_size):
    """Rows, counts, src, dst."""
    n = sum(c != 0 for c in counts)
    movers = [p for p in range(n, len(counts)) if counts[p] != 0]
    holes = [p for p in range(n) if counts[p] == 0]
    moves = list(zip(movers, holes))[:pairs]
    counts, to = list(counts), dict(moves)
    for a, b in moves:
        counts[b], counts[a] = counts[a], 0
    rows = []
    for row, m in zip(table, _clamped(lens, len(table[0]), page_size)):
        rows.append([to.get(p, p) if c < _columns(m, page_size) else p for c, p in enumerate(row)])
    src, dst = [a for a, _ in moves], [b for _, b in moves]
    return rows, counts, src + [-1] * (pairs - len(moves)), dst + [-1] * (pairs - len(moves))


def keep(slots, lens_kv, lens_q, s, path, accepted):
    """What moves: [(sequence, (page, slot) from, (page, slot) to)], in order; `slots(i, pos)` gives a position's place or None."""
    out = []
    for i, n in enumerate(lens_kv):
        m = min(max(int(lens_q[i]), 0), s) if lens_q is not None else s
        for j in range(min(max(int(accepted[i]), 0), m)):
            r = int(path[i][j])
            if not 0 <= r < m or r == j:
                continue
            a, b = (slots(i, n - m + x) if 0 <= n - m + x < n else None for x in (r, j))
            if a is not None and b is not None:
                out.append((i, a, b))
    return out


def mass(p):
    """A probability as a whole number of 2^-42, ties to even (as Python rounds); NaN as 0."""
    p = float(p)
    return 0 if math.isnan(p) else round(min(max(p, 0.0), 1.0) * UNIT)


def _masses(p):
    """The same of a whole row, exactly: fp32 values times 2^42 are exact in fp64, np.rint rounds ties to even."""
    p = np.where(np.isnan(p), 0.0, np.clip(p, 0.0, 1.0))
    return np.rint(p.astype(np.float64) * UNIT).astype(object)


def verify(tokens, probs, uniform, parents=None, draft=None, lens=None):
    """accepted, path, new_tokens of numpy arrays: tokens [b, s], probs [b, s, vocab] and draft as fp32 values, uniform [b, s]."""
    b, s, vocab = probs.shape
    accepted, paths, news = np.zeros(b, np.int64), np.full((b, s), -1, np.int64), np.full((b, s), -1, np.int64)
    for i in range(b):
        n = s if lens is None else min(max(int(lens[i]), 0), s)
        if n == 0:
            continue
        path, gone = [0], []
        known = lambda x: 0 <= x < vocab    # noqa: E731
        while True:
            at, gone, step = path[-1], [], None
            for j in range(1, n):
                up = j - 1 if parents is None else int(parents[i][j])
                if up != at or not 0 <= up < j:
                    continue
                x, u = int(tokens[i][j]), float(uniform[i][j])
                p = probs[i, at, x] if known(x) else np.float32(0)
                if draft is not None:
                    good = known(x) and u * float(draft[i, j, x]) < float(p)
                else:
                    left = max(0, UNIT - sum(mass(probs[i, at, y]) for y in set(gone) if known(y)))
                    good = u * float(left) < float(0 if x in gone else mass(p))
                if good:
                    step = j
                    break
                gone.append(x)
            if step is None:
                break
            path.append(step)
        row = whole = _masses(probs[i, path[-1]])
        if draft is not None and gone:
            with np.errstate(invalid="ignore"):
                row = _masses(probs[i, path[-1]].astype(np.float32) - draft[i, path[-1] + 1].astype(np.float32))
        elif gone:
            row = whole.copy()
            row[[y for y in gone if known(y)]] = 0
        if not row.any():
            row = whole
        sums = np.cumsum(row)
        u = float(uniform[i][0])
        part = 0 if math.isnan(u) else min(max(math.floor(u * 2.0 ** 31), 0), 2 ** 31 - 1) if math.isfinite(u) else (2 ** 31 - 1 if u > 0 else 0)
        target = int(sums[-1]) * part >> 31
        drawn = int(np.searchsorted(sums, target, side="right")) if sums[-1] else -1
        accepted[i] = len(path)
        paths[i, : len(path)] = path
        news[i, : len(path)] = [int(tokens[i][j]) for j in path[1:]] + [drawn]
    return accepted, paths, news
