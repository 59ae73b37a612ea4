"""Float64 definitions of the paged cache of a verification step: rotary
positions, 8-bit numbers, appending to pages and keeping an accepted path.

Plain loops over sequences, rows and blocks, written from the formulas.  Pins:
tests/test_oracle_cache.py (complex rotations, the 8-bit numbers listed one by
one, hand-computed scales, moves by a dictionary of tokens).
"""
import math

import numpy as np

F8_MAX = 448.0
LEAST_SCALE = 2.0 ** -100


def depths(R, parent=None):
    """Depth of each row: its index in a window, its distance from the root in a tree."""
    d = []
    for r in range(R):
        d.append(r if parent is None else 0 if r == 0 else d[parent[r]] + 1)
    return d


def rotate(x, pos, inv_freq, *, interleaved=False, magnitude=1.0, inverse=False):
    """Rows x (R, H, D) at positions pos (R,), the first 2 len(inv_freq) values turned."""
    x = np.asarray(x, dtype=np.float64)
    y, n = x.copy(), len(inv_freq)
    for r in range(x.shape[0]):
        for i, f in enumerate(inv_freq):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
            t = math.fmod(float(pos[r]) * f, 2 * math.pi) * (-1 if inverse else 1)
            c, s = magnitude * math.cos(t), magnitude * math.sin(t)
            y[r, :, a] = x[r, :, a] * c - x[r, :, b] * s
            y[r, :, b] = x[r, :, b] * c + x[r, :, a] * s
    return y


def f8_numbers():
    """The finite non-negative 8-bit numbers in ascending order (their index is their byte)."""
    return np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127])


def f8_decode(byte):
    """Values of bytes (uint8): sign, 4 exponent bits, 3 fraction bits."""
    byte = np.asarray(byte, dtype=np.uint8)
    table = np.append(f8_numbers(), np.nan)
    return np.where(byte >> 7, -1.0, 1.0) * table[byte & 127]


def f8_round(x):
    """The nearest 8-bit numbers of |x| <= 448 (ties to the even byte); what is not finite becomes NaN."""
    x = np.asarray(x, dtype=np.float64)
    table = f8_numbers()
    with np.errstate(invalid="ignore"):
        a = np.where(np.isfinite(x), np.abs(x), 0.0)
    hi = np.clip(np.searchsorted(table, a), 1, len(table) - 1)  # table[hi - 1] < a <= table[hi], or the ends
    lo = hi - 1
    up = (a - table[lo] > table[hi] - a) | ((a - table[lo] == table[hi] - a) & (hi % 2 == 0))
    out = np.copysign(table[np.where(up, hi, lo)], x)
    return np.where(np.isfinite(x), out, np.nan)


def block_scale(a, before=None):
    """(scale, growth) of a block whose new rows reach magnitude a: the least
    before * 2^j, j >= 0, with a <= 448 of it (before: the earlier tokens' scale;
    none, or one that is no positive finite number: 2^-100)."""
    if before is None or not (0 < before < math.inf):
        before = LEAST_SCALE
    j = 0
    while a > F8_MAX * before * 2.0 ** j:
        j += 1
    return before * 2.0 ** j, j


def store(pages, scales, table, rows, first, *, page, block):
    """Rows (N, H, D) float64 to tokens first .. of a sequence, in place.  pages
    (num_pages, page, H, D) and scales (num_pages, page / block, H) float64;
    scales None: 16-bit pages, stored as they are.  Rows of pages outside
    [0, num_pages) are left out."""
    at = first
    while at < first + len(rows):
        end = min(first + len(rows), (at // block + 1) * block)
        home, t0 = int(table[at // page]), at % page
        part = rows[at - first:end - first]
        if 0 <= home < len(pages):
            if scales is None:
                pages[home, t0:t0 + end - at] = part
            else:
                start = t0 // block * block
                for h in range(pages.shape[2]):
                    mine = np.abs(part[:, h])
                    mine = mine[np.isfinite(mine)]
                    before = scales[home, t0 // block, h]
                    earlier = t0 > start and 0 < before < math.inf
                    s, grown = block_scale(mine.max() if mine.size else 0.0, before if earlier else None)
                    if earlier and grown:
                        pages[home, start:t0, h] = f8_round(pages[home, start:t0, h] / 2.0 ** grown)
                    scales[home, t0 // block, h] = s
                    pages[home, t0:t0 + end - at, h] = f8_round(part[:, h] / s)
        at = end


def commit(pages, scales, table, length, nodes, n_accepted, R, *, page, block):
    """Moves a path's rows (nodes, tokens length + node) to tokens length + 1 ..,
    in place, and returns the new length.  A path has at most R - 1 nodes.  8-bit
    rows times their scales are float32 numbers.  Rows from pages outside are left out."""
    path = []
    for w in list(nodes)[:min(max(0, n_accepted), R - 1)]:
        if not 1 <= w < R:
            break
        path.append(int(w))
    rows = []
    for w in path:
        home, t = int(table[(length + w) // page]), (length + w) % page
        assert 0 <= home < len(pages)
        row = pages[home, t].copy()
        rows.append(row if scales is None else (row * scales[home, t // block][:, None]).astype(np.float32).astype(np.float64))
    if rows:
        store(pages, scales, table, np.stack(rows), length + 1, page=page, block=block)
    return length + 1 + len(path)


def gather(pages, scales, table, tokens, *, page, block):
    """The first `tokens` tokens (tokens, H, D) of a page table, as values."""
    out = []
    for t in range(tokens):
        home = int(table[t // page])
        row = pages[home, t % page]
        out.append(row if scales is None else row * scales[home, t % page // block][:, None])
    return np.stack(out) if out else np.zeros((0, *pages.shape[2:]))
