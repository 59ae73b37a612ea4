"""Float64 definitions of the operators around a verification step: the logits
adjustment, the group-quantised LM head and the attention of draft rows.

Plain loops over sequences and rows, written from the formulas.  Pins:
tests/test_oracle_operators.py (hand-computed values, scipy's softmax and
logsumexp, brute-force counting).
"""
import numpy as np


def row_paths(R, parent=None):
    """Nodes of each row's path, the root left out: rows 1..i of a window's row
    i, or the tree nodes from the root's child down to node v."""
    paths = []
    for v in range(R):
        path, w = [], v
        while w > 0:
            path.append(w)
            w = parent[w] if parent is not None else w - 1
        paths.append(path[::-1])
    return paths


def adjust_logits(x, *, tokens=None, parent=None, history=(), prompt_len=0, repetition=1.0, presence=0.0,
                  frequency=0.0, bias=(), allowed=None):
    """Adjusted rows of one sequence.  x (R, V) float64; tokens: the drafts (R -
    1 of a window, R of a tree); history: the tokens so far; bias: (token,
    value) pairs; allowed: (R, V) booleans.  Returns (y, magnitude), magnitude
    being the sum of the intermediates' sizes (for rounding bounds)."""
    x = np.asarray(x, dtype=np.float64)
    R, V = x.shape
    y, size = x.copy(), np.abs(x)
    said, told = np.zeros(V), np.zeros(V, dtype=bool)
    for i, t in enumerate(history):
        if 0 <= t < V:
            if i < prompt_len:
                told[t] = True
            else:
                said[t] += 1
    add = {}
    for t, v in bias:
        if 0 <= t < V:
            add[t] = v
    with np.errstate(invalid="ignore"):
        for r, path in enumerate(row_paths(R, parent)):
            n = said.copy()
            for w in path if tokens is not None else ():
                t = tokens[w] if parent is not None else tokens[w - 1]
                if 0 <= t < V:
                    n[t] += 1
            seen = told | (n > 0)
            y[r, seen] = np.where(y[r, seen] > 0, y[r, seen] / repetition, y[r, seen] * repetition)
            size[r] += np.abs(y[r])
            hit = n > 0
            y[r, hit] -= frequency * n[hit]
            size[r, hit] += np.abs(frequency * n[hit]) + np.abs(y[r, hit])
            y[r, hit] -= presence
            size[r, hit] += np.abs(y[r, hit])
            for t, v in add.items():
                y[r, t] += v
                size[r, t] += np.abs(y[r, t])
            if allowed is not None:
                y[r, ~allowed[r]] = -np.inf
    return y, size


def lmhead_quant(h, wq, scales, zeros=None):
    """Logits of hidden rows h (M, K) on 4-bit weights: wq (V, K / 2) bytes, the
    even k in the low half; weight (v, k) = scales[v][k // G] * (q - zeros[v][k
    // G]), zeros 8 when None.  Returns (logits, magnitude): magnitude sums
    |h| * scale * (24 + |q - zero|) per logit."""
    wq = np.asarray(wq, dtype=np.uint8)
    h, scales = np.asarray(h, dtype=np.float64), np.asarray(scales, dtype=np.float64)
    V, K = wq.shape[0], 2 * wq.shape[1]
    q = np.empty((V, K))
    q[:, 0::2], q[:, 1::2] = wq & 15, wq >> 4
    G = K // scales.shape[1]
    z = np.full(scales.shape, 8.0) if zeros is None else np.asarray(zeros, dtype=np.float64)
    w = (q - np.repeat(z, G, 1)) * np.repeat(scales, G, 1)
    size = (np.abs(q - np.repeat(z, G, 1)) + 24) * np.abs(np.repeat(scales, G, 1))
    return h @ w.T, np.abs(h) @ size.T


def attention(q, k, v, length, *, prefix_k=None, prefix_v=None, parent=None, scale=1.0):
    """Attention of one sequence's rows: q (R, Hq, D); k, v (cap, Hkv, D) with
    `length` committed keys followed by the rows' own; prefix_k, prefix_v (P,
    Hkv, D).  Row r sees the prefix, the committed keys and the keys of its
    ancestors and itself (of rows 0..r without parent).  Returns (out, lse)."""
    q, k, v = (np.asarray(a, dtype=np.float64) for a in (q, k, v))
    R, Hq, D = q.shape
    Hkv = k.shape[1]
    paths = row_paths(R, parent)
    out, lse = np.zeros((R, Hq, D)), np.zeros((R, Hq))
    for r in range(R):
        at = list(range(length)) + [length + w for w in [0] + paths[r]]
        kk, vv = k[at], v[at]
        if prefix_k is not None:
            kk = np.concatenate([np.asarray(prefix_k, dtype=np.float64), kk])
            vv = np.concatenate([np.asarray(prefix_v, dtype=np.float64), vv])
        for h in range(Hq):
            s = kk[:, h // (Hq // Hkv)] @ q[r, h] * scale
            top = s.max()
            e = np.exp(s - top)
            out[r, h] = e @ vv[:, h // (Hq // Hkv)] / e.sum()
            lse[r, h] = top + np.log(e.sum())
    return out, lse
