"""Pins of the float64 operator definitions (oracle/operators.py) against
hand-computed values, scipy and brute force."""
import numpy as np
from scipy.special import logsumexp, softmax

import oracle


def test_row_paths():
    assert oracle.row_paths(4) == [[], [1], [1, 2], [1, 2, 3]]
    assert oracle.row_paths(5, [-1, 0, 0, 1, 3]) == [[], [1], [2], [1, 3], [1, 3, 4]]


def test_adjust_by_hand():
    x = np.array([[2.0, -1.0, 0.5, 3.0], [2.0, -1.0, 0.5, 3.0]])
    y, _ = oracle.adjust_logits(x, tokens=[1], history=[0, 3, 3], prompt_len=1, repetition=2.0, presence=0.25,
                                frequency=0.5, bias=[(2, 9.0), (2, 1.0)])
    # row 0: token 0 only in the prompt, 3 twice in the output, 2 biased (last entry)
    np.testing.assert_allclose(y[0], [1.0, -1.0, 1.5, 3.0 / 2 - 1.0 - 0.25])
    # row 1 follows draft token 1
    np.testing.assert_allclose(y[1], [1.0, -2.0 - 0.5 - 0.25, 1.5, 0.25])


def test_adjust_mask_and_out_of_range_tokens():
    x = np.array([[1.0, np.nan, -np.inf]])
    y, _ = oracle.adjust_logits(x, history=[-1, 7, 2], repetition=1.5, frequency=1.0, bias=[(-3, 4.0), (9, 4.0)],
                                allowed=np.array([[True, False, True]]))
    assert y[0, 0] == 1.0 and y[0, 1] == -np.inf and y[0, 2] == -np.inf


def test_adjust_counts_by_brute_force(np_rng):
    V, parent = 11, [-1, 0, 0, 1, 1, 4]
    tok, hist = np_rng.integers(0, V, 6), np_rng.integers(0, V, 40)
    y, _ = oracle.adjust_logits(np.zeros((6, V)), tokens=tok, parent=parent, history=hist, frequency=1.0)
    chain = {0: [], 1: [1], 2: [2], 3: [1, 3], 4: [1, 4], 5: [1, 4, 5]}
    for v, path in chain.items():
        for t in range(V):
            assert -y[v, t] == list(hist).count(t) + [int(tok[w]) for w in path].count(t)


def test_lmhead_quant_by_hand():
    # K = 4, G = 2: bytes 0x91 -> q 1, 9; 0x0F -> q 15, 0
    out, _ = oracle.lmhead_quant([[1.0, 2.0, 3.0, 4.0]], [[0x91, 0x0F]], [[0.5, 2.0]])
    assert out[0, 0] == 0.5 * (1 * -7 + 2 * 1) + 2.0 * (3 * 7 + 4 * -8)
    out, _ = oracle.lmhead_quant([[1.0, 2.0, 3.0, 4.0]], [[0x91, 0x0F]], [[0.5, 2.0]], [[1, 15]])
    assert out[0, 0] == 0.5 * (0 + 2 * 8) + 2.0 * (0 + 4 * -15)


def test_attention_against_scipy(np_rng):
    R, Hq, Hkv, D, P, L = 4, 4, 2, 3, 5, 6
    q, k, v = np_rng.normal(size=(R, Hq, D)), np_rng.normal(size=(L + R, Hkv, D)), np_rng.normal(size=(L + R, Hkv, D))
    pk, pv = np_rng.normal(size=(P, Hkv, D)), np_rng.normal(size=(P, Hkv, D))
    parent = [-1, 0, 0, 2]
    sees = {0: [0], 1: [0, 1], 2: [0, 2], 3: [0, 2, 3]}
    out, lse = oracle.attention(q, k, v, L, prefix_k=pk, prefix_v=pv, parent=parent, scale=0.7)
    for r in range(R):
        mask = np.array([True] * (P + L) + [j in sees[r] for j in range(R)])
        for h in range(Hq):
            kk, vv = np.concatenate([pk, k])[:, h // 2], np.concatenate([pv, v])[:, h // 2]
            s = np.where(mask, kk @ q[r, h] * 0.7, -np.inf)
            np.testing.assert_allclose(out[r, h], softmax(s) @ vv, rtol=1e-12)
            np.testing.assert_allclose(lse[r, h], logsumexp(s), rtol=1e-12)
    # a window is the chain
    a = oracle.attention(q, k, v, L, scale=0.7)
    b = oracle.attention(q, k, v, L, parent=[-1, 0, 1, 2], scale=0.7)
    np.testing.assert_array_equal(a[0], b[0])
