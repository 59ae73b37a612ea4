"""Pins of the paged cache's float64 definitions (oracle/cache.py)."""
import math

import numpy as np
import pytest

from oracle import cache as oc


def test_rotation_is_a_complex_product(np_rng):
    x = np_rng.standard_normal((5, 3, 16))
    f = [1.0, 0.3, 0.01]
    pos = np.array([0, 1, 7, 100, -3])
    turn = np.exp(1j * pos[:, None, None] * np.array(f)) * 1.5
    y = oc.rotate(x, pos, f, magnitude=1.5)
    z = (x[..., 0:3] + 1j * x[..., 3:6]) * turn
    assert np.allclose(y[..., 0:3], z.real) and np.allclose(y[..., 3:6], z.imag) and (y[..., 6:] == x[..., 6:]).all()
    y = oc.rotate(x, pos, f, interleaved=True)
    z = (x[..., 0:6:2] + 1j * x[..., 1:6:2]) * turn / 1.5
    assert np.allclose(y[..., 0:6:2], z.real) and np.allclose(y[..., 1:6:2], z.imag)
    assert np.allclose(oc.rotate(y, pos, f, interleaved=True, inverse=True), x)


def test_the_8bit_numbers():
    n = oc.f8_numbers()
    assert len(n) == 127 and n[0] == 0 and n[1] == 2.0 ** -9 and n[8] == 2.0 ** -6 and n[56] == 1 and n[126] == 448
    assert (np.diff(n) > 0).all()
    torch = pytest.importorskip("torch")
    byte = torch.arange(256, dtype=torch.uint8)
    want = byte.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oc.f8_decode(byte.numpy()), want, equal_nan=True)


def test_rounding_to_8_bits(np_rng):
    torch = pytest.importorskip("torch")
    n = oc.f8_numbers()
    x = np.concatenate([n, (n[1:] + n[:-1]) / 2, np_rng.uniform(0, 448, 20000), np_rng.uniform(0, 2.0 ** -5, 20000)]).astype(np.float32)
    x = np.concatenate([x, -x]).astype(np.float64)
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oc.f8_round(x), want)
    assert np.isnan(oc.f8_round([np.inf, -np.inf, np.nan])).all()


@pytest.mark.parametrize("a,before,want", [
    (0.0, None, 2.0 ** -100), (448.0, None, 1.0), (np.nextafter(448.0, 500), None, 2.0), (7.0, None, 2.0 ** -6), (7.1, None, 2.0 ** -5),
    (1.0, 0.01, 0.01), (4.48, 0.01, 0.01), (4.5, 0.01, 0.02), (100.0, 0.01, 0.32), (1.0, 0.0, 2.0 ** -8), (1.0, math.inf, 2.0 ** -8),
    (1.0, math.nan, 2.0 ** -8), (1.0, -1.0, 2.0 ** -8)])
def test_scales(a, before, want):
    assert oc.block_scale(a, before)[0] == want


def test_store_and_gather(np_rng):
    pages, scales = np.full((4, 32, 2, 8), 3.0), np.full((4, 2, 2), 0.5)
    table = [2, 0, 9]
    rows = np_rng.standard_normal((30, 2, 8)) * 10
    oc.store(pages, scales, table, rows, 20, page=32, block=16)
    # token 20 is in the second block of page 2, which begins at 16: the earlier 4 keep the scale 0.5
    assert (pages[2, :20] == 3).all() and (scales[2] == 0.5).all() and (pages[1] == 3).all() and (pages[3] == 3).all()
    assert (pages[0, 18:] == 3).all() and (scales[0] != 0.5).all() and (np.log2(scales[0]) % 1 == 0).all()
    got = oc.gather(pages, scales, table, 50, page=32, block=16)
    assert (got[:20] == 1.5).all()
    assert np.abs(got[20:] - rows).max() <= 2.0 ** -4 * np.abs(rows).max() * 1.01
    # a row that outgrows the scale: the earlier ones are halved so often
    big = np.zeros((1, 2, 8))
    big[0, 1, 0] = 1000.0
    oc.store(pages, scales, table, big, 25, page=32, block=16)
    assert scales[2, 1, 0] == 0.5 and scales[2, 1, 1] == 4.0
    assert (pages[2, 16:20, 0] == 3).all() and (pages[2, 16:20, 1] == 0.375).all()
    oc.store(pages, scales, table, big, 64, page=32, block=16)  # page 9 is none
    with pytest.raises(IndexError):
        oc.gather(pages, scales, table, 65, page=32, block=16)


@pytest.mark.parametrize("eight", [False, True])
def test_commit_moves_the_path(np_rng, eight):
    R, length, page, block = 14, 27, 16, 16
    table = [3, 1, 0]
    pages = oc.f8_round(np_rng.uniform(-400, 400, (4, page, 2, 8)))
    scales = 2.0 ** np_rng.integers(-3, 3, (4, 1, 2)).astype(float) if eight else None
    value = lambda t: pages[table[t // page], t % page] * (scales[table[t // page], 0][:, None] if eight else 1)  # noqa: E731
    before = {t: value(t).copy() for t in range(48)}
    assert oc.commit(pages, scales, table, length, [2, 5, 11, -1], 3, R, page=page, block=block) == length + 4
    for i, w in enumerate([2, 5, 11]):
        # (a power of two between scales only matters for the smallest numbers)
        assert np.abs(value(length + 1 + i) - before[length + w]).max() <= (2.0 ** -4 if eight else 0)
    for t in range(length + 1):
        assert np.abs(value(t) - before[t]).max() <= (2.0 ** -4 if eight else 0)
    # a node outside the rows ends the path
    assert oc.commit(pages, scales, table, length, [1, 14, 2], 3, R, page=page, block=block) == length + 2
    assert oc.commit(pages, scales, table, length, [1], -5, R, page=page, block=block) == length + 1


@pytest.mark.parametrize("eight", [False, True])
def test_commit_stays_within_the_rows(np_rng, eight):
    """A path that names more nodes than a tree of R can have ends at the rows' own places, the last that the table has room for."""
    page, table = 16, [1, 3]
    for R, nodes, moved in ((2, [1, 1, 1, 1], 1), (4, [3, 2, 2, 1, 1, 3], 3), (1, [1, 1], 0)):
        pages = oc.f8_round(np_rng.uniform(-400, 400, (4, page, 2, 8)))
        scales = np.full((4, 1, 2), 0.5) if eight else None
        length = len(table) * page - R
        want = pages.copy()
        for i, w in enumerate(nodes[:moved]):
            want[3, length + 1 + i - page] = pages[3, length + w - page]
        assert oc.commit(pages, scales, table, length, nodes, len(nodes), R, page=page, block=page) == length + 1 + moved
        assert np.array_equal(pages, want)


def test_commit_by_other_scales_goes_through_float32():
    """3 bits' numbers times a scale of 24 bits, rounded to float32, over another scale."""
    pages, scales = np.zeros((2, 16, 1, 4)), np.array([[[np.float32(0.0123)]], [[np.float32(0.37)]]], dtype=np.float64)
    pages[0, 14, 0], pages[1, 1, 0] = 400.0, [448.0, 13.0, -0.0625, 0.001953125]
    assert oc.commit(pages, scales, [0, 1], 14, [3], 1, 4, page=16, block=16) == 16
    x = (np.array([448.0, 13.0, -0.0625, 0.001953125]).astype(np.float32) * np.float32(0.37)).astype(np.float64)
    s = float(np.float32(0.0123)) * 32             # the least with 165.76 <= 448 s
    assert scales[0, 0, 0] == s and np.array_equal(pages[0, 15, 0], oc.f8_round(x / s)) and (pages[0, 14, 0] == 12).all()
