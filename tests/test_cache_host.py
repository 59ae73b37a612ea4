"""Refusals of the paged cache's operators that need no device, and the host
side of the rotations."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

import draft_token_verification_06_amd as sv
from draft_token_verification_06_amd import _lib

FAKE = 0x100000  # never dereferenced: validation fails first
BF16, F16, F8 = 1, 2, 3


def _cache(**kw):
    a = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, dtype=F8, num_pages=100, page=64, block=32, Hkv=2, D=128,
             page_stride=0, token_stride=0, head_stride=0)
    a.update(kw)
    return _lib.PAGED_CACHE.pack(*(x or 0 for x in a.values()))


def _ints(xs):
    return None if xs is None else (ctypes.c_int32 * len(xs))(*xs)


BAD_CACHES = [
    (dict(dtype=0), -2),
    (dict(dtype=4), -2),
    (dict(dtype=F16), -2),                    # 16-bit pages hold the rows' type
    (dict(k=None), -1),
    (dict(v=None), -1),
    (dict(k=FAKE + 8), -1),
    (dict(k_scale=None), -1),
    (dict(v_scale=FAKE + 2), -1),
    (dict(num_pages=0), -1),
    (dict(Hkv=0), -1),
    (dict(Hkv=2000), -1),
    (dict(D=96), -1),
    (dict(page=8), -1),
    (dict(page=48), -1),
    (dict(page=512), -1),
    (dict(block=8), -1),
    (dict(block=24), -1),
    (dict(block=128, page=128), -1),
    (dict(block=64, page=32), -1),
    (dict(token_stride=64), -1),              # tokens overlap
    (dict(token_stride=132), -1),             # not a multiple of 16 bytes
    (dict(token_stride=-128), -1),
    (dict(token_stride=(1 << 24) + 16), -1),
    (dict(head_stride=8191 // 16 * 16), -1),  # heads overlap
    (dict(page_stride=16000), -1),            # pages overlap
    (dict(token_stride=256, head_stride=192, page_stride=1 << 20), -1),
]


def _append(cache=None, **kw):
    a = dict(cache=_cache() if cache is None else cache, table=FAKE, table_stride=0, table_pages=10, ctx_len=FAKE, row_count=None,
             parent=None, base_pos=None, k=FAKE, k_stride=0, v=FAKE, v_stride=0, q=FAKE, q_stride=0, q_out=FAKE + (1 << 30),
             q_out_stride=0, dtype=BF16, turns=FAKE, rot=128, interleaved=0, magnitude=1.0, B=2, R=5, Hq=4)
    a.update(kw)
    a["parent"] = _ints(a["parent"])
    return _lib.lib().sv_cache_append(*a.values(), None)


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_append_refuses_caches(kw, status):
    assert _append(_cache(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=0), -2),
    (dict(dtype=F8), -2),
    (dict(table=None), -1),
    (dict(table_pages=0), -1),
    (dict(table_pages=1 << 25), -1),          # more than 2^30 tokens
    (dict(table_stride=9), -1),
    (dict(ctx_len=None), -1),
    (dict(B=0), -1),
    (dict(R=0), -1),
    (dict(R=(1 << 24) + 1), -1),
    (dict(B=1 << 24, R=1 << 20), -1),         # the grid
    (dict(parent=[-1, 0, 1, 4, 0]), -4),
    (dict(parent=[0, 0, 1, 1, 0]), -4),
    (dict(base_pos=FAKE + 4), -1),
    (dict(k=None), -1),
    (dict(k=FAKE + 2), -1),
    (dict(v=None), -1),
    (dict(k_stride=248), -1),
    (dict(v_stride=260), -1),                 # not a multiple of 16 bytes
    (dict(q=None), -1),
    (dict(q_out=None), -1),
    (dict(q_stride=504), -1),
    (dict(q_out=FAKE + 512), -1),             # overlaps q
    (dict(q_out=FAKE, q_out_stride=1024), -1),  # in place with another stride
    (dict(Hq=0), -1),                         # queries without heads
    (dict(Hq=-1), -1),
    (dict(Hq=2000), -1),
    (dict(rot=0), -1),
    (dict(rot=24), -1),
    (dict(rot=144), -1),
    (dict(turns=None), -1),                   # rot without frequencies
    (dict(turns=FAKE + 4), -1),
    (dict(magnitude=float("inf")), -1),
    (dict(magnitude=float("nan")), -1),
])
def test_append_status(kw, status):
    assert _append(**kw) == status


def _attend(cache=None, **kw):
    a = dict(q=FAKE, q_stride=0, dtype=BF16, cache=_cache() if cache is None else cache, table=FAKE, table_stride=0, table_pages=10,
             prefix_table=FAKE, P=10, ctx_len=FAKE, row_count=None, parent=None, B=2, R=5, Hq=8, max_ctx=635, scale=0.1,
             out=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    a["parent"] = _ints(a["parent"])
    return _lib.lib().sv_paged_attention(*a.values(), None)


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_attention_refuses_caches(kw, status):
    assert _attend(_cache(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=0), -2),
    (dict(dtype=F8), -2),
    (dict(B=0), -1),
    (dict(R=0), -1),
    (dict(R=66, max_ctx=100), -1),
    (dict(Hq=9), -1),
    (dict(Hq=0), -1),
    (dict(P=-1), -1),
    (dict(P=0), -1),                          # a prefix table without a prefix
    (dict(prefix_table=None), -1),
    (dict(P=(1 << 24) + 1), -1),
    (dict(max_ctx=-1), -1),
    (dict(max_ctx=636), -1),                  # max_ctx + R past the table
    (dict(table=None), -1),
    (dict(table_pages=0), -1),
    (dict(table_stride=9), -1),
    (dict(ctx_len=None), -1),
    (dict(q=None), -1),
    (dict(q=FAKE + 8), -1),
    (dict(q_stride=1016), -1),
    (dict(q_stride=1028), -1),
    (dict(out=None), -1),
    (dict(out=FAKE + 8), -1),
    (dict(lse=FAKE + 2), -1),
    (dict(scale=float("nan")), -1),
    (dict(scale=float("-inf")), -1),
    (dict(parent=[-1, 0, 1, 4, 0]), -4),
    (dict(ws=None), -3),
    (dict(ws=FAKE + 16), -3),
    (dict(ws_bytes=256), -3),
])
def test_attention_status(kw, status):
    assert _attend(**kw) == status


def _commit(cache=None, **kw):
    a = dict(cache=_cache() if cache is None else cache, layers=3, layer_stride=0, table=FAKE, table_stride=0, table_pages=10, ctx_len=FAKE,
             nodes=FAKE, nodes_stride=0, max_nodes=3, n_accepted=FAKE, B=2, R=5, new_len=FAKE + 64)
    a.update(kw)
    return _lib.lib().sv_cache_commit(*a.values(), None)


@pytest.mark.parametrize("kw,status", [c for c in BAD_CACHES if c[0] != dict(dtype=F16)])
def test_commit_refuses_caches(kw, status):
    assert _commit(_cache(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(layers=0), -1),
    (dict(layers=1 << 16), -1),
    (dict(layer_stride=100 * 2 * 64 * 128 - 16), -1),  # layers overlap
    (dict(layer_stride=100 * 2 * 64 * 128 + 8), -1),
    (dict(layer_stride=-16), -1),
    (dict(table=None), -1),
    (dict(table_pages=0), -1),
    (dict(table_stride=9), -1),
    (dict(ctx_len=None), -1),
    (dict(n_accepted=None), -1),
    (dict(nodes=None), -1),                   # nodes counted but not given
    (dict(max_nodes=0), -1),
    (dict(max_nodes=65), -1),
    (dict(nodes_stride=2), -1),
    (dict(nodes=None, max_nodes=0, new_len=None), -1),  # nothing to do
    (dict(new_len=FAKE + 4), -1),             # overlaps ctx_len without being it
    (dict(B=0), -1),
    (dict(R=0), -1),
    (dict(B=1 << 25), -1),                    # the grid
])
def test_commit_status(kw, status):
    assert _commit(**kw) == status


def _rotary(**kw):
    a = dict(x=FAKE, x_stride=0, out=FAKE, out_stride=0, dtype=BF16, turns=FAKE, rot=32, interleaved=0, inverse=0, magnitude=1.0,
             base_pos=FAKE, row_count=None, parent=None, B=2, R=5, H=4, D=80)
    a.update(kw)
    a["parent"] = _ints(a["parent"])
    return _lib.lib().sv_rotary(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=F8), -2),
    (dict(dtype=-1), -2),
    (dict(x=None), -1),
    (dict(out=None), -1),
    (dict(x=FAKE + 8), -1),
    (dict(turns=None), -1),
    (dict(turns=FAKE + 4), -1),
    (dict(rot=0), -1),
    (dict(rot=41), -1),
    (dict(rot=96), -1),
    (dict(D=72), -1),
    (dict(D=528), -1),
    (dict(D=0), -1),
    (dict(H=0), -1),
    (dict(H=1025), -1),
    (dict(B=0), -1),
    (dict(R=0), -1),
    (dict(B=1 << 30, R=1 << 10), -1),
    (dict(base_pos=FAKE + 4), -1),
    (dict(magnitude=float("nan")), -1),
    (dict(x_stride=312), -1),
    (dict(x_stride=324, out_stride=324), -1),
    (dict(out_stride=400), -1),               # in place with another stride
    (dict(out=FAKE + 160), -1),               # overlaps x
    (dict(parent=[-1, 0, 1, 4, 0]), -4),
])
def test_rotary_status(kw, status):
    assert _rotary(**kw) == status


def test_turns():
    f = [1.0, 1e-4, 0.5, 7.0, -0.25, 0.0, 1e300]
    n = len(f)
    out = (ctypes.c_uint64 * n)()
    assert _lib.lib().sv_rotary_turns((ctypes.c_double * n)(*f), n, out) == 0
    for x, got in zip(f[:-1], out):
        want = Fraction(x / (2 * math.pi)) % 1 * 2 ** 64
        assert abs(int(got) - want) <= max(1, abs(Fraction(x / (2 * math.pi))) * 2 ** 64 * Fraction(1, 2 ** 52)) or x < 0
    assert (1 << 64) - int(out[4]) == int(Fraction(0.25 / (2 * math.pi)) * 2 ** 64)
    for bad in (math.inf, math.nan):
        assert _lib.lib().sv_rotary_turns((ctypes.c_double * 1)(bad), 1, out) == -1
    assert _lib.lib().sv_rotary_turns(None, 1, out) == -1
    assert _lib.lib().sv_rotary_turns((ctypes.c_double * 1)(1.0), 0, out) == -1
    t = sv.rotary_turns([math.pi, 1.0], "cpu")
    assert t.dtype == torch.int64 and t.tolist()[0] == -(1 << 63)


def test_frequencies():
    f, m = sv.rotary_frequencies(64)
    assert m == 1.0 and f[0] == 1.0 and len(f) == 32 and f[16] == pytest.approx(0.01)
    g, m = sv.rotary_frequencies(64, scaling="linear", factor=4.0)
    assert m == 1.0 and g == pytest.approx([x / 4 for x in f])
    g, m = sv.rotary_frequencies(64, scaling="base", factor=4.0)
    assert m == 1.0 and g[0] == 1.0 and g[-1] == pytest.approx(f[-1] / 4)
    g, m = sv.rotary_frequencies(64, scaling="ramp", factor=4.0, trained=4096)
    turns = [4096 * x / (2 * math.pi) for x in f]
    assert m == pytest.approx(0.1 * math.log(4.0) + 1)
    for x, y, t in zip(f, g, turns):
        assert y == pytest.approx(x if t >= 32 else x / 4 if t <= 1 else x * (t - 1) / 31 + x / 4 * (1 - (t - 1) / 31))
    for kw in (dict(rot=3), dict(rot=0), dict(rot=8, base=0.0), dict(rot=8, factor=0.0), dict(rot=8, scaling="other"),
               dict(rot=8, scaling="ramp", fast=1.0)):
        with pytest.raises(ValueError):
            sv.rotary_frequencies(**kw)


def test_binding_refuses():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    n, table = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        sv.PagedCache(k, k)                   # host memory
    with pytest.raises(ValueError):
        sv.PagedCache(k.float(), k.float())
    with pytest.raises(ValueError):
        sv.rotary(k, n.long(), n.long())
    with pytest.raises(ValueError):
        sv.cache_append(None, table, n, k[:1], k[:1])
    with pytest.raises(ValueError):
        sv.paged_attention(k[:1], None, table, n)
    with pytest.raises(ValueError):
        sv.paged_attention_workspace(0, 1, 1, 1, 64, 0, 0, "cpu")


@pytest.mark.parametrize("at,status", [(0, -1), (4, -1), (-4, -1)])
def test_commit_refuses_lengths_over_the_counts(at, status):
    """new_len is written while n_accepted is still read."""
    other = FAKE + (1 << 20)
    assert _commit(n_accepted=other, new_len=other + at) == status


class _Pages:
    """What PagedCache looks at of a device tensor."""
    def __init__(self, shape, stride, dtype=torch.bfloat16):
        self.shape, self._stride, self.dtype, self.device = torch.Size(shape), stride, dtype, torch.device("cuda", 0)

    def stride(self):
        return self._stride

    def data_ptr(self):
        return FAKE


@pytest.mark.parametrize("shape,stride", [
    ((1000, 16, 2, 64), (0, 128, 64, 1)),       # one page for all
    ((10, 16, 2, 64), (2048, 0, 64, 1)),        # one token for all
    ((1, 16, 1, 64), (1024, 0, 64, 1)),
    ((10, 16, 8, 64), (1024, 64, 0, 1)),        # one head for all
    ((3, 1000, 16, 2, 64), (2048, 0, 128, 64, 1)),
    ((3, 10, 16, 8, 64), (10240, 1024, 64, 0, 1)),
    ((3, 10, 16, 2, 64), (0, 2048, 128, 64, 1)),   # one layer for all
])
def test_expanded_pages_are_refused(shape, stride):
    """A stride of zero is no order of pages: the library would take it for a dense one and go past the storage."""
    with pytest.raises(ValueError):
        sv.PagedCache(_Pages(shape, stride), _Pages(shape, stride))


def test_strides_of_single_entries_do_not_matter():
    c = sv.PagedCache(_Pages((1, 16, 1, 64), (0, 64, 0, 1)), _Pages((1, 16, 1, 64), (0, 64, 0, 1)))
    assert _lib.PAGED_CACHE.unpack(c.args) == (FAKE, FAKE, 0, 0, BF16, 1, 16, 0, 1, 64, 0, 64, 0)


@pytest.mark.parametrize("at,wide", [(8, 320), (312, 640), (328 + 640, 640), (-8, 960), (640 * 3 + 312, 640), (960 - 312, 960), (320, 639 // 8 * 8)])
def test_rotary_refuses_parts_that_meet(at, wide):
    """Two parts of rows `wide` apart, each 320 long: out begins `at` elements behind x."""
    assert _rotary(x=FAKE + 4096, x_stride=wide, out=FAKE + 4096 + 2 * at, out_stride=wide) == -1


@pytest.mark.parametrize("kw", [
    dict(k=FAKE + (1 << 30)), dict(v=FAKE + (1 << 30) + 1024), dict(k=FAKE + (1 << 30) - 16), dict(v=FAKE + (1 << 30) + 10 * 1024 - 16),
    # one projection's rows of 4 + 2 + 2 heads of 128: the queries to the place of keys and values
    dict(q_out=FAKE + 1024, k=FAKE + 1024, v=FAKE + 1536, q_stride=1024, q_out_stride=1024, k_stride=1024, v_stride=1024),
    dict(q_out=FAKE, k=FAKE + 1024, v=FAKE + 512, q_stride=1024, q_out_stride=1024, k_stride=1024, v_stride=1024),
])
def test_append_refuses_queries_over_keys_and_values(kw):
    """q_out is written while k and v are still read."""
    assert _append(**kw) == -1
