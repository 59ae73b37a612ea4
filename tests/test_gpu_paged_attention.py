"""Attention over paged caches on the GPU against the float64 definition on the
values that the pages stand for.

Tolerance.  As for the attention of contiguous caches (N keys, h half a step of
the storage type, A the largest scale * sum |q k| of a row), with one more
rounding for each scale: keys' after the product, values' on the exponentials.
Those and the few of the statistics are within the 16 of
  |out - exact| <= (h + 2 (D + N + 16) 2^-24 (1 + A)) (sum p |v| / sum p) + h |out|
  |lse - exact| <= 2 (D + N + 16) 2^-24 (1 + A) + 2^-23 |lse|.
float16 outputs may be subnormal (half of 2^-24), and exponentials in float16 are
held 2^15 times larger, relative to the largest value scale: those below
2^-29 of it lose up to 2^-40 of it each, N 2^-40 max |v| together."""
import numpy as np
import pytest
import torch

import draft_token_verification_06_amd as sv
import oracle
from draft_token_verification_06_amd import synth
from oracle import cache as oc

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
F8 = torch.float8_e4m3fn


def host(t):
    return (t.float() if t.dtype == F8 else t).double().cpu().numpy()


def make(B, R, Hq, Hkv, D, P, tokens, dtype, held, page, block, seed, *, token_major=False, spread=3, pow2=True):
    """Queries, a cache, page tables for `tokens` tokens and a prefix of P; pages in a random order."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    each, before = (tokens + page - 1) // page, (P + page - 1) // page
    num = B * each + before + 2
    ids = torch.randperm(num, generator=g, device=DEV).to(torch.int32)
    table, prefix = ids[:B * each].view(B, each).contiguous(), ids[B * each:B * each + before].contiguous()
    shape = (num, page, Hkv, D) if token_major else (num, Hkv, page, D)
    made = []
    for _ in range(2):
        x = torch.randn(shape, generator=g, device=DEV)
        x = (x * 100).clamp(-448, 448).to(F8) if held == "f8" else x.to(DT[dtype])
        made.append(x if token_major else x.transpose(1, 2))
    if held == "f8":
        for _ in range(2):
            e = torch.randint(-7 - spread, -6 + spread, (num, page // block, Hkv), generator=g, device=DEV).double()
            made.append((torch.exp2(e) if pow2 else torch.exp2(e + torch.rand(e.shape, generator=g, device=DEV, dtype=torch.float64))).float())
    q = (torch.randn(B, R, Hq, D, generator=g, device=DEV) * 2).to(DT[dtype])
    return q, sv.PagedCache(*made), table, prefix


def dense(cache, table, tokens):
    """(keys, values) of the first tokens of a page table as float64 values."""
    page = cache.k.shape[1]
    n = (tokens + page - 1) // page
    home = table[:n].long()
    out = []
    for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x = host((t.view(torch.uint8)[home].view(F8) if t.dtype == F8 else t[home]))
        if s is not None:
            x = x * np.repeat(host(s[home]), page // s.shape[1], axis=1)[..., None]
        out.append(x.reshape(-1, *x.shape[2:])[:tokens])
    return out


def check(res, q, cache, table, lens, *, prefix=None, P=0, parent=None, scale=None, row_count=None):
    B, R, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    h = HALF_STEP[q.dtype]
    pk, pv = dense(cache, prefix, P) if P else (None, None)
    for b in range(B):
        n, rows = int(lens[b]), R if row_count is None else min(max(int(row_count[b]), 0), R)
        if rows == 0:
            continue
        par = None if parent is None else parent[:rows]
        kb, vb = dense(cache, table[b], n + rows)
        kw = dict(parent=par, scale=scale)
        qb = host(q[b, :rows])
        out, lse = oracle.attention(qb, kb, vb, n, prefix_k=pk, prefix_v=pv, **kw)
        with np.errstate(invalid="ignore"):
            weight, _ = oracle.attention(qb, kb, np.abs(vb), n, prefix_k=pk, prefix_v=None if pv is None else np.abs(pv), **kw)
        keys, values = (kb, vb) if pk is None else (np.concatenate([pk, kb]), np.concatenate([pv, vb]))
        N = len(keys)
        grp = np.repeat(np.abs(keys), Hq // kb.shape[1], axis=1)
        A = abs(scale) * np.nanmax(np.einsum("rhd,khd->rhk", np.abs(qb), np.nan_to_num(grp, posinf=0)), axis=2)
        rel = 2 * (D + N + 16) * 2.0 ** -24 * (1 + A)
        got, glse = host(res.out[b, :rows]), None if res.lse is None else host(res.lse[b, :rows])
        fine = np.isfinite(out)
        assert np.array_equal(np.isfinite(got), fine), "finite values in other places"
        with np.errstate(invalid="ignore"):
            tol = (h + rel[..., None]) * weight * (1 + 2.0 ** -6) + h * np.abs(out) + 2.0 ** -24
            if q.dtype == torch.float16:
                tol = tol + N * 2.0 ** -40 * np.abs(np.nan_to_num(values, posinf=0, neginf=0)).max()
            err = np.abs(got - out)
        assert (err[fine] <= tol[fine]).all(), (b, float((err[fine] / tol[fine]).max()))
        if glse is not None:
            assert (np.abs(glse - lse) <= rel + 2.0 ** -23 * np.abs(lse)).all(), float(np.abs(glse - lse).max())


CASES = [
    # B, R, parent, Hq, Hkv, D, P, lens, dtype, held, page, block
    (1, 1, None, 1, 1, 64, 0, [0], "bf16", "f8", 16, 16),          # one key: the row itself
    (1, 1, None, 8, 1, 128, 1, [1], "f16", "f8", 16, 16),
    (2, 1, None, 32, 8, 128, 333, [700, 0], "bf16", "f8", 64, 64),
    (3, 9, None, 8, 2, 128, 0, [127, 128, 129], "bf16", "f8", 32, 16),
    (3, 9, None, 8, 2, 64, 127, [255, 250, 1], "f16", "f8", 128, 64),
    (2, 5, None, 7, 1, 64, 257, [64, 65], "bf16", "f8", 16, 16),   # 35 stacked rows of 7 heads
    (2, 17, None, 16, 4, 128, 640, [31, 900], "f16", "f8", 64, 32),   # 68 stacked rows
    (1, 41, "432", 4, 4, 64, 0, [983], "f16", "f8", 256, 32),
    (2, 41, "432", 8, 2, 128, 100, [100, 300], "bf16", "f8", 32, 32),
    (1, 65, None, 2, 2, 64, 10, [200], "bf16", "f8", 64, 16),
    (1, 256, "star", 2, 1, 64, 33, [50], "bf16", "f8", 16, 16),
    (1, 256, "pairs", 2, 2, 128, 0, [301], "f16", "f8", 32, 16),
    (40, 4, None, 4, 1, 128, 1500, list(range(40)), "bf16", "f8", 64, 64),
    (2, 2, None, 6, 3, 128, 5, [2500, 1], "bf16", "f8", 16, 16),   # several look-ups of 1024 tokens
    (1, 1, None, 4, 2, 128, 0, [9000], "f16", "f8", 32, 32),
    (1, 4, None, 16, 1, 64, 3000, [40], "f16", "f8", 256, 64),
    (2, 1, None, 32, 8, 128, 333, [700, 0], "bf16", "16", 64, None),
    (3, 9, None, 8, 2, 64, 127, [255, 250, 1], "f16", "16", 16, None),
    (2, 41, "432", 8, 2, 128, 100, [100, 300], "bf16", "16", 32, None),
    (2, 17, None, 16, 4, 128, 640, [31, 900], "f16", "16", 128, None),
    (9, 1, None, 2, 2, 64, 0, [0, 5, 16, 1023, 1024, 1025, 2047, 3000, 129], "bf16", "16", 256, None),
    (9, 1, None, 12, 2, 64, 0, [0, 5, 16, 1023, 1024, 1025, 2047, 3000, 129], "bf16", "f8", 64, 16),
]


def _parent(kind, R):
    if kind is None:
        return None
    if kind == "432":
        return list(synth.bfs_tree((4, 3, 2)))
    return [-1] + ([0] * (R - 1) if kind == "star" else [max(0, v - 4) for v in range(1, R)])


def poison(cache, table, lens, rows, value=float("nan")):
    """NaN in the pages of each sequence behind its rows (nothing there may matter)."""
    page = cache.k.shape[1]
    for b, n in enumerate(lens):
        for t in range(n + rows, table.shape[1] * page):
            for x in (cache.k, cache.v):
                x.view(torch.uint8 if x.dtype == F8 else x.dtype)[int(table[b, t // page]), t % page] = 0x7F if x.dtype == F8 else value


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)) if len(str(c)) < 120 else None)
@pytest.mark.parametrize("token_major", [False, True])
def test_against_definition(case, token_major):
    print("paged attention", case, token_major, flush=True)
    B, R, kind, Hq, Hkv, D, P, lens, dtype, held, page, block = case
    parent = _parent(kind, R)
    q, cache, table, prefix = make(B, R, Hq, Hkv, D, P, max(lens) + R + 3, dtype, held, page, block, 17 * R + D, token_major=token_major,
                                   pow2=not token_major)
    if B * (max(lens) + R) < 1500:
        poison(cache, table, lens, R)
    length = torch.tensor(lens, dtype=torch.int32, device=DEV)
    kw = dict(prefix_table=prefix if P else None, prefix_len=P, parent=parent, return_lse=True)
    res = sv.paged_attention(q, cache, table, length, **kw)
    torch.cuda.synchronize()
    check(res, q, cache, table, lens, prefix=prefix, P=P, parent=parent)
    again = sv.paged_attention(q, cache, table, length, **kw)
    assert torch.equal(again.out, res.out) and torch.equal(again.lse, res.lse)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("R,P", [(1, 0), (9, 300), (41, 0)])
def test_equals_contiguous_caches(dtype, R, P):
    """16-bit pages hold the same numbers as a contiguous cache: the results agree within either's tolerance, and
    in most places to the bit."""
    B, Hq, Hkv, D, page = 3, 8, 2, 128, 32
    lens = [500, 33, 0]
    parent = _parent("432", R) if R == 41 else None
    q, cache, table, prefix = make(B, R, Hq, Hkv, D, P, 560, dtype, "16", page, None, 5)
    length = torch.tensor(lens, dtype=torch.int32, device=DEV)
    a = sv.paged_attention(q, cache, table, length, prefix_table=prefix if P else None, prefix_len=P, parent=parent, return_lse=True)
    k, v = (t[table.long()].reshape(B, -1, Hkv, D) for t in (cache.k, cache.v))
    pk, pv = (t[prefix.long()].reshape(-1, Hkv, D)[:P] for t in (cache.k, cache.v)) if P else (None, None)
    b = sv.attention(q, k, v, length, prefix_k=pk, prefix_v=pv, parent=parent, return_lse=True)
    torch.cuda.synchronize()
    check(a, q, cache, table, lens, prefix=prefix, P=P, parent=parent)
    check(b, q, cache, table, lens, prefix=prefix, P=P, parent=parent)


def test_scales_far_apart():
    """Blocks whose scales differ by 2^40, negative and tiny score scales: statistics and sums keep their precision."""
    for dtype in ("bf16", "f16"):
        q, cache, table, _ = make(2, 3, 8, 2, 64, 0, 700, dtype, "f8", 16, 16, 3)
        cache.v_scale.copy_(torch.exp2(torch.randint(-26, 15, cache.v_scale.shape, device=DEV).double() - 18).float())
        lens = [690, 400]
        for scale in (None, -0.05, 1e-30, 0.0):
            res = sv.paged_attention(q, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV), scale=scale, return_lse=True)
            check(res, q, cache, table, lens, scale=scale)


def test_blocks_of_zeros():
    """What cache_append leaves for blocks of zeros (scales of 2^-100) changes nothing but their own values."""
    for dtype in ("bf16", "f16"):
        q, cache, table, _ = make(1, 2, 4, 2, 64, 0, 300, dtype, "f8", 16, 16, 8)
        zero = table[0, ::3].long()
        cache.v.view(torch.uint8)[zero], cache.v_scale[zero] = 0, 2.0 ** -100
        cache.k.view(torch.uint8)[zero[1::2]], cache.k_scale[zero[1::2]] = 0, 2.0 ** -100
        n = torch.tensor([290], dtype=torch.int32, device=DEV)
        check(sv.paged_attention(q, cache, table, n, return_lse=True), q, cache, table, [290])


def test_row_count_and_bad_lengths():
    B, R = 6, 5
    q, cache, table, prefix = make(B, R, 8, 4, 128, 30, 64, "bf16", "f8", 16, 16, 3)
    lens, rc = [10, 20, 59, 60, -1, 5], [0, 2, 5, 5, 5, 99]
    for b in (0, 1):  # unused rows of the step
        for t in range(lens[b] + rc[b], 64):
            cache.k.view(torch.uint8)[int(table[b, t // 16]), t % 16] = 0x7F
            cache.v.view(torch.uint8)[int(table[b, t // 16]), t % 16] = 0xFF
    res = sv.AttentionResult(torch.full((B, R, 8, 128), 3.0, dtype=torch.bfloat16, device=DEV),
                             torch.full((B, R, 8), 3.0, device=DEV))
    sv.paged_attention(q, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV), prefix_table=prefix, prefix_len=30,
                       row_count=torch.tensor(rc, dtype=torch.int32, device=DEV), out=res)
    torch.cuda.synchronize()
    assert (res.out[0] == 3).all() and (res.out[1, 2:] == 3).all() and (res.lse[0] == 3).all() and (res.lse[1, 2:] == 3).all()
    assert torch.isnan(res.out[3:5]).all() and torch.isnan(res.lse[3:5]).all()  # 60 > 64 - R, and -1
    ok = [1, 2, 5]
    sub = sv.AttentionResult(res.out[ok], res.lse[ok])
    check(sub, q[ok], cache, table[ok], [lens[b] for b in ok], prefix=prefix, P=30, row_count=[rc[b] for b in ok])


@pytest.mark.parametrize("held", ["f8", "16"])
def test_bad_pages(held):
    """A page that is none among a sequence's tokens: its rows are NaN, the others' stay; behind its tokens: nothing."""
    B, R, page = 5, 3, 32
    q, cache, table, prefix = make(B, R, 8, 2, 64, 100, 1400, "bf16", held, page, 16, 11)
    lens = [1300, 700, 64, 0, 1390]
    good = table.clone()
    num = cache.k.shape[0]
    table[0, 3], table[1, 700 // page], table[4, 1392 // page] = -1, num, 1 << 30
    table[2, 3:], table[3, 1:] = -1, -7
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    res = sv.paged_attention(q, cache, table, n, prefix_table=prefix, prefix_len=100, return_lse=True)
    torch.cuda.synchronize()
    bad = [0, 1, 4]
    assert torch.isnan(res.out[bad]).all() and torch.isnan(res.lse[bad]).all()
    sub = sv.AttentionResult(res.out[2:4], res.lse[2:4])
    check(sub, q[2:4], cache, good[2:4], lens[2:4], prefix=prefix, P=100)
    worse = prefix.clone()
    worse[3] = -1
    res = sv.paged_attention(q, cache, good, n, prefix_table=worse, prefix_len=100, return_lse=True)
    assert torch.isnan(res.out).all() and torch.isnan(res.lse).all()
    res = sv.paged_attention(q, cache, good, n, prefix_table=worse, prefix_len=96, return_lse=True)
    torch.cuda.synchronize()
    check(res, q, cache, good, lens, prefix=prefix, P=96)


@pytest.mark.parametrize("held", ["f8", "16"])
@pytest.mark.parametrize("R,Hq", [(9, 4), (5, 20), (41, 8), (17, 16)])
def test_odd_values_of_the_step_reach_their_rows_only(held, R, Hq):
    """NaN among the step's own keys and values reaches the rows that see it and no others (16 bits: infinities too)."""
    B, Hkv, D, page = 2, 4 if Hq % 4 == 0 else 1, 64, 16
    parent = _parent("432", R) if R == 41 else None
    q, cache, table, _ = make(B, R, Hq, Hkv, D, 0, 200, "f16", held, page, 16, R)
    lens = [100, 27]
    odd = 0x7F if held == "f8" else float("nan")
    raw = lambda t: t.view(torch.uint8) if held == "f8" else t  # noqa: E731
    at = lambda b, r: (int(table[b, (lens[b] + r) // page]), (lens[b] + r) % page)  # noqa: E731
    raw(cache.v)[at(0, 3)][0, 5] = odd
    raw(cache.v)[at(1, 2)][Hkv - 1, 63] = odd if held == "f8" else float("inf")
    raw(cache.v)[at(1, 4)][0, 1] = 0xFF if held == "f8" else float("-inf")
    res = sv.paged_attention(q, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV), parent=parent, return_lse=True)
    torch.cuda.synchronize()
    check(res, q, cache, table, lens, parent=parent)


def test_kept_workspace_and_max_ctx():
    """One workspace for calls of several lengths; max_ctx bounds the lengths and changes no result."""
    q, cache, table, _ = make(3, 2, 8, 2, 128, 0, 3000, "bf16", "f8", 64, 32, 21)
    ws = sv.paged_attention_workspace(3, 2, 8, 2, 128, 0, 2998, DEV)
    ws.fill_(0xFF)
    for lens in ([2998, 0, 100], [100, 100, 100], [1, 2000, 64]):
        n = torch.tensor(lens, dtype=torch.int32, device=DEV)
        a = sv.paged_attention(q, cache, table, n, ws=ws, max_ctx=2998, return_lse=True)
        b = sv.paged_attention(q, cache, table, n, max_ctx=max(lens), return_lse=True)
        torch.cuda.synchronize()
        assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)
        check(a, q, cache, table, lens)
    r = sv.paged_attention(q, cache, table, torch.tensor([50, 51, 3], dtype=torch.int32, device=DEV), max_ctx=50)
    assert torch.isnan(r.out[1]).all() and torch.isfinite(r.out[0]).all()


def test_sequences_share_pages():
    """Two sequences with the same first pages, and one page twice in a table."""
    q, cache, table, _ = make(3, 2, 4, 2, 64, 0, 130, "bf16", "f8", 16, 16, 2)
    table[1, :4] = table[0, :4]
    table[2, 1] = table[2, 0]
    lens = [100, 80, 120]
    res = sv.paged_attention(q, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV), return_lse=True)
    torch.cuda.synchronize()
    check(res, q, cache, table, lens)


def test_far_pages():
    """Pages whose offsets pass 32 bits (bytes and elements)."""
    D, Hkv, page = 128, 8, 64
    num = (5 << 30) // (page * Hkv * D)
    cache = sv.PagedCache(*(torch.zeros(num, Hkv, page, D, dtype=torch.uint8, device=DEV).view(F8).transpose(1, 2) for _ in range(2)),
                          *(torch.full((num, 1, Hkv), 2.0 ** -7, device=DEV) for _ in range(2)))
    far = torch.tensor([[num - 1, 3, num - 2, (4 << 30) // (page * Hkv * D), num // 2]], dtype=torch.int32, device=DEV)
    x = torch.randn(1, 200, Hkv, D, device=DEV).to(torch.bfloat16)
    n = torch.tensor([40], dtype=torch.int32, device=DEV)
    sv.cache_append(cache, far, torch.zeros_like(n), x[:, :40], x[:, :40])
    sv.cache_append(cache, far, n, x, x)
    q = torch.randn(1, 1, Hkv, D, device=DEV).to(torch.bfloat16)
    n = torch.tensor([239], dtype=torch.int32, device=DEV)
    res = sv.paged_attention(q, cache, far, n, return_lse=True)
    torch.cuda.synchronize()
    check(res, q, cache, far, [239])
    assert np.abs(dense(cache, far[0], 240)[0][40:] - host(x[0])).max() < 0.3


def test_refusals_on_the_device():
    q, cache, table, prefix = make(2, 3, 8, 2, 64, 50, 100, "bf16", "f8", 16, 16, 1)
    n = torch.zeros(2, dtype=torch.int32, device=DEV)
    for kw in (dict(q=q.float()), dict(q=q[..., :32]), dict(q=q[:, :, :7]), dict(page_table=table.long()), dict(page_table=table[:1]), dict(ctx_len=None),
               dict(ctx_len=n[:1]), dict(prefix_len=50), dict(prefix_len=81, prefix_table=prefix), dict(prefix_len=50, prefix_table=prefix.long()),
               dict(parent=[-1, 0]), dict(parent=[-1, 1, 0]), dict(max_ctx=110), dict(max_ctx=-1), dict(scale=float("nan")),
               dict(ws=torch.zeros(256, dtype=torch.uint8, device=DEV)), dict(out=sv.AttentionResult(q[:1])), dict(out=sv.AttentionResult(None)),
               dict(cache=sv.paged_cache(4, 16, 2, 64, torch.float16, DEV)), dict(cache=sv.paged_cache(4, 16, 2, 64, F8, DEV, layers=2))):
        a = dict(q=q, cache=cache, page_table=table, ctx_len=n)
        a.update(kw)
        with pytest.raises((ValueError, sv.SvError)):
            sv.paged_attention(a.pop("q"), a.pop("cache"), a.pop("page_table"), a.pop("ctx_len"), **a)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("R,Hq,P", [(3, 8, 0), (17, 16, 0), (4, 8, 70), (20, 16, 200)])
def test_scales_of_zero(dtype, R, Hq, P):
    """Blocks that another program scaled by zero, the first ones of a sequence and whole sequences among them, are
    blocks of zeros (bytes that are none may count for up to 2^-117 of a unit each)."""
    q, cache, table, prefix = make(3, R, Hq, 2, 64, P, 300, dtype, "f8", 16, 16, 4)
    lens = [250, 40, 130]
    none = table[0, ::2].long().tolist() + table[1].long().tolist() + table[2, 1:3].long().tolist() + prefix[:2].long().tolist()
    cache.v_scale[none] = 0.0
    cache.k_scale[none[1::2]] = 0.0
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    res = sv.paged_attention(q, cache, table, n, prefix_table=prefix if P else None, prefix_len=P, return_lse=True)
    torch.cuda.synchronize()
    check(res, q, cache, table, lens, prefix=prefix, P=P)
    if P == 0:
        assert np.abs(host(res.out[1])).max() < 2.0 ** -100


@pytest.mark.parametrize("held", ["f8", "16"])
@pytest.mark.parametrize("R,P", [(1, 0), (4, 0), (4, 700), (17, 700)])
def test_large_scores_keep_their_differences(held, R, P):
    """float16: scores of 131072 + d, exact in float32, weigh by d alone.  Tolerance: the one above, its term of the
    scores' size A by that of their differences, as products and differences are exact here; a statistic of size S is
    rounded five times (the scale, the maximum's product, the sum, the factor ln 2 and the product by it)."""
    B, Hq, Hkv, D, page = 2, 8, 2, 64, 32
    q, cache, table, prefix = make(B, R, Hq, Hkv, D, P, 900, "f16", held, page, 32, 12)
    lens, size = [880, 300], 1 << 20
    g = torch.Generator(device=DEV).manual_seed(R)
    q.zero_()
    q[..., 0], q[..., 1] = 1024, torch.randint(1, 3, q.shape[:-1], generator=g, device=DEV).half()
    k = torch.zeros(cache.k.shape, device=DEV)
    k[..., 0] = size / 1024 if held == "16" else 256
    k[..., 1] = torch.randint(-30, 31, k.shape[:-1], generator=g, device=DEV).float() * (1 if held == "16" else 0.5)
    if held == "f8":   # powers of two apart, and numbers of 3 bits: -15 .. 15 times 1/4
        k[..., 1] = torch.randint(-15, 16, k.shape[:-1], generator=g, device=DEV).float() / 4
        cache.k_scale.fill_(4.0)
        cache.k.copy_(k.to(F8))
        assert torch.equal(cache.k.float(), k)
    else:
        cache.k.copy_(k)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    res = sv.paged_attention(q, cache, table, n, scale=0.125, prefix_table=prefix if P else None, prefix_len=P, return_lse=True)
    torch.cuda.synchronize()
    pk, pv = dense(cache, prefix, P) if P else (None, None)
    h = HALF_STEP[q.dtype]
    for b in range(B):
        kb, vb = dense(cache, table[b], lens[b] + R)
        qb = host(q[b])
        out, lse = oracle.attention(qb, kb, vb, lens[b], prefix_k=pk, prefix_v=pv, scale=0.125)
        weight, _ = oracle.attention(qb, kb, np.abs(vb), lens[b], prefix_k=pk, prefix_v=None if pv is None else np.abs(pv), scale=0.125)
        values = vb if pv is None else np.concatenate([pv, vb])
        N = len(values)
        rel = 2 * (D + N + 16) * 2.0 ** -24 * (1 + 0.125 * 120)
        tol = (h + rel) * weight * (1 + 2.0 ** -6) + h * np.abs(out) + 2.0 ** -24 + N * 2.0 ** -40 * np.abs(values).max()
        err = np.abs(host(res.out[b]) - out)
        assert (err <= tol).all(), (b, float((err / tol).max()))
        err = np.abs(host(res.lse[b]) - lse)
        assert (err <= 5 * 2.0 ** -24 * np.abs(lse) + rel).all(), (b, float(err.max()))
