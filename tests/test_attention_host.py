"""Refusals of the attention of draft rows that need no device."""
import ctypes

import pytest
import torch

import draft_token_verification_06_amd as sv
from draft_token_verification_06_amd import _lib

FAKE = 0x100000  # never dereferenced: validation fails first


def _call(**kw):
    a = dict(q=FAKE, q_stride=0, dtype=1, k=FAKE, v=FAKE, seq_stride=0, tok_stride=0, cap=64, pk=FAKE, pv=FAKE, pstride=0,
             P=10, ctx_len=FAKE, row_count=None, parent=None, B=2, R=5, Hq=8, Hkv=2, D=128, max_ctx=59, scale=0.1,
             out=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    if a["parent"] is not None:
        a["parent"] = (ctypes.c_int32 * len(a["parent"]))(*a["parent"])
    return _lib.lib().sv_attention(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=0), -2),
    (dict(dtype=9), -2),
    (dict(B=0), -1),
    (dict(R=0), -1),
    (dict(R=66, cap=200), -1),                # a window has at most SV_MAX_GAMMA + 1 rows
    (dict(Hq=9), -1),                         # not a multiple of the kv heads
    (dict(Hq=0), -1),
    (dict(Hkv=0), -1),
    (dict(Hq=2048), -1),
    (dict(D=96), -1),
    (dict(P=-1), -1),
    (dict(P=(1 << 24) + 1), -1),
    (dict(max_ctx=-1), -1),
    (dict(max_ctx=60), -1),                   # max_ctx + R > cap
    (dict(cap=0), -1),
    (dict(q=None), -1),
    (dict(k=None), -1),
    (dict(v=None), -1),
    (dict(pk=None), -1),
    (dict(pv=None), -1),
    (dict(ctx_len=None), -1),
    (dict(out=None), -1),
    (dict(q=FAKE + 8), -1),
    (dict(k=FAKE + 8), -1),
    (dict(pv=FAKE + 8), -1),
    (dict(out=FAKE + 8), -1),
    (dict(lse=FAKE + 2), -1),
    (dict(q_stride=1016), -1),                # below Hq * D
    (dict(q_stride=1028), -1),                # not a multiple of 8
    (dict(tok_stride=248), -1),
    (dict(seq_stride=-8), -1),
    (dict(pstride=255), -1),
    (dict(scale=float("nan")), -1),
    (dict(scale=float("inf")), -1),
    (dict(parent=[-1, 0, 1, 4, 0]), -4),
    (dict(ws=None), -3),
    (dict(ws=FAKE + 16), -3),
    (dict(ws_bytes=256), -3),
    (dict(B=1 << 27), -1),
])
def test_status(kw, status):
    assert _call(**kw) == status


def test_workspace_rules():
    L = _lib.lib()
    assert L.sv_attention_workspace(4, 9, 32, 8, 128, 1000, 2000) % 256 == 0
    assert L.sv_attention_workspace(4, 9, 32, 8, 128, 1000, 2000) >= 2 * 4 * 9 * 32 * 130 * 4
    assert L.sv_attention_workspace(4, 9, 32, 8, 80, 1000, 2000) == 0
    assert L.sv_attention_workspace(4, 9, 32, 5, 128, 1000, 2000) == 0
    with pytest.raises(ValueError):
        sv.attention_workspace(0, 1, 1, 1, 64, 0, 0, "cpu")


def test_binding_refuses():
    q, k, n = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 9, 2, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        sv.attention(q, k, k, n)              # host memory
    with pytest.raises(ValueError):
        sv.attention(q.float(), k, k, n)
