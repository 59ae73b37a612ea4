"""Refusals of the 4-bit LM head that need no device."""
import pytest
import torch

import draft_token_verification_06_amd as sv
from draft_token_verification_06_amd import _lib

FAKE = 0x100000  # never dereferenced: validation fails first


def _call(**kw):
    a = dict(hidden=FAKE, stride=0, dtype=1, weights=FAKE, scales=FAKE, zeros=None, M=4, K=256, V=100, group=64,
             out=FAKE, out_stride=0, out_dtype=0, ws=None, ws_bytes=0)
    a.update(kw)
    return _lib.lib().sv_lmhead_quant(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=0), -2),
    (dict(dtype=5), -2),
    (dict(out_dtype=2), -2),                 # float16 rows from bf16 states
    (dict(M=0), -1),
    (dict(M=65536), -1),
    (dict(M=33), -3),                        # more rows than 32 need a workspace
    (dict(M=33, ws=FAKE, ws_bytes=1024), -3),
    (dict(M=33, ws=FAKE + 16, ws_bytes=1 << 20), -3),
    (dict(V=0), -1),
    (dict(V=(1 << 21) + 1), -1),
    (dict(group=16), -1),
    (dict(group=96), -1),
    (dict(K=0), -1),
    (dict(K=96), -1),                        # not a multiple of 64
    (dict(K=192, group=128), -1),            # not a multiple of the group
    (dict(K=65536 + 64), -1),
    (dict(hidden=None), -1),
    (dict(weights=None), -1),
    (dict(scales=None), -1),
    (dict(out=None), -1),
    (dict(hidden=FAKE + 8), -1),
    (dict(weights=FAKE + 4), -1),
    (dict(scales=FAKE + 1), -1),
    (dict(out=FAKE + 2), -1),
    (dict(stride=248), -1),
    (dict(stride=260), -1),                  # rows off the 16-byte grid
    (dict(out_stride=99), -1),
])
def test_status(kw, status):
    assert _call(**kw) == status


def test_workspace_rules():
    L = _lib.lib()
    size = L.sv_lmhead_quant_workspace
    assert size(32, 4096, 5000, 128) == 0
    assert size(33, 4096, 200000, 128) >= 33 * (4096 * 2 + 32 * 4)
    assert size(33, 4096, 200000, 128) % 256 == 0
    assert size(200, 4096, 4000, 128) >= 200 * (4096 * 2 + 32 * 4) + 2 * 200 * 4000 * 4  # K shared out
    assert size(33, 4096, 5000, 96) == 0
    assert size(0, 4096, 5000, 128) == 0
    assert size(33, 4096, 0, 128) == 0


def test_binding_refuses():
    h = torch.zeros(2, 128, dtype=torch.bfloat16)
    w, s = torch.zeros(10, 64, dtype=torch.uint8), torch.zeros(10, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sv.lmhead_quant(h, w, s)             # host memory
    with pytest.raises(ValueError):
        sv.lmhead_quant(h.float(), w, s)


def test_every_size_of_the_rules_is_accepted():
    """Calls of many rows go by the tiles they launch (64 or 80 rows, 128
    columns), and the workspace is sized for what a call accepts."""
    size = _lib.lib().sv_lmhead_quant_workspace
    for M, V in ((40000, 128256), (65535, 128256), (65535, 1 << 20), (9000, 1 << 21), (32, 1 << 21)):
        assert M <= 32 or _call(M=M, V=V) == -3              # only the workspace is missing
        assert (size(M, 256, V, 64) > 0) == (M > 32)
    assert _call(M=65535, V=1 << 21) == -1 and size(65535, 256, 1 << 21, 64) == 0   # 2^24 workgroups of 256 work-items
