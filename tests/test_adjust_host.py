"""Refusals of the logits adjustment that need no device: the C entry returns a
status before any device work, the binding raises ValueError."""
import ctypes

import pytest
import torch

import draft_token_verification_06_amd as sv
from draft_token_verification_06_amd import _lib

FAKE = 0x100000  # never dereferenced: validation fails first


def _call(**kw):
    a = dict(logits=FAKE, seq_stride=0, out=FAKE + (1 << 24), out_seq_stride=0, dtype=1, tokens=FAKE, tokens_stride=0, parent=None,
             row_count=None, B=2, R=5, V=100, history=FAKE, history_stride=0, history_cap=16, history_len=None,
             prompt_len=None, repetition=FAKE, presence=None, frequency=None, bias_tokens=None, bias_values=None,
             n_bias=0, allowed=None, allowed_seq_stride=0, allowed_row_stride=0)
    a.update(kw)
    if a["parent"] is not None:
        a["parent"] = (ctypes.c_int32 * len(a["parent"]))(*a["parent"])
    return _lib.lib().sv_adjust_logits(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), -2),
    (dict(B=0), -1),
    (dict(R=0), -1),
    (dict(V=0), -1),
    (dict(V=(1 << 21) + 1), -1),
    (dict(R=66), -1),                                    # a window has at most SV_MAX_GAMMA + 1 rows
    (dict(logits=None), -1),
    (dict(out=None), -1),
    (dict(logits=FAKE + 1), -1),                         # misaligned bf16
    (dict(out=FAKE + (1 << 24) + 1), -1),
    (dict(seq_stride=499), -1),                          # below R * V
    (dict(out_seq_stride=499), -1),
    (dict(out=FAKE + 2), -1),                            # overlaps the input without being it
    (dict(out=FAKE, out_seq_stride=600), -1),            # in place with another stride
    (dict(tokens=None), -1),                             # penalties on several rows need tokens
    (dict(tokens_stride=3), -1),
    (dict(history_cap=-1), -1),
    (dict(history=None), -1),
    (dict(history_stride=15), -1),
    (dict(n_bias=-1), -1),
    (dict(n_bias=1), -1),                                # entries without pointers
    (dict(n_bias=65536, bias_tokens=FAKE, bias_values=FAKE), -1),
    (dict(allowed=FAKE + 2), -1),
    (dict(allowed=FAKE, allowed_row_stride=-1), -1),
    (dict(parent=[-1, 0, 5, 0, 0]), -4),
    (dict(parent=[0, 0, 0, 0, 0]), -4),
    (dict(B=1 << 24, R=1, V=100), -1),                   # 2^24 workgroups of 256 work-items
])
def test_status(kw, status):
    assert _call(**kw) == status


def test_binding_refuses():
    x = torch.zeros(2, 3, 40)
    with pytest.raises(ValueError):
        sv.adjust_logits(x)                              # host memory
    with pytest.raises(ValueError):
        sv.adjust_logits(x[0])
    with pytest.raises(ValueError):
        sv.adjust_logits(x.double())
