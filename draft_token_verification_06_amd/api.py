"""Python binding of the C ABI in include/sv.h, sv_step.h and sv_cache.h:
argument marshalling only.

Tensors must live on a ROCm device; every computation runs in the HIP
library on the current torch stream of that device.  Results come back as
device tensors; nothing synchronises.  No call keeps an autograd history:
outputs require no gradient, whatever the inputs do.
"""
import ctypes
import math
from dataclasses import dataclass
from typing import Optional

import torch

from ._lib import PAGED_CACHE, lib

SV_OP_WINDOW, SV_OP_GREEDY, SV_OP_TREE, SV_OP_LMHEAD = 0, 1, 2, 3
SV_TREE_GREEDY, SV_TREE_STOCHASTIC, SV_TREE_MULTI_CANDIDATE = 0, 1, 2
_TREE_MODES = {"greedy": SV_TREE_GREEDY, "stochastic": SV_TREE_STOCHASTIC,
               "multi_candidate": SV_TREE_MULTI_CANDIDATE}
_DTYPE_CODE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
SV_DT_F8E4M3 = 3
_PAGE_CODE = {torch.bfloat16: 1, torch.float16: 2, torch.float8_e4m3fn: SV_DT_F8E4M3}


class SvError(RuntimeError):
    def __init__(self, status):
        self.status = status
        super().__init__(f"specverify status {status}: {lib().sv_strerror(status).decode()}")


def _check(status):
    if status != 0:
        raise SvError(status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _logits(t, rows, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype not in _DTYPE_CODE:
        raise ValueError(f"{name}: dtype {t.dtype} is not float32, bfloat16 or float16")
    if t.dim() != 3 or t.shape[1] != rows:
        raise ValueError(f"{name}: expected shape (B, {rows}, V), got {tuple(t.shape)}")
    V = t.shape[2]
    if t.stride(2) != 1 or t.stride(1) != V:
        raise ValueError(f"{name}: rows of one sequence must be contiguous")
    return t.stride(0)


def _i32(t, shape, name):
    if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected a contiguous int32 device tensor of shape {tuple(shape)}")


def _optional(t, dtype, B, name):
    if t is None:
        return None
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != (B,):
        raise ValueError(f"{name}: expected a contiguous {dtype} device tensor of shape ({B},)")
    return t


def _same_device(dev, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")


def _ws_bytes(ws, dev):
    """Byte size of a caller-supplied workspace (a contiguous device tensor)."""
    if not ws.is_cuda or not ws.is_contiguous() or ws.device != dev:
        raise ValueError(f"workspace: expected a contiguous device tensor on {dev}")
    return ws.numel() * ws.element_size()


def _out_tensor(t, dtype, shape, dev, name):
    if t is None:
        return
    if t.dtype != dtype or t.device != dev or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on {dev}")


def _check_window_out(out, B, gamma, dev):
    if out.n_accepted is None or out.out_tokens is None:
        raise ValueError("n_accepted and out_tokens are required outputs")
    _out_tensor(out.n_accepted, torch.int32, (B,), dev, "n_accepted")
    _out_tensor(out.out_tokens, torch.int32, (B, gamma + 1), dev, "out_tokens")
    _out_tensor(out.p_draft, torch.float32, (B, gamma), dev, "p_draft")
    _out_tensor(out.q_draft, torch.float32, (B, gamma), dev, "q_draft")


def workspace_size(op, B, n, V, dtype):
    return int(lib().sv_workspace_size(op, B, n, V, _DTYPE_CODE[dtype]))


def workspace(op, B, n, V, dtype, device):
    nbytes = workspace_size(op, B, n, V, dtype)
    if nbytes == 0:
        raise ValueError("invalid sizes for a workspace")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


@dataclass
class WindowResult:
    n_accepted: torch.Tensor
    out_tokens: torch.Tensor
    p_draft: Optional[torch.Tensor] = None
    q_draft: Optional[torch.Tensor] = None


@dataclass
class TreeResult:
    n_accepted: torch.Tensor
    best_node: torch.Tensor
    out_tokens: torch.Tensor
    out_nodes: torch.Tensor


SV_PART_ROW_STATS, SV_PART_DECIDE_SAMPLE = 1, 2


def verify_window(target, draft, tokens, *, seed=0, tag=0, window_len=None, seq_ids=None,
                  base_pos=None, return_probs=False, ws=None, out=None, part=None, early_exit=False):
    """Stochastic window verification: sv_verify_window, one half of it
    (sv_verify_window_part) when part is SV_PART_ROW_STATS / SV_PART_DECIDE_SAMPLE,
    or sv_verify_window_early_exit when early_exit is set."""
    B, rows, V = target.shape
    gamma = rows - 1
    ts = _logits(target, gamma + 1, "target")
    ds = _logits(draft, gamma, "draft")
    if draft.dtype != target.dtype or draft.shape[0] != B or draft.shape[2] != V:
        raise ValueError("draft must match target in dtype, batch and vocabulary")
    _i32(tokens, (B, gamma), "tokens")
    _optional(window_len, torch.int32, B, "window_len")
    _optional(seq_ids, torch.int64, B, "seq_ids")
    _optional(base_pos, torch.int64, B, "base_pos")
    dev = target.device
    _same_device(dev, draft=draft, tokens=tokens, window_len=window_len, seq_ids=seq_ids,
                 base_pos=base_pos)
    if ws is None:
        ws = workspace(SV_OP_WINDOW, B, gamma, V, target.dtype, dev)
        ws_bytes = ws.numel()
    else:
        ws_bytes = _ws_bytes(ws, dev)
    if out is None:
        out = WindowResult(torch.empty(B, dtype=torch.int32, device=dev),
                           torch.empty(B, gamma + 1, dtype=torch.int32, device=dev))
        if return_probs:
            out.p_draft = torch.empty(B, gamma, dtype=torch.float32, device=dev)
            out.q_draft = torch.empty(B, gamma, dtype=torch.float32, device=dev)
    else:
        _check_window_out(out, B, gamma, dev)
    if early_exit:
        if part is not None:
            raise ValueError("early_exit has no parts")
        head = (lib().sv_verify_window_early_exit,)
    else:
        head = (lib().sv_verify_window,) if part is None else (lib().sv_verify_window_part, part)
    with torch.cuda.device(dev):
        _check(head[0](
            *head[1:], _ptr(target), ts, _ptr(draft), ds, _DTYPE_CODE[target.dtype],
            _ptr(tokens), _ptr(window_len), B, gamma, V,
            ctypes.c_uint64(seed), ctypes.c_uint64(tag), _ptr(seq_ids), _ptr(base_pos),
            _ptr(out.n_accepted), _ptr(out.out_tokens), _ptr(out.p_draft), _ptr(out.q_draft),
            _ptr(ws), ws_bytes, _stream(dev)))
    return out


def verify_window_noalloc(target, draft, tokens, *, seed=0, tag=0, window_len=None, seq_ids=None,
                          base_pos=None, return_probs=False, out=None):
    """sv_verify_window_noalloc: the stochastic window on the library's static
    per-GPU scratch, with no workspace.  Calls on one GPU must not overlap."""
    B, rows, V = target.shape
    gamma = rows - 1
    ts = _logits(target, gamma + 1, "target")
    ds = _logits(draft, gamma, "draft")
    if draft.dtype != target.dtype or draft.shape[0] != B or draft.shape[2] != V:
        raise ValueError("draft must match target in dtype, batch and vocabulary")
    _i32(tokens, (B, gamma), "tokens")
    _optional(window_len, torch.int32, B, "window_len")
    _optional(seq_ids, torch.int64, B, "seq_ids")
    _optional(base_pos, torch.int64, B, "base_pos")
    dev = target.device
    _same_device(dev, draft=draft, tokens=tokens, window_len=window_len, seq_ids=seq_ids,
                 base_pos=base_pos)
    if out is None:
        out = WindowResult(torch.empty(B, dtype=torch.int32, device=dev),
                           torch.empty(B, gamma + 1, dtype=torch.int32, device=dev))
        if return_probs:
            out.p_draft = torch.empty(B, gamma, dtype=torch.float32, device=dev)
            out.q_draft = torch.empty(B, gamma, dtype=torch.float32, device=dev)
    else:
        _check_window_out(out, B, gamma, dev)
    with torch.cuda.device(dev):
        _check(lib().sv_verify_window_noalloc(
            _ptr(target), ts, _ptr(draft), ds, _DTYPE_CODE[target.dtype],
            _ptr(tokens), _ptr(window_len), B, gamma, V,
            ctypes.c_uint64(seed), ctypes.c_uint64(tag), _ptr(seq_ids), _ptr(base_pos),
            _ptr(out.n_accepted), _ptr(out.out_tokens), _ptr(out.p_draft), _ptr(out.q_draft),
            _stream(dev)))
    return out


def verify_window_lmhead(h_target, w_target, h_draft, w_draft, tokens, *, seed=0, tag=0,
                         window_len=None, seq_ids=None, base_pos=None, return_probs=False, ws=None):
    """Window verification on logits from hidden states, LM head fused:
    sv_verify_window_lmhead.  h_target (B, gamma+1, Ht), w_target (V, Ht),
    h_draft (B, gamma, Hd), w_draft (V, Hd), all bf16 and contiguous."""
    B, rows, Ht = h_target.shape
    gamma = rows - 1
    V = w_target.shape[0]
    for name, t in (("h_target", h_target), ("w_target", w_target), ("h_draft", h_draft),
                    ("w_draft", w_draft)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous bf16 device tensor")
    Hd = h_draft.shape[2]
    if h_draft.shape[:2] != (B, gamma) or w_target.shape != (V, Ht) or w_draft.shape != (V, Hd):
        raise ValueError("hidden / unembedding shapes do not agree")
    _i32(tokens, (B, gamma), "tokens")
    _optional(window_len, torch.int32, B, "window_len")
    _optional(seq_ids, torch.int64, B, "seq_ids")
    _optional(base_pos, torch.int64, B, "base_pos")
    dev = h_target.device
    _same_device(dev, w_target=w_target, h_draft=h_draft, w_draft=w_draft, tokens=tokens,
                 window_len=window_len, seq_ids=seq_ids, base_pos=base_pos)
    if ws is None:
        ws = workspace(SV_OP_LMHEAD, B, gamma, V, torch.bfloat16, dev)
        ws_bytes = ws.numel()
    else:
        ws_bytes = _ws_bytes(ws, dev)
    out = WindowResult(torch.empty(B, dtype=torch.int32, device=dev),
                       torch.empty(B, gamma + 1, dtype=torch.int32, device=dev))
    if return_probs:
        out.p_draft = torch.empty(B, gamma, dtype=torch.float32, device=dev)
        out.q_draft = torch.empty(B, gamma, dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        _check(lib().sv_verify_window_lmhead(
            _ptr(h_target), _ptr(w_target), Ht, _ptr(h_draft), _ptr(w_draft), Hd,
            _ptr(tokens), _ptr(window_len), B, gamma, V,
            ctypes.c_uint64(seed), ctypes.c_uint64(tag), _ptr(seq_ids), _ptr(base_pos),
            _ptr(out.n_accepted), _ptr(out.out_tokens), _ptr(out.p_draft), _ptr(out.q_draft),
            _ptr(ws), ws_bytes, _stream(dev)))
    return out


def verify_greedy(target, tokens, *, window_len=None, ws=None, out=None):
    """Greedy window verification: sv_verify_greedy."""
    B, rows, V = target.shape
    gamma = rows - 1
    ts = _logits(target, gamma + 1, "target")
    _i32(tokens, (B, gamma), "tokens")
    _optional(window_len, torch.int32, B, "window_len")
    dev = target.device
    _same_device(dev, tokens=tokens, window_len=window_len)
    if ws is None:
        ws = workspace(SV_OP_GREEDY, B, gamma, V, target.dtype, dev)
        ws_bytes = ws.numel()
    else:
        ws_bytes = _ws_bytes(ws, dev)
    if out is None:
        out = WindowResult(torch.empty(B, dtype=torch.int32, device=dev),
                           torch.empty(B, gamma + 1, dtype=torch.int32, device=dev))
    else:
        if out.n_accepted is None or out.out_tokens is None:
            raise ValueError("n_accepted and out_tokens are required outputs")
        _out_tensor(out.n_accepted, torch.int32, (B,), dev, "n_accepted")
        _out_tensor(out.out_tokens, torch.int32, (B, gamma + 1), dev, "out_tokens")
    with torch.cuda.device(dev):
        _check(lib().sv_verify_greedy(
            _ptr(target), ts, _DTYPE_CODE[target.dtype], _ptr(tokens), _ptr(window_len),
            B, gamma, V, _ptr(out.n_accepted), _ptr(out.out_tokens),
            _ptr(ws), ws_bytes, _stream(dev)))
    return out


def tree_max_depth(parent):
    arr = (ctypes.c_int32 * len(parent))(*parent)
    d = lib().sv_tree_max_depth(arr, len(parent))
    if d < 0:
        raise SvError(d)
    return d


def verify_tree(target, draft, node_tokens, parent, *, mode="stochastic", seed=0, tag=0,
                seq_ids=None, base_pos=None, ws=None):
    """Token-tree verification: sv_verify_tree.  parent is a host sequence;
    mode "greedy", "stochastic" or "multi_candidate"."""
    B, N, V = target.shape
    if len(parent) != N:
        raise ValueError("parent must have one entry per tree node")
    if target.stride(2) != 1 or target.stride(1) != V or target.stride(0) != N * V:
        raise ValueError("target must be contiguous (B, N, V)")
    if mode not in _TREE_MODES:
        raise ValueError(f"unknown tree mode {mode!r}")
    code = _TREE_MODES[mode]
    sampled = code != SV_TREE_GREEDY
    if sampled:
        if draft is None or draft.shape != target.shape or draft.dtype != target.dtype \
                or not draft.is_contiguous():
            raise ValueError("sampled modes need contiguous draft logits shaped like target")
    _i32(node_tokens, (B, N), "node_tokens")
    _optional(seq_ids, torch.int64, B, "seq_ids")
    _optional(base_pos, torch.int64, B, "base_pos")
    D = tree_max_depth(parent)
    dev = target.device
    if not target.is_cuda or target.dtype not in _DTYPE_CODE:
        raise ValueError("target: expected float32, bfloat16 or float16 device logits")
    _same_device(dev, draft=draft if sampled else None, node_tokens=node_tokens, seq_ids=seq_ids,
                 base_pos=base_pos)
    if ws is None:
        ws = workspace(SV_OP_TREE, B, N, V, target.dtype, dev)
        ws_bytes = ws.numel()
    else:
        ws_bytes = _ws_bytes(ws, dev)
    res = TreeResult(torch.empty(B, dtype=torch.int32, device=dev),
                     torch.empty(B, dtype=torch.int32, device=dev),
                     torch.empty(B, D + 1, dtype=torch.int32, device=dev),
                     torch.empty(B, max(D, 1), dtype=torch.int32, device=dev)[:, :D])
    par = (ctypes.c_int32 * N)(*parent)
    with torch.cuda.device(dev):
        _check(lib().sv_verify_tree(
            _ptr(target), _ptr(draft if sampled else None),
            _DTYPE_CODE[target.dtype], _ptr(node_tokens), par, B, N, V, code,
            ctypes.c_uint64(seed), ctypes.c_uint64(tag), _ptr(seq_ids), _ptr(base_pos),
            _ptr(res.n_accepted), _ptr(res.best_node), _ptr(res.out_tokens), _ptr(res.out_nodes),
            _ptr(ws), ws_bytes, _stream(dev)))
    return res


# Checks of the operators below.  They run before every launch, small calls
# are bound by them, so each is one test of what it names.
def _vec(t, dtype, B, dev, name):
    """Address of a contiguous (B,) device tensor, or None."""
    if t is None:
        return None
    if t.dtype != dtype or t.device != dev or t.shape != (B,) or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape ({B},) on {dev}")
    return t.data_ptr()


def _rows_i32(t, B, cols, dev, name):
    """Row stride of an int32 device tensor (B, >= cols) with unit column stride."""
    if t.dtype != torch.int32 or t.device != dev or t.dim() != 2:
        raise ValueError(f"{name}: expected an int32 tensor of shape ({B}, >={cols}) on {dev}")
    n, width = t.shape
    row, col = t.stride()
    if n != B or width < cols or (width > 1 and col != 1) or (B > 1 and row < width):
        raise ValueError(f"{name}: expected shape ({B}, >={cols}) with unit column stride, rows not overlapping")
    return row if B > 1 else width


def _seq_stride(t, name):
    """Sequence stride of (B, R, V) logits whose rows are dense and whose sequences do not overlap (0 = dense)."""
    B, R, V = t.shape
    seq, row, col = t.stride()
    if (V > 1 and col != 1) or (R > 1 and row != V):
        raise ValueError(f"{name}: rows of one sequence must be contiguous")
    if B > 1 and seq < R * V:
        raise ValueError(f"{name}: sequences overlap")
    return seq if B > 1 else 0


def _parents(parent, R):
    if parent is None:
        return None
    if len(parent) != R:
        raise ValueError("parent must have one entry per row")
    return (ctypes.c_int32 * R)(*parent)


# The handle of a device's current stream (what torch.cuda.current_stream wraps
# in an object; asking for the handle alone takes a tenth of the time).
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    lambda index: torch.cuda.current_stream(index).cuda_stream


def _launch(dev, fn, *args):
    """Calls fn on dev's current stream with dev current."""
    index = dev.index
    if torch.cuda.current_device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(index))
    if status != 0:
        raise SvError(status)


def adjust_logits(logits, *, tokens=None, parent=None, history=None, history_len=None, prompt_len=None,
                  repetition=None, presence=None, frequency=None, bias_tokens=None, bias_values=None,
                  allowed=None, row_count=None, out=None):
    """Penalties, biases and grammar masks on logits rows: sv_adjust_logits.

    logits (B, R, V) as verify_window / verify_tree take them.  Row i of a
    window follows tokens[:, :i]; with parent (a host sequence of R entries)
    row v follows the tokens of its path.  history (B, cap) int32 with
    history_len and prompt_len (B,) int32; repetition, presence, frequency (B,)
    float32; bias_tokens / bias_values (B, n) int32 / float32; allowed int32
    (B, R, ceil(V / 32)) bit masks (rows or sequences may be expanded);
    row_count (B,) int32.  Returns out (a new tensor when None; out=logits
    works in place)."""
    dtype, dev = logits.dtype, logits.device
    if logits.dim() != 3 or dtype not in _DTYPE_CODE or dev.type != "cuda":
        raise ValueError("logits: expected a float32, bfloat16 or float16 device tensor of shape (B, R, V)")
    B, R, V = logits.shape
    stride = _seq_stride(logits, "logits")
    par = _parents(parent, R)
    tokens_ptr = history_ptr = bias_ptr = values_ptr = allowed_ptr = None
    tokens_stride = history_stride = cap = n_bias = mask_seq = mask_row = 0
    if tokens is not None:
        tokens_stride = _rows_i32(tokens, B, R if parent is not None else R - 1, dev, "tokens")
        tokens_ptr = tokens.data_ptr()
    elif R > 1 and not (repetition is None and presence is None and frequency is None):
        raise ValueError("penalties on more than one row need the rows' tokens")
    if history is not None:
        history_stride = _rows_i32(history, B, 0, dev, "history")
        cap = history.shape[1]
        history_ptr = history.data_ptr()
    elif history_len is not None or prompt_len is not None:
        raise ValueError("history_len and prompt_len need a history")
    if (bias_tokens is None) != (bias_values is None):
        raise ValueError("bias_tokens and bias_values go together")
    if bias_tokens is not None:
        n_bias = bias_tokens.shape[-1]
        for t, want, name in ((bias_tokens, torch.int32, "bias_tokens"), (bias_values, torch.float32, "bias_values")):
            if t.dtype != want or t.device != dev or t.shape != (B, n_bias) or not t.is_contiguous():
                raise ValueError(f"{name}: expected a contiguous {want} tensor of shape ({B}, {n_bias}) on {dev}")
        bias_ptr, values_ptr = bias_tokens.data_ptr(), bias_values.data_ptr()
    if allowed is not None:
        W = (V + 31) // 32
        if allowed.dtype != torch.int32 or allowed.device != dev or allowed.shape != (B, R, W) \
                or (W > 1 and allowed.stride(2) != 1):
            raise ValueError(f"allowed: expected an int32 tensor of shape ({B}, {R}, {W}) with unit word stride on {dev}")
        mask_seq, mask_row = allowed.stride(0), allowed.stride(1)
        allowed_ptr = allowed.data_ptr()
    args = (_vec(history_len, torch.int32, B, dev, "history_len"), _vec(prompt_len, torch.int32, B, dev, "prompt_len"),
            _vec(repetition, torch.float32, B, dev, "repetition"), _vec(presence, torch.float32, B, dev, "presence"),
            _vec(frequency, torch.float32, B, dev, "frequency"))
    rows_ptr = _vec(row_count, torch.int32, B, dev, "row_count")
    out_stride = 0
    if out is None:
        out = torch.empty((B, R, V), dtype=dtype, device=dev)
    else:
        if out.dtype != dtype or out.device != dev or out.shape != logits.shape:
            raise ValueError("out must match logits in dtype, device and shape")
        out_stride = _seq_stride(out, "out")
    _launch(dev, lib().sv_adjust_logits, logits.data_ptr(), stride, out.data_ptr(), out_stride, _DTYPE_CODE[dtype],
            tokens_ptr, tokens_stride, par, rows_ptr, B, R, V, history_ptr, history_stride, cap, *args,
            bias_ptr, values_ptr, n_bias, allowed_ptr, mask_seq, mask_row)
    return out


def lmhead_quant_workspace(M, K, V, group, device):
    """A workspace for lmhead_quant calls of these sizes, or None where they need none."""
    nbytes = int(lib().sv_lmhead_quant_workspace(M, K, V, group))
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def lmhead_quant(hidden, weights, scales, zeros=None, *, out_dtype=torch.float32, out=None, ws=None):
    """Logits from hidden states on 4-bit weights with group scales:
    sv_lmhead_quant.  hidden (..., K) bf16 or fp16; weights (V, K / 2) uint8,
    scales (V, K / group) of hidden's dtype, zeros (V, K / group) uint8 or None.
    Returns (..., V) logits of out_dtype (float32 or hidden's dtype), or fills
    out.  ws: a lmhead_quant_workspace, for more than 32 rows."""
    dtype, dev = hidden.dtype, hidden.device
    if (dtype != torch.bfloat16 and dtype != torch.float16) or dev.type != "cuda" or hidden.dim() < 1:
        raise ValueError("hidden: expected a bf16 or fp16 device tensor")
    K, lead = hidden.shape[-1], hidden.shape[:-1]
    if weights.dtype != torch.uint8 or weights.device != dev or weights.dim() != 2 or 2 * weights.shape[1] != K \
            or not weights.is_contiguous():
        raise ValueError(f"weights: expected a contiguous uint8 tensor of shape (V, {K // 2}) on {dev}")
    V = weights.shape[0]
    if scales.dtype != dtype or scales.device != dev or scales.dim() != 2 or scales.shape[0] != V \
            or scales.shape[1] < 1 or K % scales.shape[1] or not scales.is_contiguous():
        raise ValueError(f"scales: expected a contiguous {dtype} tensor of shape ({V}, {K} / group) on {dev}")
    if zeros is not None and (zeros.dtype != torch.uint8 or zeros.device != dev or zeros.shape != scales.shape
                              or not zeros.is_contiguous()):
        raise ValueError(f"zeros: expected a contiguous uint8 tensor of shape {tuple(scales.shape)} on {dev}")
    if out is None:
        if out_dtype != torch.float32 and out_dtype != dtype:
            raise ValueError(f"out_dtype: expected float32 or {dtype}")
        out = torch.empty((*lead, V), dtype=out_dtype, device=dev)
    elif (out.dtype != torch.float32 and out.dtype != dtype) or out.device != dev or out.shape != (*lead, V) \
            or not out.is_contiguous():
        raise ValueError(f"out: expected a contiguous float32 or {dtype} tensor of shape {(*lead, V)} on {dev}")
    M = out.numel() // V if V else 0
    if M == 0:
        return out
    try:
        rows = hidden if hidden.dim() == 2 else hidden.view(M, K)
    except RuntimeError:
        raise ValueError("hidden: rows must be one stride apart") from None
    if rows.stride(1) != 1 or (M > 1 and rows.stride(0) < K):
        raise ValueError("hidden: rows must be contiguous and not overlap")
    group = K // scales.shape[1]
    if ws is None and M > 32:
        ws = lmhead_quant_workspace(M, K, V, group, dev)
    ws_bytes = 0 if ws is None else _ws_bytes(ws, dev)
    _launch(dev, lib().sv_lmhead_quant, rows.data_ptr(), rows.stride(0) if M > 1 else 0, _DTYPE_CODE[dtype],
            weights.data_ptr(), scales.data_ptr(), None if zeros is None else zeros.data_ptr(),
            M, K, V, group, out.data_ptr(), 0, _DTYPE_CODE[out.dtype], None if ws is None else ws.data_ptr(), ws_bytes)
    return out


@dataclass
class AttentionResult:
    out: torch.Tensor
    lse: Optional[torch.Tensor] = None


def attention_workspace(B, R, Hq, Hkv, D, P, max_ctx, device):
    """A workspace for attention calls of these sizes."""
    nbytes = int(lib().sv_attention_workspace(B, R, Hq, Hkv, D, P, max_ctx))
    if nbytes == 0:
        raise ValueError("invalid sizes for an attention workspace")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _keys_values(k, v, dtype, dev, H, D, name):
    """Strides of a pair of (..., tokens, H, D) tensors with dense heads."""
    if k.dtype != dtype or v.dtype != dtype or k.device != dev or v.device != dev or k.shape != v.shape:
        raise ValueError(f"{name}: expected two {dtype} tensors of one shape on {dev}")
    if k.shape[-2:] != (H, D):
        raise ValueError(f"{name}: expected heads of shape ({H}, {D}), got {tuple(k.shape[-2:])}")
    st = k.stride()
    if v.stride() != st:
        raise ValueError(f"{name}: keys and values must have the same strides")
    if st[-1] != 1 or (H > 1 and st[-2] != D) or (k.shape[-3] > 1 and st[-3] < H * D):
        raise ValueError(f"{name}: the heads of a token must be contiguous, tokens not overlapping")
    return st


def attention(q, k_cache, v_cache, ctx_len, *, prefix_k=None, prefix_v=None, parent=None, row_count=None,
              scale=None, max_ctx=None, return_lse=False, out=None, ws=None):
    """Attention of a window's or tree's rows over a shared prefix, the cached
    context and the rows' ancestors: sv_attention.

    q (B, R, Hq, D); k_cache, v_cache (B, cap, Hkv, D) with ctx_len[b]
    committed tokens followed by the step's R rows; prefix_k, prefix_v (P, Hkv,
    D) or None.  parent (a host sequence) makes the rows a tree.  scale defaults
    to D ** -0.5, max_ctx (an upper bound of ctx_len) to cap - R.  out: an
    AttentionResult to fill."""
    dtype, dev = q.dtype, q.device
    if q.dim() != 4 or (dtype != torch.bfloat16 and dtype != torch.float16) or dev.type != "cuda":
        raise ValueError("q: expected a bf16 or fp16 device tensor of shape (B, R, Hq, D)")
    B, R, Hq, D = q.shape
    qs = q.stride()
    if qs[3] != 1 or (Hq > 1 and qs[2] != D):
        raise ValueError("q: the heads of a row must be contiguous")
    q_stride = qs[1] if R > 1 else qs[0] if B > 1 else 0
    if (B > 1 and R > 1 and qs[0] != R * q_stride) or (B * R > 1 and q_stride < Hq * D):
        raise ValueError("q: rows must be one stride apart and not overlap")
    if k_cache.dim() != 4 or k_cache.shape[0] != B:
        raise ValueError(f"k_cache: expected shape ({B}, cap, Hkv, {D}), got {tuple(k_cache.shape)}")
    cap, Hkv = k_cache.shape[1], k_cache.shape[2]
    st = _keys_values(k_cache, v_cache, dtype, dev, Hkv, D, "k_cache and v_cache")
    if Hkv < 1 or Hq % Hkv:
        raise ValueError("the query heads must be a multiple of the kv heads")
    seq_stride, tok_stride = st[0] if B > 1 else 0, st[1] if cap > 1 else 0
    if B > 1 and seq_stride <= 0:
        raise ValueError("k_cache and v_cache: sequences overlap")
    P = prefix_stride = 0
    pk = pv = None
    if (prefix_k is None) != (prefix_v is None):
        raise ValueError("prefix_k and prefix_v go together")
    if prefix_k is not None:
        if prefix_k.dim() != 3:
            raise ValueError(f"prefix_k: expected shape (P, {Hkv}, {D}), got {tuple(prefix_k.shape)}")
        P = prefix_k.shape[0]
        prefix_st = _keys_values(prefix_k, prefix_v, dtype, dev, Hkv, D, "prefix_k and prefix_v")
        if P > 0:
            prefix_stride = prefix_st[0] if P > 1 else 0
            pk, pv = prefix_k.data_ptr(), prefix_v.data_ptr()
    if ctx_len is None:
        raise ValueError("ctx_len is required")
    len_ptr = _vec(ctx_len, torch.int32, B, dev, "ctx_len")
    rows_ptr = _vec(row_count, torch.int32, B, dev, "row_count")
    par = _parents(parent, R)
    if max_ctx is None:
        max_ctx = cap - R
    if scale is None:
        scale = D ** -0.5
    L = lib()
    if ws is None:
        ws_bytes = L.sv_attention_workspace(B, R, Hq, Hkv, D, P, max_ctx)
        if ws_bytes == 0:
            raise ValueError("sizes outside the rules of sv_attention")
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    else:
        ws_bytes = _ws_bytes(ws, dev)
    if out is None:
        out = AttentionResult(torch.empty((B, R, Hq, D), dtype=dtype, device=dev),
                              torch.empty((B, R, Hq), dtype=torch.float32, device=dev) if return_lse else None)
    else:
        if out.out is None:
            raise ValueError("out is a required output")
        _out_tensor(out.out, dtype, (B, R, Hq, D), dev, "out")
        _out_tensor(out.lse, torch.float32, (B, R, Hq), dev, "lse")
    _launch(dev, L.sv_attention, q.data_ptr(), q_stride, _DTYPE_CODE[dtype], k_cache.data_ptr(), v_cache.data_ptr(),
            seq_stride, tok_stride, cap, pk, pv, prefix_stride, P, len_ptr, rows_ptr, par, B, R, Hq, Hkv, D, max_ctx, scale,
            out.out.data_ptr(), None if out.lse is None else out.lse.data_ptr(), ws.data_ptr(), ws_bytes)
    return out


class PagedCache:
    """Pages of keys and values: sv_paged_cache of include/sv_cache.h.

    k, v (num_pages, page, Hkv, D) in any non-overlapping order with unit
    stride along D: bf16 or fp16, or float8_e4m3fn with k_scale, v_scale
    (num_pages, page / block, Hkv) float32, contiguous.  One more leading
    dimension on all of them holds the layers of a model, behind each other
    (layer(i) is one of them).  A handle on those tensors: they keep their
    storage while it is used.  paged_cache() allocates one."""
    __slots__ = ("k", "v", "k_scale", "v_scale", "layers", "layer_stride", "code", "page", "heads", "dim", "device", "args")

    def __init__(self, k, v, k_scale=None, v_scale=None):
        # (small calls are bound by the host: one comparison a property)
        dtype, dev, shape, st = k.dtype, k.device, k.shape, k.stride()
        code = _PAGE_CODE.get(dtype)
        if code is None or dev.type != "cuda" or len(shape) not in (4, 5):
            raise ValueError("k: expected a bf16, fp16 or float8_e4m3fn device tensor of shape (num_pages, page, Hkv, D), or (layers, ..)")
        if v.dtype != dtype or v.device != dev or v.shape != shape or v.stride() != st:
            raise ValueError("v must match k in dtype, device, shape and strides")
        if len(shape) == 4:
            num_pages, page, Hkv, D = shape
            page_stride, token_stride, head_stride, unit = st
            self.layers = self.layer_stride = 0
        else:
            self.layers, num_pages, page, Hkv, D = shape
            self.layer_stride, page_stride, token_stride, head_stride, unit = st
            if self.layers > 1 and self.layer_stride <= 0:
                raise ValueError("k and v: layers overlap")
        if unit != 1:
            raise ValueError("k and v: the values of a head must be contiguous")
        if 0 in shape:
            raise ValueError("k and v: expected pages")
        # (the library takes a stride of zero for a dense one)
        if token_stride <= 0 or (num_pages > 1 and page_stride <= 0) or (Hkv > 1 and head_stride <= 0):
            raise ValueError("k and v: pages, tokens or heads overlap")
        block, ks, vs = 0, 0, 0
        if code == SV_DT_F8E4M3:
            blocks = k_scale.shape[-2] if k_scale is not None and k_scale.dim() > 2 else 0
            want = (*shape[:-3], blocks, Hkv)
            if not 0 < blocks <= page or page % blocks or v_scale is None or k_scale.shape != want or v_scale.shape != want \
                    or k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32 or k_scale.device != dev or v_scale.device != dev \
                    or not k_scale.is_contiguous() or not v_scale.is_contiguous():
                raise ValueError(f"k_scale, v_scale: 8-bit pages need contiguous float32 tensors (.., num_pages, page / block, Hkv) on {dev}")
            block, ks, vs = page // blocks, k_scale.data_ptr(), v_scale.data_ptr()
        elif k_scale is not None or v_scale is not None:
            raise ValueError("16-bit pages have no scales")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.code, self.page, self.heads, self.dim, self.device = code, page, Hkv, D, dev
        # strides of dimensions of one entry do not matter (0: dense)
        self.args = PAGED_CACHE.pack(k.data_ptr(), v.data_ptr(), ks, vs, code, num_pages, page, block, Hkv, D,
                                     page_stride if num_pages > 1 else 0, token_stride, head_stride if Hkv > 1 else 0)

    def layer(self, i):
        """The pages of layer i, on the same memory."""
        if not 0 <= i < self.layers:
            raise IndexError(f"layer {i} of {self.layers}")
        return PagedCache(self.k[i], self.v[i], *(None if t is None else t[i] for t in (self.k_scale, self.v_scale)))


def paged_cache(num_pages, page, Hkv, D, dtype, device, *, block=None, layers=None):
    """A PagedCache of zeros, the tokens of a head and page contiguous.  dtype
    torch.float8_e4m3fn: with a scale for each `block` tokens (default: the
    page, 64 at most)."""
    lead = (num_pages,) if layers is None else (layers, num_pages)
    k, v = (torch.zeros((*lead, Hkv, page, D), dtype=dtype, device=device).transpose(-2, -3) for _ in range(2))
    if dtype != torch.float8_e4m3fn:
        return PagedCache(k, v)
    block = min(page, 64) if block is None else block
    return PagedCache(k, v, *(torch.zeros((*lead, page // block, Hkv), device=device) for _ in range(2)))


def rotary_frequencies(rot, base=10000.0, *, scaling=None, factor=1.0, trained=4096, fast=32.0, slow=1.0):
    """(inv_freq, magnitude) of rot turned values: radians per position, as a
    list of rot / 2 floats, and the factor on the turned values.

    scaling None: base ** (-2 i / rot).  For contexts `factor` times longer than
    the `trained` length: "linear" divides every frequency by factor, "base"
    raises the base by factor ** (rot / (rot - 2)) (the fastest pair stays, the
    slowest is divided by factor), "ramp" keeps the pairs that make more than
    `fast` turns within the trained length, divides those that make fewer than
    `slow` by factor, blends linearly in between, and scales the values by 0.1
    log(factor) + 1."""
    if rot < 2 or rot % 2 or base <= 0 or factor <= 0:
        raise ValueError("rot must be even and positive, base and factor positive")
    if scaling == "base":
        base *= factor ** (rot / (rot - 2)) if rot > 2 else factor
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    if scaling is None or scaling == "base":
        return f, 1.0
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling != "ramp":
        raise ValueError(f"unknown scaling {scaling!r}")
    if fast <= slow:
        raise ValueError("fast must exceed slow")
    keep = [min(max((trained * x / (2 * math.pi) - slow) / (fast - slow), 0.0), 1.0) for x in f]
    return [x * w + x / factor * (1 - w) for x, w in zip(f, keep)], (0.1 * math.log(factor) + 1 if factor > 1 else 1.0)


def rotary_turns(inv_freq, device):
    """The frequencies (a host sequence, radians per position) as rotary and
    cache_append take them, a device int64 tensor: sv_rotary_turns."""
    n = len(inv_freq)
    src, out = (ctypes.c_double * n)(*inv_freq), (ctypes.c_uint64 * n)()
    _check(lib().sv_rotary_turns(src, n, out))
    return torch.tensor([x - (1 << 64) if x >> 63 else x for x in out], dtype=torch.int64).to(device)


def _turns(turns, D, dev):
    """(address, turned values) of a frequency tensor, or (None, 0)."""
    if turns is None:
        return None, 0
    if turns.dtype != torch.int64 or turns.device != dev or turns.dim() != 1 or not turns.is_contiguous():
        raise ValueError(f"turns: expected a contiguous int64 tensor of shape (rot / 2,) on {dev}")
    return turns.data_ptr(), 2 * turns.shape[0]


def _rows(t, B, R, H, D, dtype, dev, name):
    """Row stride of a (B, R, H, D) tensor with dense heads and rows one stride apart (0 = dense)."""
    if t.dtype != dtype or t.device != dev or t.shape != (B, R, H, D):
        raise ValueError(f"{name}: expected a {dtype} tensor of shape ({B}, {R}, {H}, {D}) on {dev}, got {t.dtype} {tuple(t.shape)}")
    s0, s1, s2, s3 = t.stride()
    if s3 != 1 or (H > 1 and s2 != D):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    row = s1 if R > 1 else s0 if B > 1 else 0
    if (B > 1 and R > 1 and s0 != R * row) or (B * R > 1 and row < H * D):
        raise ValueError(f"{name}: rows must be one stride apart and not overlap")
    return row


def rotary(x, turns, base_pos=None, *, parent=None, interleaved=False, magnitude=1.0, inverse=False, row_count=None, out=None):
    """Rows turned to their positions: sv_rotary.

    x (B, R, H, D) float32, bf16 or fp16; turns: rotary_turns of the pairs'
    frequencies, (rot / 2,) int64.  Row r stands at base_pos[b] + r, or with
    parent (a host sequence) at base_pos[b] + its depth; base_pos (B,) int64 or
    None (0).  inverse turns back: with the same magnitude, the gradient, which the
    caller's backward pass asks for.  out: a tensor like x (x itself: in place), a
    new one when None."""
    dtype, dev = x.dtype, x.device
    if x.dim() != 4 or dtype not in _DTYPE_CODE or dev.type != "cuda":
        raise ValueError("x: expected a float32, bf16 or fp16 device tensor of shape (B, R, H, D)")
    B, R, H, D = x.shape
    stride = _rows(x, B, R, H, D, dtype, dev, "x")
    if turns is None:
        raise ValueError("turns is required")
    turns_ptr, rot = _turns(turns, D, dev)
    if out is None:
        out, out_stride = torch.empty((B, R, H, D), dtype=dtype, device=dev), 0
    else:
        out_stride = _rows(out, B, R, H, D, dtype, dev, "out")
    _launch(dev, lib().sv_rotary, x.data_ptr(), stride, out.data_ptr(), out_stride, _DTYPE_CODE[dtype], turns_ptr, rot,
            bool(interleaved), bool(inverse), magnitude, _vec(base_pos, torch.int64, B, dev, "base_pos"),
            _vec(row_count, torch.int32, B, dev, "row_count"), _parents(parent, R), B, R, H, D)
    return out


def _one_layer(cache, dtype, dev):
    """Refuses caches on another device, of several layers, or of 16-bit pages of another type than dtype."""
    if cache.device != dev:
        raise ValueError(f"cache is on {cache.device}, expected {dev}")
    if cache.layers:
        raise ValueError("cache: expected one layer (cache.layer(i))")
    if cache.code != SV_DT_F8E4M3 and cache.code != _DTYPE_CODE[dtype]:
        raise ValueError(f"16-bit pages hold {cache.k.dtype}, the rows are {dtype}")


def cache_append(cache, page_table, ctx_len, k, v, *, q=None, turns=None, base_pos=None, parent=None, interleaved=False,
                 magnitude=1.0, row_count=None, q_out=None):
    """Stores rows' keys, turned, and values in their sequences' pages, and turns
    their queries: sv_cache_append.

    cache: a PagedCache (one layer); page_table (B, pages) int32; row r becomes
    token ctx_len[b] + r.  k, v (B, R, Hkv, D) bf16 or fp16, q (B, R, Hq, D) or
    None (each may be a part of one projection's rows).  turns, base_pos, parent,
    interleaved, magnitude as in rotary (turns None: not turned; base_pos None:
    ctx_len; behind a prefix of P tokens that the batch shares it is P + ctx_len).
    Returns q_out (a new tensor when None; q itself: in place), or
    None without q."""
    dtype, dev = k.dtype, k.device
    if k.dim() != 4 or (dtype != torch.bfloat16 and dtype != torch.float16) or dev.type != "cuda":
        raise ValueError("k: expected a bf16 or fp16 device tensor of shape (B, R, Hkv, D)")
    _one_layer(cache, dtype, dev)
    B, R, Hkv, D = k.shape[0], k.shape[1], cache.heads, cache.dim
    k_stride, v_stride = _rows(k, B, R, Hkv, D, dtype, dev, "k"), _rows(v, B, R, Hkv, D, dtype, dev, "v")
    table_stride = _rows_i32(page_table, B, 1, dev, "page_table")
    if ctx_len is None:
        raise ValueError("ctx_len is required")
    turns_ptr, rot = _turns(turns, D, dev)
    Hq = q_stride = out_stride = 0
    q_ptr = out_ptr = None
    if q is not None:
        Hq = q.shape[2] if q.dim() == 4 else 0
        q_stride = _rows(q, B, R, Hq, D, dtype, dev, "q")
        if q_out is None:
            q_out = torch.empty((B, R, Hq, D), dtype=dtype, device=dev)
        else:
            out_stride = _rows(q_out, B, R, Hq, D, dtype, dev, "q_out")
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out needs q")
    _launch(dev, lib().sv_cache_append, cache.args, page_table.data_ptr(), table_stride, page_table.shape[1],
            _vec(ctx_len, torch.int32, B, dev, "ctx_len"), _vec(row_count, torch.int32, B, dev, "row_count"), _parents(parent, R),
            _vec(base_pos, torch.int64, B, dev, "base_pos"), k.data_ptr(), k_stride, v.data_ptr(), v_stride, q_ptr, q_stride,
            out_ptr, out_stride, _DTYPE_CODE[dtype], turns_ptr, rot, bool(interleaved), magnitude, B, R, Hq)
    return q_out


def cache_commit(cache, page_table, ctx_len, nodes, n_accepted, *, rows, new_len=None):
    """Moves an accepted path's keys and values behind the context, in all layers
    of the cache, and advances the lengths: sv_cache_commit.

    nodes, n_accepted: out_nodes and n_accepted of verify_tree (nodes None: a
    window, only the lengths); rows: the rows of the step.  Returns new_len (a
    new tensor when None; ctx_len itself: in place)."""
    dev = cache.device
    if ctx_len is None or n_accepted is None:
        raise ValueError("ctx_len and n_accepted are required")
    B = page_table.shape[0]
    table_stride = _rows_i32(page_table, B, 1, dev, "page_table")
    nodes_ptr, nodes_stride, most = None, 0, 0
    if nodes is not None and nodes.shape[-1] > 0:
        nodes_stride = _rows_i32(nodes, B, 1, dev, "nodes")
        nodes_ptr, most = nodes.data_ptr(), nodes.shape[1]
    if new_len is None:
        new_len = torch.empty(B, dtype=torch.int32, device=dev)
    _launch(dev, lib().sv_cache_commit, cache.args, max(cache.layers, 1), cache.layer_stride if cache.layers > 1 else 0,
            page_table.data_ptr(), table_stride, page_table.shape[1], _vec(ctx_len, torch.int32, B, dev, "ctx_len"), nodes_ptr,
            nodes_stride, most, _vec(n_accepted, torch.int32, B, dev, "n_accepted"), B, rows,
            _vec(new_len, torch.int32, B, dev, "new_len"))
    return new_len


def paged_attention_workspace(B, R, Hq, Hkv, D, P, max_ctx, device):
    """A workspace for paged_attention calls of these sizes."""
    nbytes = int(lib().sv_paged_attention_workspace(B, R, Hq, Hkv, D, P, max_ctx))
    if nbytes == 0:
        raise ValueError("invalid sizes for an attention workspace")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def paged_attention(q, cache, page_table, ctx_len, *, prefix_table=None, prefix_len=0, parent=None, row_count=None,
                    scale=None, max_ctx=None, return_lse=False, out=None, ws=None):
    """Attention of a window's or tree's rows over paged caches: sv_paged_attention.

    As attention(), with keys and values in the pages of cache (a PagedCache, one
    layer): page_table (B, pages) int32 for the sequences' own tokens, prefix_table
    (ceil(prefix_len / page),) int32 for the prefix_len tokens in front that all
    share.  max_ctx defaults to the table's room for a context."""
    dtype, dev = q.dtype, q.device
    if q.dim() != 4 or (dtype != torch.bfloat16 and dtype != torch.float16) or dev.type != "cuda":
        raise ValueError("q: expected a bf16 or fp16 device tensor of shape (B, R, Hq, D)")
    _one_layer(cache, dtype, dev)
    B, R, Hq, D = q.shape
    q_stride = _rows(q, B, R, Hq, cache.dim, dtype, dev, "q")
    if Hq % cache.heads:
        raise ValueError("the query heads must be a multiple of the kv heads")
    table_stride = _rows_i32(page_table, B, 1, dev, "page_table")
    prefix_ptr = None
    if prefix_len:
        if prefix_table is None or prefix_table.dtype != torch.int32 or prefix_table.device != dev or prefix_table.dim() != 1 \
                or not prefix_table.is_contiguous() or prefix_table.shape[0] * cache.page < prefix_len:
            raise ValueError(f"prefix_table: expected a contiguous int32 tensor of the {prefix_len} tokens' pages on {dev}")
        prefix_ptr = prefix_table.data_ptr()
    if ctx_len is None:
        raise ValueError("ctx_len is required")
    if max_ctx is None:
        max_ctx = min(page_table.shape[1] * cache.page - R, 1 << 24)
    if scale is None:
        scale = D ** -0.5
    L = lib()
    if ws is None:
        ws_bytes = L.sv_paged_attention_workspace(B, R, Hq, cache.heads, D, prefix_len, max_ctx)
        if ws_bytes == 0:
            raise ValueError("sizes outside the rules of sv_paged_attention")
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    else:
        ws_bytes = _ws_bytes(ws, dev)
    if out is None:
        out = AttentionResult(torch.empty((B, R, Hq, D), dtype=dtype, device=dev),
                              torch.empty((B, R, Hq), dtype=torch.float32, device=dev) if return_lse else None)
    else:
        if out.out is None:
            raise ValueError("out is a required output")
        _out_tensor(out.out, dtype, (B, R, Hq, D), dev, "out")
        _out_tensor(out.lse, torch.float32, (B, R, Hq), dev, "lse")
    _launch(dev, L.sv_paged_attention, q.data_ptr(), q_stride, _DTYPE_CODE[dtype], cache.args, page_table.data_ptr(), table_stride,
            page_table.shape[1], prefix_ptr, prefix_len, _vec(ctx_len, torch.int32, B, dev, "ctx_len"),
            _vec(row_count, torch.int32, B, dev, "row_count"), _parents(parent, R), B, R, Hq, max_ctx, scale,
            out.out.data_ptr(), None if out.lse is None else out.lse.data_ptr(), ws.data_ptr(), ws_bytes)
    return out


def rollback(buf_tokens, buf_len, stage, verified, verified_len, *, len_offset=0):
    """Per-stage buffer rollback: sv_rollback (in place on buf_tokens/buf_len).
    Row s of `verified` must hold at least verified_len[s] + len_offset tokens
    (at most cap are read); that length lives on the device and is not checked here."""
    S, K, cap = buf_tokens.shape
    _i32(buf_tokens, (S, K, cap), "buf_tokens")
    _i32(buf_len, (S, K), "buf_len")
    if verified.dtype != torch.int32 or not verified.is_cuda or verified.dim() != 2 \
            or verified.shape[0] != S or verified.stride(1) != 1:
        raise ValueError("verified: expected an int32 device tensor (S, >=L) with unit column stride")
    _i32(verified_len, (S,), "verified_len")
    dev = buf_tokens.device
    _same_device(dev, buf_len=buf_len, verified=verified, verified_len=verified_len)
    with torch.cuda.device(dev):
        _check(lib().sv_rollback(
            _ptr(buf_tokens), _ptr(buf_len), S, K, cap, stage,
            _ptr(verified), verified.stride(0), _ptr(verified_len), len_offset, _stream(dev)))


def probe_read(buf, sink=None):
    """Streams buf through the library's read-bandwidth probe kernel.  buf is
    read as one contiguous byte range; sink takes one 32-bit word per
    workgroup (sv_probe_blocks of the byte count)."""
    if not buf.is_cuda or not buf.is_contiguous():
        raise ValueError("buf: expected a contiguous device tensor")
    nbytes = buf.numel() * buf.element_size()
    nb = int(lib().sv_probe_blocks(nbytes))
    if sink is None:
        sink = torch.empty(nb, dtype=torch.int32, device=buf.device)
    elif (sink.dtype not in (torch.int32, torch.uint32) or sink.device != buf.device
          or not sink.is_contiguous() or sink.numel() < nb):
        raise ValueError(f"sink: expected a contiguous 32-bit tensor of at least {nb} entries on {buf.device}")
    with torch.cuda.device(buf.device):
        _check(lib().sv_probe_read(_ptr(buf), nbytes, _ptr(sink), _stream(buf.device)))
    return sink
