"""The serving operators around the draft head (include/lmhead.h, "Serving
operators around the head").

    plan = page_plan(lens, new_lens, table, free_pages, free_count, P, max_tokens)
    o = chunk_attention(q, k_cache, v_cache, table, lens, plan.cu, k=k, v=v, slots=plan.slots,
                        granted=plan.granted)
    logits = q4_gather_logits(codes, scales, h, ids, group)
    parent, token, score = beam_select(logits, scores, beams, k, ids=ids)
    h, table = beam_reorder(parent, [h, table], beams)

Codes and scales of a 4-bit head come from prep.quantise_rows.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional, Sequence

import torch

from ._lib import check, load
from ._memory import result, scratch, stream_handle

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


# the current device's index without torch.cuda's checks around it
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


class PagePlan(NamedTuple):
    slots: torch.Tensor
    positions: torch.Tensor
    cu: torch.Tensor
    granted: torch.Tensor
    free_left: torch.Tensor


# Every call of these operators is a few microseconds of GPU work at its
# smallest, so the checks before it are written to cost little: one comparison
# chain a tensor, messages built only when they are raised.

def _wrong(t: torch.Tensor, dtype, shape, device, name: str) -> Exception:
    if t.dtype != dtype or not t.is_contiguous():
        return TypeError(f"{name}: expected a contiguous {dtype} tensor, got {t.dtype} "
                         f"(contiguous={t.is_contiguous()})")
    return ValueError(f"{name}: expected shape {tuple(shape)} on {device}, got {tuple(t.shape)} "
                      f"on {t.device}")


def _dense(t: Optional[torch.Tensor], dtype, shape, device, name: str) -> int:
    """The address of a contiguous tensor of this type, shape and device."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise _wrong(t, dtype, shape, device, name)
    return t.data_ptr()


def _cuda(t: torch.Tensor, name: str) -> torch.device:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA tensor")
    # launches, the error word and the library's per-device state are the current
    # device's: another device's stream and addresses must not meet them
    if t.device.index != _current_device():
        raise ValueError(f"{name}: on {t.device}, which is not the current device")
    return t.device


def page_plan(lens: torch.Tensor, new_lens: torch.Tensor, table: torch.Tensor,
              free_pages: torch.Tensor, free_count: torch.Tensor, page_size: int, max_tokens: int,
              out: Optional[PagePlan] = None, stream=None) -> PagePlan:
    """Pages and slots of every request's new tokens; `table` (S x width) is
    filled in place. Returns PagePlan(slots, positions, cu, granted, free_left),
    int32 (see lmhead_page_plan)."""
    dev = _cuda(lens, "lens")
    i32 = torch.int32
    if lens.dim() != 1 or table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("lens, table, free_pages: expected requests, requests x pages and pages")
    S, width, cap = lens.shape[0], table.shape[1], free_pages.shape[0]
    if out is None:
        if max_tokens < 1 or S < 1:
            raise ValueError("max_tokens: must be positive, as must the number of requests")
        # one allocation, its parts one behind the other
        buf = result(2 * max_tokens + 2 * S + 2, i32, dev, stream)
        at = buf.data_ptr()
        ptrs = (at, at + 4 * max_tokens, at + 8 * max_tokens, at + 8 * max_tokens + 4 * (S + 1),
                at + 8 * max_tokens + 4 * (2 * S + 1))
        out = PagePlan(*buf.split_with_sizes((max_tokens, max_tokens, S + 1, S, 1)))
    else:
        slots, positions, cu, granted, free_left = out
        ptrs = (_dense(slots, i32, (max_tokens,), dev, "slots"),
                _dense(positions, i32, (max_tokens,), dev, "positions"),
                _dense(cu, i32, (S + 1,), dev, "cu"), _dense(granted, i32, (S,), dev, "granted"),
                _dense(free_left, i32, (1,), dev, "free_left"))
    check(load().lmhead_page_plan(
        _dense(lens, i32, (S,), dev, "lens"), _dense(new_lens, i32, (S,), dev, "new_lens"), S,
        _dense(table, i32, (S, width), dev, "table"), width,
        _dense(free_pages, i32, (cap,), dev, "free_pages"), cap,
        _dense(free_count, i32, (1,), dev, "free_count"), page_size, max_tokens, *ptrs,
        stream_handle(stream, dev)), "page_plan")
    return out


@functools.lru_cache(maxsize=4096)
def _attention_bytes(device, S: int, T: int, heads: int, kv_heads: int, dim: int) -> int:
    with torch.cuda.device(device):
        return int(load().lmhead_chunk_attention_workspace_size(S, T, heads, kv_heads, dim))


def _heads_tensor(t: torch.Tensor, dtype, shape, device, name: str):
    """Address and strides (elements) of a tensor whose last dimension alone
    has to be contiguous."""
    st = t.stride()
    if t.dtype is not dtype or st[-1] != 1:
        raise TypeError(f"{name}: expected {dtype} with a contiguous last dimension, got {t.dtype} "
                        f"with strides {st}")
    if t.shape != shape or t.device != device:
        raise _wrong(t, dtype, shape, device, name) if t.is_contiguous() else ValueError(
            f"{name}: expected shape {tuple(shape)} on {device}, got {tuple(t.shape)} on {t.device}")
    return (t.data_ptr(),) + st[:-1]


def chunk_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    table: torch.Tensor, lens: torch.Tensor, cu: torch.Tensor,
                    k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None,
                    slots: Optional[torch.Tensor] = None, tree: Optional[torch.Tensor] = None,
                    window: int = 0, scale: Optional[float] = None, with_lse: bool = False,
                    workspace=None, out=None, stream=None,
                    granted: Optional[torch.Tensor] = None):
    """Attention of T new tokens (q: T x heads x dim) over the paged caches
    (pages x page_size x kv_heads x dim, any strides with dim contiguous), after
    writing k and v (T x kv_heads x dim) to `slots`, if given. lens: tokens
    cached before; cu: starts of the requests' tokens. Causal within a request,
    over the last `window` keys if window > 0, or by `tree` (int64 bits of the
    new tokens each new token sees, besides all cached ones). granted: a plan's (0:
    the request was refused; its rows are zero, its lse -inf). Returns out, or
    (out, lse) with with_lse or when `out` is such a pair (see
    lmhead_chunk_attention)."""
    dev = _cuda(q, "q")
    if q.dim() != 3 or k_cache.dim() != 4 or table.dim() != 2:
        raise ValueError("q, k_cache, table: expected tokens x heads x dim, pages x page_size x "
                         "kv_heads x dim and requests x pages")
    T, heads, dim = q.shape
    pages, P, kv_heads, _ = k_cache.shape
    dt = q.dtype
    if dt not in (torch.bfloat16, torch.float16):
        raise TypeError(f"q: expected bf16 or fp16, got {dt}")
    S, width = table.shape
    cache = (pages, P, kv_heads, dim)
    qa, q_tok, q_head = _heads_tensor(q, dt, (T, heads, dim), dev, "q")
    kca, kc_page, kc_tok, kc_head = _heads_tensor(k_cache, dt, cache, dev, "k_cache")
    vca, vc_page, vc_tok, vc_head = _heads_tensor(v_cache, dt, cache, dev, "v_cache")
    ka = va = k_tok = k_head = v_tok = v_head = 0
    if k is not None or v is not None:
        if k is None or v is None or slots is None:
            raise ValueError("k, v, slots: are given together")
        ka, k_tok, k_head = _heads_tensor(k, dt, (T, kv_heads, dim), dev, "k")
        va, v_tok, v_head = _heads_tensor(v, dt, (T, kv_heads, dim), dev, "v")
    # the stride of a dimension of one means nothing
    if kv_heads == 1:
        kc_head = vc_head = k_head = v_head = 0
    if pages == 1:
        kc_page, vc_page = max(kc_page, dim), max(vc_page, dim)
    if T == 1:
        q_tok = k_tok = v_tok = 0
    if heads == 1:
        q_head = 0
    o, lse = out if isinstance(out, (tuple, list)) else (out, None)
    if o is None:
        o = result((T, heads, dim), dt, dev, stream)
    if lse is None and with_lse:
        lse = result((T, heads), torch.float32, dev, stream)
    if slots is not None and slots.shape[0] != T:
        # a plan's buffers may be longer than the step's tokens
        if slots.dim() != 1 or slots.shape[0] < T:
            raise ValueError("slots: expected a slot per token")
        slots = slots[:T]
    i32 = torch.int32
    ws = scratch(workspace, _attention_bytes(dev, S, T, heads, kv_heads, dim), dev, stream)
    check(load().lmhead_chunk_attention_granted(
        _DTYPES[dt], qa, q_tok, q_head, ka, k_tok, k_head, va, v_tok, v_head, kca, kc_page, kc_tok,
        kc_head, vca, vc_page, vc_tok, vc_head, pages, P,
        _dense(table, i32, (S, width), dev, "table"), width, _dense(lens, i32, (S,), dev, "lens"),
        _dense(cu, i32, (S + 1,), dev, "cu"), _dense(granted, i32, (S,), dev, "granted"),
        _dense(slots, i32, (T,), dev, "slots"),
        _dense(tree, torch.int64, (T,), dev, "tree"), S, T, heads, kv_heads, dim, window,
        dim ** -0.5 if scale is None else scale, _dense(o, dt, (T, heads, dim), dev, "out"),
        _dense(lse, torch.float32, (T, heads), dev, "lse"), ws.data_ptr(), ws.numel(),
        stream_handle(stream, dev)), "chunk_attention")
    return o if lse is None else (o, lse)


def _q4(name, codes, scales, h, ids, group, mins, out, stream):
    dev = _cuda(h, "h")
    dt = h.dtype
    if dt not in (torch.bfloat16, torch.float16):
        raise TypeError(f"h: expected bf16 or fp16, got {dt}")
    if h.dim() != 2 or codes.dim() != 2 or (ids is not None and ids.dim() != 2):
        raise ValueError("h, codes, ids: expected vectors x d, rows x d/2 and vectors x candidates")
    M, d = h.shape
    n = codes.shape[0]
    if group not in (32, 64, 128) or d % group or d < group:
        raise ValueError(f"group: must be 32, 64 or 128 and divide d = {d}, got {group}")
    K = n if ids is None else ids.shape[1]
    if out is None:
        out = result((M, K), torch.float32, dev, stream)
    args = [_DTYPES[dt], _dense(codes, torch.uint8, (n, d // 2), dev, "codes"),
            _dense(scales, dt, (n, d // group), dev, "scales"),
            _dense(mins, dt, (n, d // group), dev, "mins"), _dense(h, dt, (M, d), dev, "h")]
    o = _dense(out, torch.float32, (M, K), dev, "out")
    if ids is None:
        check(load().lmhead_q4_head(*args, n, d, group, M, o, stream_handle(stream, dev)), name)
    else:
        check(load().lmhead_q4_gather_logits(
            *args, _dense(ids, torch.int32, (M, K), dev, "ids"), n, d, group, M, K, o,
            stream_handle(stream, dev)), name)
    return out


def q4_head(codes: torch.Tensor, scales: torch.Tensor, h: torch.Tensor, group: int,
            mins: Optional[torch.Tensor] = None, workspace=None,
            out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Logits (M x n, fp32) of every row of a 4-bit head: codes n x d/2 uint8,
    scales (and mins) n x d/group of h's type (see lmhead_q4_head). Needs no
    scratch: `workspace` is taken like the other heads' and left alone."""
    return _q4("q4_head", codes, scales, h, None, group, mins, out, stream)


def q4_gather_logits(codes: torch.Tensor, scales: torch.Tensor, h: torch.Tensor,
                     ids: torch.Tensor, group: int, mins: Optional[torch.Tensor] = None,
                     workspace=None, out: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """Exact logits (M x K, fp32) of the candidate rows ids (M x K) of a 4-bit
    head (see lmhead_q4_gather_logits); `workspace` as for q4_head."""
    return _q4("q4_gather_logits", codes, scales, h, ids, group, mins, out, stream)


@functools.lru_cache(maxsize=4096)
def _beam_bytes(device, S: int, beams: int, n: int, k: int) -> int:
    with torch.cuda.device(device):
        return int(load().lmhead_beam_workspace_size(S, beams, n, k))


def beam_select(logits: torch.Tensor, scores: torch.Tensor, beams: int, k: int,
                ids: Optional[torch.Tensor] = None, finished: Optional[torch.Tensor] = None,
                eos: int = -1, workspace=None, out=None, stream=None):
    """The k best continuations of each sequence over its beams' rows of logits
    (S*beams x n, rows may be strided): (parent, token, score), each S x k.
    scores: S*beams fp32 log-probabilities so far; ids: the entries' tokens;
    finished: bool, beams that have ended (see lmhead_beam_select)."""
    dev = _cuda(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits: expected beams x entries")
    if logits.dtype not in _DTYPES:
        raise TypeError(f"logits: expected bf16, fp16 or fp32, got {logits.dtype}")
    rows, n = logits.shape
    if beams < 1 or rows < 1 or rows % beams or n < 1:
        raise ValueError(f"beams: {beams} does not divide {rows} rows of {n} entries")
    if not 1 <= k <= 32:
        raise ValueError("k: must be 1 to 32")
    stride, one = logits.stride()
    if one != 1 and n > 1:
        raise TypeError("logits: expected contiguous rows")
    if rows == 1:
        stride = n
    elif stride < n:
        raise ValueError("logits: rows overlap")
    S = rows // beams
    i32 = torch.int32
    if out is None:
        parent, token = result((S, k), i32, dev, stream), result((S, k), i32, dev, stream)
        score = result((S, k), torch.float32, dev, stream)
        ptrs = (parent.data_ptr(), token.data_ptr(), score.data_ptr())
    else:
        parent, token, score = out
        ptrs = (_dense(parent, i32, (S, k), dev, "parent"), _dense(token, i32, (S, k), dev, "token"),
                _dense(score, torch.float32, (S, k), dev, "score"))
    ws = scratch(workspace, _beam_bytes(dev, S, beams, n, k), dev, stream)
    # a bool is a byte
    kind = torch.uint8 if finished is None or finished.dtype is torch.uint8 else torch.bool
    check(load().lmhead_beam_select(
        _DTYPES[logits.dtype], logits.data_ptr(), stride,
        _dense(scores, torch.float32, (rows,), dev, "scores"),
        _dense(ids, i32, (rows, n), dev, "ids"),
        _dense(finished, kind, (rows,), dev, "finished"), S, beams, n, k, eos, *ptrs,
        ws.data_ptr(), ws.numel(), stream_handle(stream, dev)), "beam_select")
    return parent, token, score


_Table = ctypes.c_int64 * 24  # up to 8 sources, destinations and sizes


def beam_reorder(parent: torch.Tensor, states: Sequence[torch.Tensor], beams: int, out=None,
                 stream=None):
    """Each state tensor (S*beams rows of any type, contiguous) by the parents
    chosen (S x k): a list of tensors of S*k rows, zeros where parent is -1."""
    dev = _cuda(parent, "parent")
    if parent.dim() != 2 or parent.numel() == 0:
        raise ValueError("parent: expected sequences x k")
    S, k = parent.shape
    n, rows = len(states), S * beams
    if not 1 <= n <= 8 or beams < 1:
        raise ValueError("states, beams: expected 1 to 8 tensors and a positive number of beams")
    if out is not None and len(out) != n:
        raise ValueError("out: expected one tensor per state")
    res, table = [], _Table()
    for i, t in enumerate(states):
        shape, dt = t.shape, t.dtype
        if t.dim() < 1 or shape[0] != rows or t.device != dev or not t.is_contiguous():
            raise ValueError(f"states[{i}]: expected {rows} contiguous rows on {dev}")
        want = (S * k, *shape[1:])
        o = out[i] if out is not None else result(want, dt, dev, stream)
        res.append(o)
        table[i] = t.data_ptr()
        table[8 + i] = _dense(o, dt, want, dev, "out") if out is not None else o.data_ptr()
        table[16 + i] = t.numel() // rows * t.element_size()
    at = ctypes.addressof(table)
    check(load().lmhead_beam_reorder(
        _dense(parent, torch.int32, (S, k), dev, "parent"), S, beams, k, n, at, at + 64, at + 128,
        stream_handle(stream, dev)), "beam_reorder")
    return res
