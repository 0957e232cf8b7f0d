"""The serving operators around the draft head (include/lmhead.h, "Serving
operators around the head").

    plan = page_plan(lens, new_lens, table, free_pages, free_count, P, max_tokens)
    o = chunk_attention(q, k_cache, v_cache, table, lens, plan.cu, k=k, v=v, slots=plan.slots)
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

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class PagePlan(NamedTuple):
    slots: torch.Tensor
    positions: torch.Tensor
    cu: torch.Tensor
    granted: torch.Tensor
    free_left: torch.Tensor


def _need(ok: bool, name: str, what: str) -> None:
    if not ok:
        raise ValueError(f"{name}: {what}")


def _dense(t: Optional[torch.Tensor], dtype, shape, device, name: str) -> int:
    """The address of a contiguous tensor of this type, shape and device."""
    if t is None:
        return 0
    if t.dtype != dtype or not t.is_contiguous():
        raise TypeError(f"{name}: expected a contiguous {dtype} tensor, got {t.dtype} "
                        f"(contiguous={t.is_contiguous()})")
    if t.shape != shape or t.device != device:
        raise ValueError(f"{name}: expected shape {tuple(shape)} on {device}, got {tuple(t.shape)} "
                         f"on {t.device}")
    return t.data_ptr()


def _cuda(t: torch.Tensor, name: str) -> torch.device:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA tensor")
    return t.device


def _stream(stream, device) -> int:
    return (stream if stream is not None else torch.cuda.current_stream(device)).cuda_stream


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """A new tensor that the call's stream may use: one that is not the current
    stream has to be named to the allocator."""
    t = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None:
        t.record_stream(stream)
    return t


def _workspace(workspace, nbytes: int, device, stream) -> torch.Tensor:
    if workspace is None:
        return _empty(max(nbytes, 256), torch.uint8, device, stream)
    return workspace.get(nbytes, device) if hasattr(workspace, "get") else workspace


def page_plan(lens: torch.Tensor, new_lens: torch.Tensor, table: torch.Tensor,
              free_pages: torch.Tensor, free_count: torch.Tensor, page_size: int, max_tokens: int,
              out: Optional[PagePlan] = None, stream=None) -> PagePlan:
    """Pages and slots of every request's new tokens; `table` (S x width) is
    filled in place. Returns PagePlan(slots, positions, cu, granted, free_left),
    int32 (see lmhead_page_plan)."""
    dev = _cuda(lens, "lens")
    i32 = torch.int32
    _need(lens.dim() == 1, "lens", "expected one length per request")
    _need(table.dim() == 2, "table", "expected requests x pages")
    _need(free_pages.dim() == 1, "free_pages", "expected a list of page ids")
    S, width, cap = lens.shape[0], table.shape[1], free_pages.shape[0]
    if out is None:
        _need(max_tokens >= 1 and S >= 1, "max_tokens", "must be positive, as must the requests")
        buf = _empty(2 * max_tokens + 2 * S + 2, i32, dev, stream)
        out = PagePlan(*buf.split([max_tokens, max_tokens, S + 1, S, 1]))
    check(load().lmhead_page_plan(
        _dense(lens, i32, (S,), dev, "lens"), _dense(new_lens, i32, (S,), dev, "new_lens"), S,
        _dense(table, i32, (S, width), dev, "table"), width,
        _dense(free_pages, i32, (cap,), dev, "free_pages"), cap,
        _dense(free_count, i32, (1,), dev, "free_count"), page_size, max_tokens,
        _dense(out.slots, i32, (max_tokens,), dev, "slots"),
        _dense(out.positions, i32, (max_tokens,), dev, "positions"),
        _dense(out.cu, i32, (S + 1,), dev, "cu"), _dense(out.granted, i32, (S,), dev, "granted"),
        _dense(out.free_left, i32, (1,), dev, "free_left"), _stream(stream, dev)), "page_plan")
    return out


@functools.lru_cache(maxsize=4096)
def _attention_bytes(device, S: int, T: int, heads: int, kv_heads: int, dim: int) -> int:
    with torch.cuda.device(device):
        return int(load().lmhead_chunk_attention_workspace_size(S, T, heads, kv_heads, dim))


def _heads_tensor(t: torch.Tensor, dtype, shape, device, name: str):
    """Address and strides (elements) of a tensor whose last dimension alone
    has to be contiguous."""
    if t.dtype != dtype or t.stride(-1) != 1:
        raise TypeError(f"{name}: expected {dtype} with a contiguous last dimension, got {t.dtype} "
                        f"with strides {t.stride()}")
    if t.shape != shape or t.device != device:
        raise ValueError(f"{name}: expected shape {tuple(shape)} on {device}, got {tuple(t.shape)} "
                         f"on {t.device}")
    return (t.data_ptr(),) + t.stride()[:-1]


def chunk_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    table: torch.Tensor, lens: torch.Tensor, cu: torch.Tensor,
                    k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None,
                    slots: Optional[torch.Tensor] = None, tree: Optional[torch.Tensor] = None,
                    window: int = 0, scale: Optional[float] = None, with_lse: bool = False,
                    workspace=None, out=None, stream=None):
    """Attention of T new tokens (q: T x heads x dim) over the paged caches
    (pages x page_size x kv_heads x dim, any strides with dim contiguous), after
    writing k and v (T x kv_heads x dim) to `slots`, if given. lens: tokens
    cached before; cu: starts of the requests' tokens. Causal within a request,
    over the last `window` keys if window > 0, or by `tree` (int64 bits of the
    new tokens each new token sees, besides all cached ones). Returns out, or
    (out, lse) with with_lse or when `out` is such a pair (see
    lmhead_chunk_attention)."""
    dev = _cuda(q, "q")
    _need(q.dim() == 3, "q", "expected tokens x heads x dim")
    _need(k_cache.dim() == 4, "k_cache", "expected pages x page_size x kv_heads x dim")
    T, heads, dim = q.shape
    pages, P, kv_heads, _ = k_cache.shape
    dt = q.dtype
    if dt not in (torch.bfloat16, torch.float16):
        raise TypeError(f"q: expected bf16 or fp16, got {dt}")
    _need(table.dim() == 2, "table", "expected requests x pages")
    S, width = table.shape
    cache = (pages, P, kv_heads, dim)
    qa, q_tok, q_head = _heads_tensor(q, dt, (T, heads, dim), dev, "q")
    kca, kc_page, kc_tok, kc_head = _heads_tensor(k_cache, dt, cache, dev, "k_cache")
    vca, vc_page, vc_tok, vc_head = _heads_tensor(v_cache, dt, cache, dev, "v_cache")
    ka = va = k_tok = k_head = v_tok = v_head = 0
    if k is not None or v is not None:
        _need(k is not None and v is not None and slots is not None, "k, v, slots",
              "are given together")
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
        o = _empty((T, heads, dim), dt, dev, stream)
    if lse is None and with_lse:
        lse = _empty((T, heads), torch.float32, dev, stream)
    if slots is not None and slots.shape[0] != T:
        # a plan's buffers may be longer than the step's tokens
        _need(slots.dim() == 1 and slots.shape[0] > T, "slots", "expected a slot per token")
        slots = slots[:T]
    i32 = torch.int32
    ws = _workspace(workspace, _attention_bytes(dev, S, T, heads, kv_heads, dim), dev, stream)
    check(load().lmhead_chunk_attention(
        _DTYPES[dt], qa, q_tok, q_head, ka, k_tok, k_head, va, v_tok, v_head, kca, kc_page, kc_tok,
        kc_head, vca, vc_page, vc_tok, vc_head, pages, P,
        _dense(table, i32, (S, width), dev, "table"), width, _dense(lens, i32, (S,), dev, "lens"),
        _dense(cu, i32, (S + 1,), dev, "cu"), _dense(slots, i32, (T,), dev, "slots"),
        _dense(tree, torch.int64, (T,), dev, "tree"), S, T, heads, kv_heads, dim, window,
        dim ** -0.5 if scale is None else scale, _dense(o, dt, (T, heads, dim), dev, "out"),
        _dense(lse, torch.float32, (T, heads), dev, "lse"), ws.data_ptr(), ws.numel(),
        _stream(stream, dev)), "chunk_attention")
    return o if lse is None else (o, lse)


def _q4(name, codes, scales, h, ids, group, mins, out, stream):
    dev = _cuda(h, "h")
    dt = h.dtype
    if dt not in (torch.bfloat16, torch.float16):
        raise TypeError(f"h: expected bf16 or fp16, got {dt}")
    _need(h.dim() == 2, "h", "expected vectors x d")
    _need(codes.dim() == 2, "codes", "expected rows x d/2")
    _need(group in (32, 64, 128), "group", "must be 32, 64 or 128")
    M, d = h.shape
    n = codes.shape[0]
    _need(d % group == 0 and d >= group, "group", f"does not divide d = {d}")
    K = n
    if ids is not None:
        _need(ids.dim() == 2, "ids", "expected vectors x candidates")
        K = ids.shape[1]
    if out is None:
        out = _empty((M, K), torch.float32, dev, stream)
    args = [_DTYPES[dt], _dense(codes, torch.uint8, (n, d // 2), dev, "codes"),
            _dense(scales, dt, (n, d // group), dev, "scales"),
            _dense(mins, dt, (n, d // group), dev, "mins"), _dense(h, dt, (M, d), dev, "h")]
    o = _dense(out, torch.float32, (M, K), dev, "out")
    if ids is None:
        check(load().lmhead_q4_head(*args, n, d, group, M, o, _stream(stream, dev)), name)
    else:
        check(load().lmhead_q4_gather_logits(
            *args, _dense(ids, torch.int32, (M, K), dev, "ids"), n, d, group, M, K, o,
            _stream(stream, dev)), name)
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
    _need(logits.dim() == 2, "logits", "expected beams x entries")
    if logits.dtype not in _DTYPES:
        raise TypeError(f"logits: expected bf16, fp16 or fp32, got {logits.dtype}")
    rows, n = logits.shape
    _need(beams >= 1 and rows >= 1 and rows % beams == 0, "beams", f"does not divide {rows} rows")
    _need(n >= 1, "logits", "no entries")
    _need(1 <= k <= 32, "k", "must be 1 to 32")
    if logits.stride(1) != 1 and n > 1:
        raise TypeError("logits: expected contiguous rows")
    S = rows // beams
    stride = logits.stride(0) if rows > 1 else n
    _need(stride >= n, "logits", "rows overlap")
    if out is None:
        parent, token = _empty((2, S, k), torch.int32, dev, stream).unbind(0)
        score = _empty((S, k), torch.float32, dev, stream)
    else:
        parent, token, score = out
    nbytes = _beam_bytes(dev, S, beams, n, k)
    ws = _workspace(workspace, nbytes, dev, stream)
    if finished is not None and finished.dtype == torch.bool:
        finished = finished.view(torch.uint8)
    i32 = torch.int32
    check(load().lmhead_beam_select(
        _DTYPES[logits.dtype], logits.data_ptr(), stride,
        _dense(scores, torch.float32, (rows,), dev, "scores"),
        _dense(ids, i32, (rows, n), dev, "ids"),
        _dense(finished, torch.uint8, (rows,), dev, "finished"), S, beams, n, k, eos,
        _dense(parent, i32, (S, k), dev, "parent"), _dense(token, i32, (S, k), dev, "token"),
        _dense(score, torch.float32, (S, k), dev, "score"), ws.data_ptr(), ws.numel(),
        _stream(stream, dev)), "beam_select")
    return parent, token, score


def beam_reorder(parent: torch.Tensor, states: Sequence[torch.Tensor], beams: int, out=None,
                 stream=None):
    """Each state tensor (S*beams rows of any type, contiguous) by the parents
    chosen (S x k): a list of tensors of S*k rows, zeros where parent is -1."""
    dev = _cuda(parent, "parent")
    _need(parent.dim() == 2 and parent.numel() > 0, "parent", "expected sequences x k")
    S, k = parent.shape
    n = len(states)
    _need(1 <= n <= 8, "states", "1 to 8 tensors")
    _need(beams >= 1, "beams", "must be positive")
    if out is None:
        out = [_empty((S * k,) + tuple(t.shape[1:]), t.dtype, dev, stream) for t in states]
    _need(len(out) == n, "out", "one tensor per state")
    src, dst, size = (ctypes.c_void_p * n)(), (ctypes.c_void_p * n)(), (ctypes.c_int64 * n)()
    for i, (t, o) in enumerate(zip(states, out)):
        src[i] = _dense(t, t.dtype, (S * beams,) + tuple(t.shape[1:]), dev, f"states[{i}]")
        dst[i] = _dense(o, t.dtype, (S * k,) + tuple(t.shape[1:]), dev, f"out[{i}]")
        size[i] = t.numel() // (S * beams) * t.element_size()
    check(load().lmhead_beam_reorder(
        _dense(parent, torch.int32, (S, k), dev, "parent"), S, beams, k, n, src, dst, size,
        _stream(stream, dev)), "beam_reorder")
    return out
