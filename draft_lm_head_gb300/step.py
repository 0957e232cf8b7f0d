"""The operators of a step over the paged cache (include/lmhead.h, "Operators of
a step over the paged cache").

    rotary(q, k, positions, turns)                       # in place
    o, lse = chunk_attention(q, kc, vc, table, lens, plan.cu, k=k, v=v, slots=plan.slots,
                             tree=bits, with_lse=True, granted=plan.granted)
    ...                                                  # the target's p behind each node
    tokens, path, accepted = verify_tree(p, drafts, parent, plan.cu, r, u, depth,
                                         granted=plan.granted)
    new = cache_keep([kc, vc], table, path, first=lens)  # the accepted rows
    left = page_release(lens, new, table, free_pages, plan.free_left, P, cu=plan.cu,
                        granted=plan.granted)

where a node's position is the root's and its depth on top: `read` + depth, with the tokens
read so far (plan.positions are places in the cache, lens + i: right for chains, and as
long as nothing was evicted). And, for a cache that outgrows its room,

    cache_weights(q, kc, table, lens, plan.cu, lse, weights, granted=plan.granted)
    kept = cache_select(weights, table, lens, budget, sinks=4, recent=256)
    new = cache_keep([kc, vc, weights], table, kept)
    left = page_release(lens, new, table, free_pages, free_count, P)

(the weights of a tree's step go between verify_tree and cache_keep, with -inf in the lse
of nodes that are not on `path`, where rejected drafts are not to count, and `weights` among
the caches that cache_keep moves). The frequencies of rotary come from prep.rotary_turns.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Sequence

import torch

from ._lib import check, load
from ._memory import result, scratch, stream_handle
from .serving import _DTYPES, _cuda, _dense, _heads_tensor


def _strides(t: torch.Tensor):
    """Strides, with those of dimensions of one (which mean nothing) as in a
    contiguous tensor."""
    st, shape = t.stride(), t.shape
    if 1 not in shape:
        return st
    st, at = list(st), 1
    for i in range(len(shape) - 1, -1, -1):
        if shape[i] == 1:
            st[i] = at
        at = max(at, st[i] * shape[i])
    return st


def _prefix(t: torch.Tensor, T: int, name: str) -> torch.Tensor:
    """The first T of a plan's buffer, which may be longer than the step's tokens."""
    if t.shape[0] == T:
        return t
    if t.dim() != 1 or t.shape[0] < T:
        raise ValueError(f"{name}: expected one per token")
    return t[:T]


def _rows(t: torch.Tensor, dtype, shape, dev, name: str):
    _heads_tensor(t, dtype, shape, dev, name)
    st = _strides(t)
    return t.data_ptr(), st[0], st[1]


def rotary(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor,
           turns: torch.Tensor, interleaved: bool = False, backward: bool = False,
           magnitude: float = 1.0, out=None, stream=None):
    """Rotary positions of q (T x heads x dim) and k (T x kv_heads x dim, or None)
    of bf16, fp16 or fp32, any strides with dim contiguous: in place, or into the
    pair `out`, which is returned. positions: T int32 (a plan's for a chain of tokens, a
    tree's by depth), negative ones leave their rows unwritten. turns: int64 from prep.rotary_turns, for the first
    2 * len(turns) elements of a head. backward: the rotation's transpose, the
    gradient's way back (see lmhead_rotary)."""
    dev = _cuda(q, "q")
    if q.dim() != 3 or (k is not None and k.dim() != 3) or turns.dim() != 1:
        raise ValueError("q, k, turns: expected tokens x heads x dim and one frequency a pair")
    T, heads, dim = q.shape
    dt = q.dtype
    if dt not in _DTYPES:
        raise TypeError(f"q: expected bf16, fp16 or fp32, got {dt}")
    oq, ok = (q, k) if out is None else out
    if (ok is None) != (k is None):
        raise ValueError("out: expected a pair like q and k")
    rot = 2 * turns.shape[0]
    qa = _rows(q, dt, (T, heads, dim), dev, "q")
    oqa = qa if oq is q else _rows(oq, dt, (T, heads, dim), dev, "out")
    ka = oka = (0, 0, 0)
    kv_heads = 0
    if k is not None:
        kv_heads = k.shape[1]
        ka = _rows(k, dt, (T, kv_heads, dim), dev, "k")
        oka = ka if ok is k else _rows(ok, dt, (T, kv_heads, dim), dev, "out")
    positions = _prefix(positions, T, "positions")
    check(load().lmhead_rotary(
        _DTYPES[dt], *qa, *ka, _dense(positions, torch.int32, (T,), dev, "positions"),
        _dense(turns, torch.int64, (rot // 2,), dev, "turns"), T, heads, kv_heads, dim, rot,
        interleaved, backward, magnitude, *oqa, *oka, stream_handle(stream, dev)), "rotary")
    return oq, ok


def verify_tree(p: torch.Tensor, tokens: torch.Tensor, parent: torch.Tensor, cu: torch.Tensor,
                r: torch.Tensor, u: torch.Tensor, depth: int,
                cand_ids: Optional[torch.Tensor] = None, cand_q: Optional[torch.Tensor] = None,
                granted: Optional[torch.Tensor] = None, out=None, stream=None):
    """Which path of each request's draft tree the target accepts, and the token
    behind it: (tokens, path, accepted), S x (depth + 1) twice and S, int32. p: T x n
    fp32, the target's distribution behind each node; tokens, parent: T int32; cu:
    starts of the requests' nodes; r, u: T and S uniforms; cand_ids, cand_q: T x K,
    what each node's children were drawn from without replacement, or None where they
    are given (see lmhead_verify_tree)."""
    dev = _cuda(p, "p")
    i32, f32 = torch.int32, torch.float32
    if p.dim() != 2 or cu.dim() != 1 or not 0 <= depth < 64:
        raise ValueError("p, cu, depth: expected nodes x entries, starts and 0 to 63 drafts")
    T, n = p.shape
    S = cu.shape[0] - 1
    K = 0
    if cand_ids is not None or cand_q is not None:
        if cand_ids is None or cand_q is None or cand_ids.dim() != 2:
            raise ValueError("cand_ids, cand_q: are given together, nodes x candidates")
        K = cand_ids.shape[1]
        if K < 1:  # (no address would tell them from none given)
            raise ValueError("cand_ids, cand_q: expected one candidate or more")
    W = depth + 1
    if out is None:
        out = (result((S, W), i32, dev, stream), result((S, W), i32, dev, stream), result((S,), i32, dev, stream))
    said, path, accepted = out
    check(load().lmhead_verify_tree(
        _dense(p, f32, (T, n), dev, "p"), n, _dense(tokens, i32, (T,), dev, "tokens"),
        _dense(parent, i32, (T,), dev, "parent"), _dense(cu, i32, (S + 1,), dev, "cu"),
        _dense(granted, i32, (S,), dev, "granted"), _dense(r, f32, (T,), dev, "r"),
        _dense(u, f32, (S,), dev, "u"), _dense(cand_ids, i32, (T, K), dev, "cand_ids"),
        _dense(cand_q, f32, (T, K), dev, "cand_q"), K, S, T, depth, _dense(said, i32, (S, W), dev, "tokens"),
        _dense(path, i32, (S, W), dev, "path"), _dense(accepted, i32, (S,), dev, "accepted"),
        stream_handle(stream, dev)), "verify_tree")
    return said, path, accepted


_Caches = ctypes.c_int64 * 40  # up to 8 addresses, strides of pages, tokens and heads, and row sizes


def cache_keep(caches: Sequence[torch.Tensor], table: torch.Tensor, kept: torch.Tensor,
               first: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """Moves rows of paged caches together, in place: row first + i of a request
    becomes what its row first + kept[i] was. caches: 1 to 8 tensors pages x page_size
    x kv_heads (x dim, contiguous), any types and strides; kept: S x n for all heads
    or S x kv_heads x n, negative entries leave their rows alone; first: S, or None
    for 0. Returns the new lengths, S int32 (see lmhead_cache_keep)."""
    count = len(caches)
    if not 1 <= count <= 8:
        raise ValueError("caches: expected 1 to 8 tensors")
    dev = _cuda(caches[0], "caches")
    if kept.dim() not in (2, 3) or table.dim() != 2:
        raise ValueError("kept, table: expected requests (x heads) x rows and requests x pages")
    S, n = kept.shape[0], kept.shape[-1]
    lead = caches[0].shape[:3]
    if len(lead) != 3:
        raise ValueError("caches: expected pages x page_size x kv_heads (x dim)")
    pages, P, kv_heads = lead
    arr = _Caches()
    for i, t in enumerate(caches):
        shape = t.shape
        if len(shape) not in (3, 4) or shape[:3] != lead or t.device != dev:
            raise ValueError(f"caches[{i}]: expected {tuple(lead)} (x dim) on {dev}")
        size, st = t.element_size(), _strides(t)
        if len(shape) == 4:
            if st[3] != 1:
                raise TypeError(f"caches[{i}]: expected a contiguous last dimension")
            arr[32 + i] = size * shape[3]
        else:
            arr[32 + i] = size
        arr[i] = t.data_ptr()
        arr[8 + i], arr[16 + i], arr[24 + i] = st[0] * size, st[1] * size, st[2] * size
    i32 = torch.int32
    want = (S, n) if kept.dim() == 2 else (S, kv_heads, n)
    if out is None:
        out = result((S,), i32, dev, stream)
    at = ctypes.addressof(arr)
    check(load().lmhead_cache_keep(
        count, at, at + 64, at + 128, at + 192, at + 256, pages, P, kv_heads,
        _dense(table, i32, (S, table.shape[1]), dev, "table"), table.shape[1],
        _dense(kept, i32, want, dev, "kept"), n, kept.dim() == 3,
        _dense(first, i32, (S,), dev, "first"), S, _dense(out, i32, (S,), dev, "out"),
        stream_handle(stream, dev)), "cache_keep")
    return out


def page_release(lens: torch.Tensor, new_lens: torch.Tensor, table: torch.Tensor,
                 free_pages: torch.Tensor, free_count: torch.Tensor, page_size: int,
                 cu: Optional[torch.Tensor] = None, granted: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gives the pages of requests that have become shorter back: free_pages (a
    page plan's, with room for them) is extended in place behind its first
    free_count entries, the new count (1 int32) is returned. No other request may hold
    the pages that go. A request held lens
    tokens, and its cu[s+1] - cu[s] new ones if cu is given and granted is not 0; it
    holds new_lens from now on (see lmhead_page_release)."""
    dev = _cuda(lens, "lens")
    i32 = torch.int32
    if lens.dim() != 1 or table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("lens, table, free_pages: expected requests, requests x pages and pages")
    S, width, cap = lens.shape[0], table.shape[1], free_pages.shape[0]
    if out is None:
        out = result((1,), i32, dev, stream)
    check(load().lmhead_page_release(
        _dense(lens, i32, (S,), dev, "lens"), _dense(new_lens, i32, (S,), dev, "new_lens"),
        _dense(cu, i32, (S + 1,), dev, "cu"), _dense(granted, i32, (S,), dev, "granted"), S,
        _dense(table, i32, (S, width), dev, "table"), width,
        _dense(free_pages, i32, (cap,), dev, "free_pages"), cap,
        _dense(free_count, i32, (1,), dev, "free_count"), page_size,
        _dense(out, i32, (1,), dev, "out"), stream_handle(stream, dev)), "page_release")
    return out


@functools.lru_cache(maxsize=4096)
def _weights_bytes(device, S: int) -> int:
    with torch.cuda.device(device):
        return int(load().lmhead_cache_weights_workspace_size(S))


def _weights_tensor(t: torch.Tensor, dev):
    """Address and strides of pages x page_size x kv_heads fp32."""
    if t.dim() != 3 or t.dtype is not torch.float32 or t.device != dev:
        raise ValueError(f"weights: expected fp32 pages x page_size x kv_heads on {dev}")
    return (t.data_ptr(), *_strides(t))


def cache_weights(q: torch.Tensor, k_cache: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
                  cu: torch.Tensor, lse: torch.Tensor, weights: torch.Tensor,
                  tree: Optional[torch.Tensor] = None, window: int = 0,
                  scale: Optional[float] = None, decay: float = 1.0,
                  granted: Optional[torch.Tensor] = None, workspace=None, stream=None) -> torch.Tensor:
    """Adds up, in place, how much attention each cached token has drawn: weights
    (pages x page_size x kv_heads fp32, any strides) times decay, plus the softmax
    weights that the chunk's tokens give it; new tokens' entries start from nothing.
    q, k_cache (the chunk's K in it), table, lens, cu, tree, window, scale, granted as
    of chunk_attention, lse what it returned, -inf for rows that are not to count, as
    those of rejected drafts (see lmhead_cache_weights)."""
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
    qa = _rows(q, dt, (T, heads, dim), dev, "q")
    _heads_tensor(k_cache, dt, (pages, P, kv_heads, dim), dev, "k_cache")
    kc = _strides(k_cache)
    w = _weights_tensor(weights, dev)
    if weights.shape != (pages, P, kv_heads):
        raise ValueError(f"weights: expected shape {(pages, P, kv_heads)}, got {tuple(weights.shape)}")
    i32, f32 = torch.int32, torch.float32
    ws = scratch(workspace, _weights_bytes(dev, S), dev, stream)
    check(load().lmhead_cache_weights(
        _DTYPES[dt], *qa, k_cache.data_ptr(), *kc[:3], pages, P,
        _dense(table, i32, (S, width), dev, "table"), width, _dense(lens, i32, (S,), dev, "lens"),
        _dense(cu, i32, (S + 1,), dev, "cu"), _dense(granted, i32, (S,), dev, "granted"),
        _dense(tree, torch.int64, (T,), dev, "tree"), _dense(lse, f32, (T, heads), dev, "lse"), S, T,
        heads, kv_heads, dim, window, dim ** -0.5 if scale is None else scale, decay, *w,
        ws.data_ptr(), ws.numel(), stream_handle(stream, dev)), "cache_weights")
    return weights


def cache_select(weights: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, budget: int,
                 sinks: int = 0, recent: int = 0, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """The tokens of each request and K/V head that stay in a cache cut down to
    `budget`: the first `sinks`, the last `recent` and those with the largest weights
    between, S x kv_heads x budget places (int32, ascending, then -1), which
    cache_keep takes. Rotary positions of later tokens go on as if nothing had gone, a
    plan's do not (see lmhead_cache_select)."""
    dev = _cuda(weights, "weights")
    w = _weights_tensor(weights, dev)
    if table.dim() != 2 or budget < 1:
        raise ValueError("table, budget: expected requests x pages and a positive number")
    pages, P, kv_heads = weights.shape
    S, width = table.shape
    i32 = torch.int32
    if out is None:
        out = result((S, kv_heads, budget), i32, dev, stream)
    check(load().lmhead_cache_select(
        *w, pages, P, kv_heads, _dense(table, i32, (S, width), dev, "table"), width,
        _dense(lens, i32, (S,), dev, "lens"), S, budget, sinks, recent,
        _dense(out, i32, (S, kv_heads, budget), dev, "out"), stream_handle(stream, dev)),
        "cache_select")
    return out
