"""The serving operators around the draft head (include/lmhead.h, "Serving
operators around the head").

    plan = page_plan(lens, new_lens, table, free_pages, free_count, P, max_tokens)
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from ._lib import check, load


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
