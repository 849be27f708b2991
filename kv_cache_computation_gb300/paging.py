"""Page bookkeeping of a serving step on the GPU (mac_page_step of include/mac.h)."""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _native as N
from .attention import _check, _dev, _on, _stream_ptr, _table

# bits of PageStep.status
OUT_OF_PAGES, ROW_FULL, OUT_OF_RANGE, TOO_MANY_TOKENS, RING_FULL = 1, 2, 4, 8, 16


class _PageStep(NamedTuple):
    lengths: torch.Tensor      # [batch] tokens each request holds after the step
    free_state: torch.Tensor   # [2] head and count of the free ring after the step
    starts: torch.Tensor       # [batch + 1] request b's new tokens are the packed tokens starts[b]:starts[b+1]
    positions: torch.Tensor    # [max_tokens] 0-based position of each packed token (0 past the last)
    slots: torch.Tensor        # [max_tokens] page * 16 + offset, or -1: not stored
    status: torch.Tensor       # [1] 0, or the bits above


class PageStep(_PageStep):
    """What page_step returns: six int32 tensors on the GPU (lengths, free_state, starts, positions, slots, status), and
    `unreleased`: of a step in place, [batch] the tokens of each finished request whose pages could not be freed
    (status RING_FULL, or OUT_OF_RANGE: one is not of the pool), 0 for all others; else None, since the lengths passed
    still say it."""
    unreleased = None


def new_page_pool(num_pages, device=None):
    """(free_pages, free_state) of a pool whose pages are all free."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return (torch.arange(num_pages, dtype=torch.int32, device=device),
            torch.tensor([0, num_pages], dtype=torch.int32, device=device))


def page_step(lengths, new_tokens, page_table, free_pages, free_state, max_tokens, in_place=False,
              stream=None, rejected=None) -> PageStep:
    """Pages, positions and slots for one step's new tokens, from the lengths on the GPU.

    lengths, new_tokens int32 [batch]: tokens each request holds and its new
    ones (negative: the request is finished, its pages are freed).  page_table
    int32 [batch, columns] and free_pages int32 [num_pages] are updated in
    place; lengths and free_state come back as new tensors, or, with in_place,
    in the tensors passed (for a captured step that runs on).  Where a finished
    request's pages cannot be freed (status RING_FULL, or OUT_OF_RANGE: one is
    not of the pool) they stay those of its table row: unreleased keeps its
    length, which becomes 0.

    rejected int32 [batch]: tokens taken back from the end of each request
    before its new ones (drafts that were not accepted); the pages it then
    does not need are freed.  Lengths must not be set back in any other way:
    the pages past them would be lost.
    """
    device = lengths.device
    B = lengths.shape[0]
    li, ni = _dev(lengths, "lengths", torch.int32, (B,)), _dev(new_tokens, "new_tokens", torch.int32, (B,), device)
    table, row, cols = _table(page_table, B, device)
    n = free_pages.numel()
    ring = _dev(free_pages, "free_pages", torch.int32, (n,), device)
    state = _dev(free_state, "free_state", torch.int32, (2,), device)
    back = None if rejected is None else _dev(rejected, "rejected", torch.int32, (B,), device)
    with _on(device, stream):
        new = lengths.new_empty
        out = (lengths if in_place else new(B), free_state if in_place else new(2), new(B + 1), new(max_tokens),
               new(max_tokens), new(1))
        unreleased = new(B) if in_place else None
        lo, so, starts, pos, slot, status = [t.data_ptr() for t in out]
        st = N.lib().mac_page_step_ex(B, max_tokens, n, li, ni, lo, table, row, cols, ring, state, so, starts, pos, slot,
                                      status, back, unreleased.data_ptr() if in_place else None,
                                      _stream_ptr(stream, device))
    if st:
        _check("mac_page_step_ex", st)
    step = PageStep(*out)
    if in_place:
        step.unreleased = unreleased
    return step
