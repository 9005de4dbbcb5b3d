"""Block tables and slot maps from request lengths: buffers around moe_pages_update.

``PagePlan`` owns the maps of a step's new tokens; the block table, the pool of
free pages and the lengths belong to the caller, as for ``LatentAttention``.
"""
from __future__ import annotations

import torch

from . import MoeError, moe_pages_status, moe_pages_update
from .norm import check_device, check_tensor


class PagePlan:
    def __init__(self, batch, page_size, num_pages, max_pages, max_new, device="cuda"):
        """For steps of up to max_new new tokens over ``batch`` sequences of up to max_pages pages."""
        self.batch, self.page_size, self.num_pages = batch, page_size, num_pages
        self.max_pages, self.max_new = max_pages, max_new
        dev = torch.device(device)
        self.ws = torch.zeros(16, dtype=torch.uint8, device=dev)
        i32 = dict(dtype=torch.int32, device=dev)
        self.seq = torch.empty(max_new, **i32)
        self.pos = torch.empty(max_new, **i32)
        self.slot = torch.empty(max_new, **i32)
        self.starts = torch.empty(batch + 1, **i32)
        self._shapes = (torch.Size((batch,)), torch.Size((batch, max_pages)), torch.Size((num_pages,)), torch.Size((1,)))

    def new_pool(self):
        """An empty block table, all pages free, their count, and lengths of zero."""
        i32 = dict(dtype=torch.int32, device=self.ws.device)
        return (torch.full((self.batch, self.max_pages), -1, **i32), torch.arange(self.num_pages - 1, -1, -1, **i32),
                torch.full((1,), self.num_pages, **i32), torch.zeros(self.batch, **i32))

    def update(self, seq_lens, target, block_table, free_pages, free_count, lens_out=None, count_out=None, stream=0):
        """Bring the sequences from seq_lens to target tokens; lengths and count are updated in place unless given a place.

        Returns (seq, pos, slot) of the new tokens, padded to max_new; ``starts`` has their ranges."""
        lens_out = seq_lens if lens_out is None else lens_out
        count_out = free_count if count_out is None else count_out
        b, t, n, one = self._shapes
        # (a step takes a few microseconds on the GPU: one plain loop costs half of what seven calls of check_tensor do)
        dev = self.ws.get_device()
        if dev != torch.cuda.current_device():
            check_device(self.ws)
        for x, shape in ((seq_lens, b), (target, b), (block_table, t), (free_pages, n), (free_count, one), (lens_out, b),
                         (count_out, one)):
            if x.dtype is not torch.int32 or x.shape != shape or x.get_device() != dev or not x.is_contiguous():
                check_tensor("one of the arrays", x, torch.int32, shape)
                check_device(x)
        moe_pages_update(self.batch, self.page_size, self.num_pages, self.max_pages, self.max_new, seq_lens.data_ptr(),
                         target.data_ptr(), block_table.data_ptr(), free_pages.data_ptr(), free_count.data_ptr(),
                         lens_out.data_ptr(), count_out.data_ptr(), self.seq.data_ptr(), self.pos.data_ptr(),
                         self.slot.data_ptr(), self.starts.data_ptr(), self.ws.data_ptr(), stream)
        return self.seq, self.pos, self.slot

    def status(self, clear=True, stream=0):
        return moe_pages_status(self.ws.data_ptr(), clear, stream)

    def check_status(self):
        code, site = self.status()
        if code:
            raise MoeError("device status (site %d)" % site, code)
