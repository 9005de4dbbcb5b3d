"""Latent attention over a paged cache: buffers around moe_mla_append and moe_mla_decode.

``LatentAttention`` owns the workspace and the outputs of one shape; the cache,
the block table and the lengths belong to the caller (layers of a network share
a block table, each with a cache of its own).
"""
from __future__ import annotations

import torch

from . import (MOE_ERR_INVALID_ARG, MoeError, mla_config, moe_mla_append, moe_mla_decode, moe_mla_status,
               moe_mla_workspace_size)
from .norm import check_tensor


class LatentAttention:
    def __init__(self, batch, heads, latent=512, rope=64, page_size=64, num_pages=1, max_pages=1, scale=1.0,
                 device="cuda"):
        self.cfg = mla_config(batch, heads, latent, rope, page_size, num_pages, max_pages, scale)
        self.batch, self.heads, self.latent, self.rope = batch, heads, latent, rope
        self.page_size, self.num_pages, self.max_pages = page_size, num_pages, max_pages
        dev = torch.device(device)
        self.ws = torch.empty(moe_mla_workspace_size(self.cfg), dtype=torch.uint8, device=dev)
        self.ws[:16].zero_()                       # the status word
        self.out = torch.empty((batch, heads, latent), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((batch, heads), dtype=torch.float32, device=dev)

    def new_cache(self) -> torch.Tensor:
        return torch.zeros((self.num_pages, self.page_size, self.latent + self.rope), dtype=torch.bfloat16,
                           device=self.ws.device)

    def _check_cache(self, cache, block_table):
        check_tensor("cache", cache, torch.bfloat16, (self.num_pages, self.page_size, self.latent + self.rope))
        check_tensor("block_table", block_table, torch.int32, (self.batch, self.max_pages))

    def append(self, kv, cache, block_table, seq, pos, gamma=None, eps=1e-6, cos_sin=None, stream=0):
        """Write tokens kv [n][latent + rope] (rows may be pitched) at positions pos of sequences seq into the cache."""
        n, row = seq.numel(), self.latent + self.rope
        if not kv.is_cuda or kv.dtype is not torch.bfloat16 or kv.shape != (n, row) or (n and kv.stride(1) != 1):
            raise MoeError("kv: a CUDA bfloat16 tensor of shape (n, %d) with dense rows is wanted" % row,
                           MOE_ERR_INVALID_ARG)
        self._check_cache(cache, block_table)
        check_tensor("seq", seq, torch.int32, (n,))
        check_tensor("pos", pos, torch.int32, (n,))
        if gamma is not None:
            check_tensor("gamma", gamma, torch.bfloat16, (self.latent,))
        if cos_sin is not None:
            check_tensor("cos_sin", cos_sin, torch.float32, (cos_sin.shape[0], self.rope))
        moe_mla_append(self.cfg, n, kv.data_ptr(), kv.stride(0) if n > 1 else row,
                       gamma.data_ptr() if gamma is not None else 0, eps,
                       cos_sin.data_ptr() if cos_sin is not None else 0,
                       cos_sin.shape[0] if cos_sin is not None else 0, seq.data_ptr(), pos.data_ptr(),
                       block_table.data_ptr(), cache.data_ptr(), self.ws.data_ptr(), stream)

    def decode(self, q, cache, block_table, seq_lens, stream=0, out=None, lse=None):
        """Attention of q [batch][heads][latent + rope] (dense rows, any pitch) over the cached tokens; returns out."""
        out = self.out if out is None else out
        lse = self.lse if lse is None else lse
        row = self.latent + self.rope
        if not q.is_cuda or q.dtype is not torch.bfloat16 or q.shape != (self.batch, self.heads, row) or \
                (q.numel() and q.stride(2) != 1):
            raise MoeError("q: a CUDA bfloat16 tensor of shape %s with dense rows is wanted" %
                           ((self.batch, self.heads, row),), MOE_ERR_INVALID_ARG)
        self._check_cache(cache, block_table)
        check_tensor("seq_lens", seq_lens, torch.int32, (self.batch,))
        check_tensor("out", out, torch.bfloat16, (self.batch, self.heads, self.latent))
        check_tensor("lse", lse, torch.float32, (self.batch, self.heads))
        # the stride of a dimension of one is arbitrary
        sh = q.stride(1) if self.heads > 1 else row
        sb = q.stride(0) if self.batch > 1 else sh * self.heads
        moe_mla_decode(self.cfg, q.data_ptr(), sb, sh, cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
                       out.data_ptr(), lse.data_ptr(), self.ws.data_ptr(), stream)
        return out

    def status(self, clear=True, stream=0):
        return moe_mla_status(self.cfg, self.ws.data_ptr(), clear, stream)

    def check_status(self):
        code, site = self.status()
        if code:
            raise MoeError("device status (site %d)" % site, code)
