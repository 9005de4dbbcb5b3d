"""Latent attention over a paged cache: buffers around moe_mla_append, moe_mla_decode and moe_mla_decode_tree.

``LatentAttention`` owns the workspace and the outputs of one shape; the cache,
the block table and the lengths belong to the caller (layers of a network share
a block table, each with a cache of its own).
"""
from __future__ import annotations

import math

import torch

from . import (MOE_ERR_INVALID_ARG, MoeError, mla_config, moe_mla_append, moe_mla_decode, moe_mla_decode_tree,
               moe_mla_status, moe_mla_workspace_size)
from .norm import check_device, check_tensor


class LatentAttention:
    def __init__(self, batch, heads, latent=512, rope=64, page_size=64, num_pages=1, max_pages=1, scale=1.0,
                 device="cuda", drafts=0):
        """drafts: most drafted tokens of a sequence, if decode_tree is to have outputs of its own."""
        self.cfg = mla_config(batch, heads, latent, rope, page_size, num_pages, max_pages, scale)
        self.batch, self.heads, self.latent, self.rope = batch, heads, latent, rope
        self.page_size, self.num_pages, self.max_pages = page_size, num_pages, max_pages
        dev = torch.device(device)
        self.ws = torch.empty(moe_mla_workspace_size(self.cfg), dtype=torch.uint8, device=dev)
        self.ws[:16].zero_()                       # the status word
        self.out = torch.empty((batch, heads, latent), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((batch, heads), dtype=torch.float32, device=dev)
        self.tree_out = torch.empty((batch, drafts, heads, latent), dtype=torch.bfloat16, device=dev)
        self.tree_lse = torch.empty((batch, drafts, heads), dtype=torch.float32, device=dev)

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

    def decode_tree(self, q, cache, block_table, seq_lens, tree=None, drafts=None, stream=0, out=None, lse=None):
        """Attention of drafted tokens, the last ones of each sequence; returns out [batch][n][heads][latent].

        q [batch][n][heads][latent + rope]: dense rows, any pitch, a token's heads as far apart as its neighbours' (q of
        shape [batch][n * heads][..], viewed). tree int64 [batch][n]: bit j of word i: token i sees drafted token j (None: a
        chain). drafts int32 [batch]: drafted tokens of each sequence (None: n each). out and lse default to tree_out and
        tree_lse: with fewer tokens than those hold, to [batch][n].. lying dense at their front."""
        row = self.latent + self.rope
        n = q.shape[1] if q.dim() == 4 else 0
        if not q.is_cuda or q.dtype is not torch.bfloat16 or n < 1 or q.shape != (self.batch, n, self.heads, row) or \
                (q.numel() and q.stride(3) != 1):
            raise MoeError("q: a CUDA bfloat16 tensor of shape %s with dense rows is wanted" %
                           ((self.batch, "n", self.heads, row),), MOE_ERR_INVALID_ARG)
        out = self._front(self.tree_out, n) if out is None else out
        lse = self._front(self.tree_lse, n) if lse is None else lse
        # the stride of a dimension of one is arbitrary
        sh = q.stride(2) if self.heads > 1 else (q.stride(1) if n > 1 else row)
        if self.heads > 1 and n > 1 and q.stride(1) != self.heads * sh:
            raise MoeError("q: a token's heads follow the token's before it at the same pitch", MOE_ERR_INVALID_ARG)
        sb = q.stride(0) if self.batch > 1 else sh * self.heads * n
        self._check_cache(cache, block_table)
        check_tensor("seq_lens", seq_lens, torch.int32, (self.batch,))
        if tree is not None:
            check_tensor("tree", tree, torch.int64, (self.batch, n))
        if drafts is not None:
            check_tensor("drafts", drafts, torch.int32, (self.batch,))
        check_tensor("out", out, torch.bfloat16, (self.batch, n, self.heads, self.latent))
        check_tensor("lse", lse, torch.float32, (self.batch, n, self.heads))
        check_device(q, cache, block_table, seq_lens, tree, drafts, out, lse, self.ws)
        moe_mla_decode_tree(self.cfg, n, q.data_ptr(), sb, sh, cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
                            drafts.data_ptr() if drafts is not None else 0, tree.data_ptr() if tree is not None else 0,
                            out.data_ptr(), lse.data_ptr(), self.ws.data_ptr(), stream)
        return out

    @staticmethod
    def _front(t, n):
        """The front of the buffer t [batch][drafts].. as [batch][n].. (t itself where it does not hold as much)."""
        if n >= t.shape[1]:
            return t
        shape = (t.shape[0], n, *t.shape[2:])
        return t.view(-1)[:math.prod(shape)].view(shape)

    def status(self, clear=True, stream=0):
        return moe_mla_status(self.cfg, self.ws.data_ptr(), clear, stream)

    def check_status(self):
        code, site = self.status()
        if code:
            raise MoeError("device status (site %d)" % site, code)
