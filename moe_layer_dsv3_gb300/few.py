"""The MoE layer for a few tokens: buffers around moe_few_forward.

``FewTokenMoE`` owns the workspace and the outputs for up to T tokens of one layer
shape, and its quantised weights, unless it is given those of a ``MoELayer``.
"""
from __future__ import annotations

import torch

from . import (MOE_ERR_INVALID_ARG, MoeError, config, moe_few_forward, moe_few_status, moe_few_workspace_size,
               moe_quantize_weights, moe_weights_size)
from .norm import check_device, check_tensor


class FewTokenMoE:
    def __init__(self, T, d, E, k, n_groups=1, topk_groups=1, I=128, n_shared=0, wq=None, device="cuda"):
        """Up to T <= 64 tokens a call. wq: the weights of a ``MoELayer`` of this shape (its ``wq``), to be shared with it."""
        self.T, self.d, self.E, self.k, self.I, self.S = T, d, E, k, I, n_shared
        self._shape = (d, E, k, n_groups, topk_groups, I, n_shared)
        self.cfg = config(T, *self._shape)
        self._cfgs = {T: self.cfg}
        dev = torch.device(device)
        self.ws = torch.zeros(moe_few_workspace_size(self.cfg), dtype=torch.uint8, device=dev)
        n = moe_weights_size(self.cfg)
        if wq is None:
            wq = torch.zeros(n, dtype=torch.uint8, device=dev)
        else:
            check_tensor("wq", wq, torch.uint8, (n,))
            if wq.device != self.ws.device:
                raise MoeError("wq: weights of %s for a layer on %s" % (wq.device, self.ws.device), MOE_ERR_INVALID_ARG)
        self.wq = wq
        self.topk_idx = torch.empty((T, k), dtype=torch.int32, device=dev)
        self.topk_w = torch.empty((T, k), dtype=torch.float32, device=dev)
        self.y = torch.empty((T, d), dtype=torch.bfloat16, device=dev)

    def quantize_weights(self, w_gu, w_d, ws_gu=None, ws_d=None, stream=0):
        """bf16 masters w_gu [E][2I][d], w_d [E][d][I] (and the shared expert's [1][..][..]) into the MXFP8 weights."""
        check_tensor("w_gu", w_gu, torch.bfloat16, (self.E, 2 * self.I, self.d))
        check_tensor("w_d", w_d, torch.bfloat16, (self.E, self.d, self.I))
        if self.S:
            if ws_gu is None or ws_d is None:
                raise MoeError("ws_gu, ws_d: the shared expert's weights are wanted", MOE_ERR_INVALID_ARG)
            check_tensor("ws_gu", ws_gu, torch.bfloat16, (self.S, 2 * self.I, self.d))
            check_tensor("ws_d", ws_d, torch.bfloat16, (self.S, self.d, self.I))
        check_device(w_gu, w_d, *((ws_gu, ws_d) if self.S else ()), self.wq)
        moe_quantize_weights(self.cfg, w_gu.data_ptr(), w_d.data_ptr(), ws_gu.data_ptr() if self.S else 0,
                             ws_d.data_ptr() if self.S else 0, self.wq.data_ptr(), stream)

    def forward(self, x, w_router, bias, stream=0, y=None):
        """Route x [t][d] (t <= T), run the experts and write y (default: the first t rows of self.y), which is returned.

        The choice and the gates are in the first t rows of ``topk_idx`` and ``topk_w``."""
        t = x.shape[0]
        if t > self.T:
            raise MoeError("x: %d tokens where %d are the most" % (t, self.T), MOE_ERR_INVALID_ARG)
        check_tensor("x", x, torch.bfloat16, (t, self.d))
        check_tensor("w_router", w_router, torch.bfloat16, (self.E, self.d))
        check_tensor("bias", bias, torch.float32, (self.E,))
        if y is None:
            y = self.y[:t]
        check_tensor("y", y, torch.bfloat16, (t, self.d))
        check_device(x, w_router, bias, y, self.wq, self.ws)
        cfg = self._cfgs.get(t)
        if cfg is None:
            cfg = self._cfgs[t] = config(t, *self._shape)
        moe_few_forward(cfg, x.data_ptr(), w_router.data_ptr(), bias.data_ptr(), self.wq.data_ptr(), self.topk_idx.data_ptr(),
                        self.topk_w.data_ptr(), y.data_ptr(), self.ws.data_ptr(), stream)
        return y

    def status(self, clear=True, stream=0):
        return moe_few_status(self.cfg, self.ws.data_ptr(), clear, stream)

    def check_status(self):
        code, site = self.status()
        if code:
            raise MoeError("device status (site %d)" % site, code)
