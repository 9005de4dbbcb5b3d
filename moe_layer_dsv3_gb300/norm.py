"""Residual add + RMSNorm with MX output, and its gradient: buffers around the C entry points.

``AddRMSNorm`` owns the outputs of one (T, d) shape. PyTorch is used only for
device memory; the work runs in moe_add_rmsnorm and moe_add_rmsnorm_backward.
"""
from __future__ import annotations

import torch

from . import (MOE_ERR_INVALID_ARG, MoeError, moe_add_rmsnorm, moe_add_rmsnorm_backward,
               moe_add_rmsnorm_backward_workspace)


def check_tensor(name, t, dtype, shape):
    """A dense CUDA tensor of this type and shape, or MOE_ERR_INVALID_ARG (the library sees only an address)."""
    if not t.is_cuda or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise MoeError("%s: a dense CUDA %s tensor of shape %s is wanted" % (name, dtype, tuple(shape)),
                       MOE_ERR_INVALID_ARG)


class AddRMSNorm:
    """h = x + residual, y = h rstd gamma; with mx=True also MX(y) as codes and row-major scales."""

    def __init__(self, T, d, eps=1e-6, mx=False, device="cuda"):
        self.T, self.d, self.eps, self.mx = T, d, eps, mx
        dev = torch.device(device)
        bf = dict(dtype=torch.bfloat16, device=dev)
        self.ws = torch.empty(moe_add_rmsnorm_backward_workspace(T, d), dtype=torch.uint8, device=dev)
        self.h = torch.empty((T, d), **bf)
        self.y = torch.empty((T, d), **bf)
        self.rstd = torch.empty(T, dtype=torch.float32, device=dev)
        self.dx = torch.empty((T, d), **bf)
        self.dgamma = torch.empty(d, dtype=torch.float32, device=dev)
        self.codes = torch.empty((T, d), dtype=torch.uint8, device=dev) if mx else None
        self.scales = torch.empty((T, d // 32), dtype=torch.uint8, device=dev) if mx else None
        self._saved = None

    def forward(self, x, gamma, residual=None, stream=0, layer=None):
        """Write h (with a residual; otherwise x stands for it), y and rstd, and return y.

        ``layer``: a MoELayer of the same T and d made with MOE_FLAG_X_QUANTIZED.
        MX(y) then goes straight into its workspace, and layer.forward(y, ...)
        reads it there instead of quantising y.
        """
        check_tensor("x", x, torch.bfloat16, (self.T, self.d))
        check_tensor("gamma", gamma, torch.bfloat16, (self.d,))
        if residual is not None:
            check_tensor("residual", residual, torch.bfloat16, (self.T, self.d))
        codes = scales = tiled = 0
        if layer is not None:
            if (layer.T, layer.d) != (self.T, self.d):
                raise MoeError("AddRMSNorm.forward: the layer has another shape", MOE_ERR_INVALID_ARG)
            codes, scales, tiled = (layer.ws_tensor(n).data_ptr() for n in ("XQ", "XQ_SFC", "XQ_SF"))
        elif self.mx:
            codes, scales = self.codes.data_ptr(), self.scales.data_ptr()
        moe_add_rmsnorm(self.T, self.d, x.data_ptr(), residual.data_ptr() if residual is not None else 0,
                        gamma.data_ptr(), self.eps, self.h.data_ptr() if residual is not None else 0,
                        self.y.data_ptr(), self.rstd.data_ptr(), codes, scales, tiled, stream)
        self._saved = self.h if residual is not None else x
        return self.y

    def backward(self, dy, gamma, dres=None, stream=0, h=None, rstd=None):
        """Write dx (the gradient of x and residual) and dgamma, and return dx.

        h and rstd default to those of the last forward call. Without a residual that call keeps x itself as h, so x
        has to hold the same values until here; the norm's own h, y, rstd, dx and dgamma last until its next call.
        """
        h = self._saved if h is None else h
        rstd = self.rstd if rstd is None else rstd
        if h is None:
            raise MoeError("AddRMSNorm.backward: no forward call and no h", MOE_ERR_INVALID_ARG)
        for name, t in (("dy", dy), ("h", h), ("dres", dres)):
            if t is not None:
                check_tensor(name, t, torch.bfloat16, (self.T, self.d))
        check_tensor("gamma", gamma, torch.bfloat16, (self.d,))
        check_tensor("rstd", rstd, torch.float32, (self.T,))
        moe_add_rmsnorm_backward(self.T, self.d, dy.data_ptr(), dres.data_ptr() if dres is not None else 0,
                                 h.data_ptr(), gamma.data_ptr(), rstd.data_ptr(), self.dx.data_ptr(),
                                 self.dgamma.data_ptr(), self.ws.data_ptr(), stream)
        return self.dx
