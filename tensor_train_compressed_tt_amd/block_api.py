"""Torch-tensor front end of include/ttc_block.h: what stands between the
TT-linear layers of a transformer block.  Checks shapes, allocates the
caller-owned buffers with torch and passes device addresses and the current
HIP stream to the C entry points.  No arithmetic happens here."""

from __future__ import annotations

import torch

from . import (
    make_norm_desc,
    ttc_norm_bwd,
    ttc_norm_fwd,
    ttc_norm_workspace,
)
from .torch_api import _ACT, _nbytes, _need, _need_buf, _stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _bytes(n: int, device) -> torch.Tensor:
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


class LayerNorm:
    """Layer norm of rows of ``dim`` elements with the residual sum before it.

    ``x_dtype`` (float32 or bfloat16) is the residual stream's type, ``y_dtype``
    (float32, bfloat16 or float8_e4m3fn; the same if None) that of what the next
    layer reads.  gamma, beta and their gradients are fp32.
    """

    def __init__(self, dim, x_dtype=torch.float32, y_dtype=None, eps=1e-5):
        self.dim = int(dim)
        self.x_dtype = x_dtype
        self.y_dtype = x_dtype if y_dtype is None else y_dtype
        if self.x_dtype not in (torch.float32, torch.bfloat16) or self.y_dtype not in _ACT:
            raise ValueError(f"no layer norm from {self.x_dtype} to {self.y_dtype}")
        self.desc = make_norm_desc(self.dim, _ACT[self.x_dtype], _ACT[self.y_dtype], eps)

    def workspace(self, T: int):
        return ttc_norm_workspace(self.desc, T)

    def forward(self, x, gamma, beta, res=None, h=None, out=None, saved=None):
        """(y, h, saved): h = x + res, or x itself without res."""
        T, dim = int(x.shape[0]), self.dim
        _need(x, "x", self.x_dtype, (T, dim))
        _need(gamma, "gamma", torch.float32, (dim,))
        _need(beta, "beta", torch.float32, (dim,))
        if res is not None:
            _need(res, "res", self.x_dtype, (T, dim))
            if h is None:
                h = torch.empty_like(x)
            _need(h, "h", self.x_dtype, (T, dim))
        elif h is not None:
            raise ValueError("h is written only where res is given")
        if out is None:
            out = torch.empty((T, dim), dtype=self.y_dtype, device=x.device)
        _need(out, "out", self.y_dtype, (T, dim))
        if saved is None:
            saved = _bytes(self.workspace(T)[0], x.device)
        _need_buf(saved, "saved")
        ttc_norm_fwd(self.desc, T, x.data_ptr(), _ptr(res), gamma.data_ptr(), beta.data_ptr(), _ptr(h), out.data_ptr(),
                     saved.data_ptr(), _nbytes(saved), _stream())
        return out, (x if res is None else h), saved

    def backward(self, dy, h, gamma, saved, dh=None, dx=None, dgamma=None, dbeta=None, scratch=None):
        """(dx, dgamma, dbeta); dx is the gradient of x and of res alike, with
        ``dh``, the gradient that reaches h from elsewhere, added."""
        T, dim = int(h.shape[0]), self.dim
        _need(dy, "dy", self.y_dtype, (T, dim))
        _need(h, "h", self.x_dtype, (T, dim))
        _need(gamma, "gamma", torch.float32, (dim,))
        _need_buf(saved, "saved")
        if dh is not None:
            _need(dh, "dh", self.x_dtype, (T, dim))
        if dx is None:
            dx = torch.empty_like(h)
        _need(dx, "dx", self.x_dtype, (T, dim))
        if dgamma is None:
            dgamma = torch.empty_like(gamma)
        if dbeta is None:
            dbeta = torch.empty_like(gamma)
        _need(dgamma, "dgamma", torch.float32, (dim,))
        _need(dbeta, "dbeta", torch.float32, (dim,))
        if scratch is None:
            scratch = _bytes(self.workspace(T)[1], h.device)
        _need_buf(scratch, "scratch")
        ttc_norm_bwd(self.desc, T, dy.data_ptr(), h.data_ptr(), gamma.data_ptr(), _ptr(dh), saved.data_ptr(),
                     _nbytes(saved), dx.data_ptr(), dgamma.data_ptr(), dbeta.data_ptr(), scratch.data_ptr(),
                     _nbytes(scratch), _stream())
        return dx, dgamma, dbeta
