"""A linear layer in fp8 whose heads Muon orthogonalises one by one.

Host-side orchestration of fp8_quantize, fp8_gemm and ns_blocks_update for one
projection of an attention layer: it owns the layer's buffers (through torch)
and calls the C ABI in the order of a training step.  All arithmetic runs in
libmuon's kernels.

    y  = x W^T                           forward       (W in e4m3 blocks of 128 x 128)
    dx = dy W                            backward      (dy in e5m2, W transposed)
    M <- beta M + alpha dy^T x           backward      (the gradient is never written)
    W <- (1 - eta decay) W - eta scale NS(M)   step    (each head by itself)
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _abi


def _rows(t: torch.Tensor) -> torch.Tensor:
    """``t`` [rows, cols] as the quantiser reads it, contiguous rows from a 16-byte aligned start: a copy where it is not."""
    rows, cols = t.shape
    if (cols <= 1 or t.stride(1) == 1) and (rows <= 1 or t.stride(0) >= cols) and t.data_ptr() % 16 == 0:
        return t
    return t.clone(memory_format=torch.contiguous_format)


class BlockLinear:
    """One projection ``W`` [out, in] with its fp8 codes and its momentum.

    ``heads`` says how W is cut for the update: ``"rows"`` (head h is rows h d .. of a
    query, key or value projection), ``"cols"`` (columns of an output projection);
    ``head_dim`` = d, at most MUON_BLOCKS_MAX_SHORT.  ``W`` (fp32 or bf16) is updated in
    place; the momentum is fp32 unless ``m_dtype`` says otherwise.
    """

    def __init__(self, W: torch.Tensor, head_dim: int, heads: str = "rows", m_dtype=torch.float32,
                 beta: float = 0.95, alpha: Optional[float] = None, eta: float = 0.02, decay: float = 0.0,
                 scale: float = 1.0, coeffs=(3.4445, -4.7750, 2.0315), ns_steps: int = 5):
        if W.dim() != 2 or not W.is_contiguous():
            raise ValueError("W must be a contiguous [out, in] matrix")
        if heads not in ("rows", "cols"):
            raise ValueError("heads must be 'rows' or 'cols'")
        cut = W.shape[0 if heads == "rows" else 1]
        if not 0 < head_dim <= _abi.MUON_BLOCKS_MAX_SHORT or cut % head_dim != 0:
            raise ValueError(f"head_dim must divide {cut} and lie in 1 .. {_abi.MUON_BLOCKS_MAX_SHORT}")
        self.W = W
        self.M = torch.zeros(W.shape, dtype=m_dtype, device=W.device)
        self.beta = float(beta)
        self.alpha = float(1.0 - beta if alpha is None else alpha)
        out, inp = W.shape
        self.wq, self.ws = _abi.fp8_buffers(out, inp, device=W.device)
        self.wqt, self.wst = _abi.fp8_buffers(inp, out, device=W.device)
        self._update = _abi.PreparedNSBlocks([(self._blocks(self.M, heads, head_dim), self._blocks(W, heads, head_dim))],
                                             *coeffs, ns_steps, eta=eta, decay=decay, scale=scale)
        self._accumulating = False      # a backward since the last step: later ones add without beta
        self._generation = 0            # how often the codes were written: a backward needs those of its forward
        self.requantize()

    @staticmethod
    def _blocks(t: torch.Tensor, heads: str, d: int) -> torch.Tensor:
        rows, cols = t.shape
        return t.view(rows // d, d, cols) if heads == "rows" else t.view(rows, cols // d, d).permute(1, 0, 2)

    def requantize(self) -> None:
        """Codes of W and of its transpose, from the current W (after the caller wrote to it)."""
        _abi.fp8_quantize(self.W, self.wq, self.ws, self.wqt, self.wst, block_rows=_abi.MUON_FP8_GROUP)
        self._generation += 1

    def forward(self, x: torch.Tensor, train: bool = True):
        """(y, saved) for x [tokens, in] in bf16 or fp32; ``saved`` (None unless ``train``) goes to backward."""
        if x.dim() != 2 or x.shape[1] != self.W.shape[1]:
            raise ValueError(f"x must be [tokens, {self.W.shape[1]}]")
        x = _rows(x)
        tokens, inp = x.shape
        xq, xs = _abi.fp8_buffers(tokens, inp, device=x.device)
        saved = _abi.fp8_buffers(inp, tokens, device=x.device) if train else None
        _abi.fp8_quantize(x, xq, xs, *(saved if train else (None, None)))
        y = torch.empty((tokens, self.W.shape[0]), dtype=x.dtype, device=x.device)
        _abi.fp8_gemm(xq, xs, self.wq, self.ws, y)
        return y, (*saved, tokens, self._generation) if train else None

    def backward(self, dy: torch.Tensor, saved, need_dx: bool = True) -> Optional[torch.Tensor]:
        """Adds dy^T x to the momentum (decayed by beta once per step) and returns dx.

        dx needs the weights of the forward: after a :meth:`step` or :meth:`requantize` in between it raises."""
        xqt, xst, tokens, generation = saved
        out = self.W.shape[0]
        if dy.shape != (tokens, out):
            raise ValueError(f"dy must be [{tokens}, {out}], as the forward's y")
        if need_dx and generation != self._generation:
            raise RuntimeError("the weights were requantised after this forward: their codes, which dx needs, are gone "
                               "(run backward before step(), or without the input gradient)")
        dy = _rows(dy)
        dq, ds = _abi.fp8_buffers(tokens, out, "e5m2", device=dy.device) if need_dx else (None, None)
        dqt, dst = _abi.fp8_buffers(out, tokens, "e5m2", device=dy.device)
        _abi.fp8_quantize(dy, dq, ds, dqt, dst)
        _abi.fp8_gemm(dqt, dst, xqt, xst, self.M, alpha=self.alpha, beta=1.0 if self._accumulating else self.beta)
        self._accumulating = True
        if not need_dx:
            return None
        dx = torch.empty((tokens, self.W.shape[1]), dtype=dy.dtype, device=dy.device)
        _abi.fp8_gemm(dq, ds, self.wqt, self.wst, dx)
        return dx

    def step(self) -> None:
        """The update of W from the momentum, head by head, and the codes of the new W."""
        self._update()
        self._accumulating = False
        self.requantize()

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        """y for x [..., in], differentiable: backward goes through :meth:`backward`."""
        if x.dim() == 0 or x.shape[-1] != self.W.shape[1]:
            raise ValueError(f"x must be [..., {self.W.shape[1]}]")
        flat = x.reshape(-1, x.shape[-1])
        if torch.is_grad_enabled():
            # W is no leaf of autograd (its gradient goes into M), so the node hangs on x or on an empty anchor
            anchor = torch.empty(0, device=x.device, requires_grad=True)
            y = _BlockLinearFn.apply(flat, anchor, self)
        else:
            y = self.forward(flat, train=False)[0]
        return y.view(*x.shape[:-1], self.W.shape[0])


class _BlockLinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, anchor, layer):
        y, saved = layer.forward(x.detach())
        ctx.layer, ctx.rest = layer, saved[2:]
        ctx.save_for_backward(*saved[:2])
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        dx = ctx.layer.backward(dy, (*ctx.saved_tensors, *ctx.rest), ctx.needs_input_grad[0])
        return dx, None, None
