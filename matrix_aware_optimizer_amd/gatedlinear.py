"""The two projections of a gated feed-forward block, trained with Muon and answering in 8 bits.

Host-side orchestration of glu_forward, glu_backward, glu_weight_grad,
ns_orthogonalize and apply_update_dense for one block, and of int8_quantize and
int8_glu for its answers.  All arithmetic runs in libmuon's kernels.

    h  = act(x Wg^T) * (x Wu^T)                          forward
    dx, and M <- beta M + alpha dW for both matrices     backward (the gradients are never written)
    W <- W - eta NS(M) for both                          step     (each matrix orthogonalised by itself)
    h from int8 codes, a scale per output and token      quantize, answer
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _abi
from .blocklinear import _no_tangent, _rows


class GatedLinear:
    """``Wg`` and ``Wu`` [out, in] (contiguous, bf16) with their momenta; updated in place.

    The momenta are fp32 unless ``m_dtype`` says otherwise; ``act`` is one of silu, gelu, gelu_tanh, relu."""

    def __init__(self, Wg: torch.Tensor, Wu: torch.Tensor, act: str = "silu", m_dtype=torch.float32, beta: float = 0.95,
                 alpha: Optional[float] = None, eta: float = 0.02, coeffs=(3.4445, -4.7750, 2.0315), ns_steps: int = 5):
        for W in (Wg, Wu):
            if W.dim() != 2 or not W.is_contiguous() or W.dtype != torch.bfloat16 or W.shape != Wg.shape or W.device != Wg.device:
                raise ValueError("Wg and Wu must be contiguous bf16 [out, in] matrices of one shape on one device")
        if Wg.data_ptr() == Wu.data_ptr() and Wg.numel() > 0:
            raise ValueError("Wg and Wu must be two matrices")
        _abi._act_code(act)
        self.Wg, self.Wu, self.act = Wg, Wu, act
        self.Mg, self.Mu = (torch.zeros(W.shape, dtype=m_dtype, device=W.device) for W in (Wg, Wu))
        self.beta = float(beta)
        self.alpha = float(1.0 - beta if alpha is None else alpha)
        self.eta, self.coeffs, self.ns_steps = float(eta), tuple(float(c) for c in coeffs), int(ns_steps)
        self._accumulating = False      # a backward since the last step: later ones add without beta
        self._changes = 0
        # The int8 form of the weights keeps its place, so that a captured answer reads the codes of today.  The scales are NaN
        # where the codes are not those of the weights: an answer that a graph replays on them is NaN, not another weights' value.
        out = Wg.shape[0]
        with torch.inference_mode(False):
            self._scales = torch.full((2, -(-out // 4) * 4), float("nan"), dtype=torch.float32, device=Wg.device)[:, :out]
            self._replays = torch.zeros(1, dtype=torch.int32, device=Wg.device)     # of captured steps, which the host does not see
        self._captured = False          # there are such steps
        self._codes = None              # of Wg and of Wu, from the first quantize() on
        self._quantized = None          # state of the weights that the codes are of

    def _state(self):
        """Changes whenever the weights do, by step() or by torch operations on them (inference tensors have no such count)."""
        return (self._changes, *(0 if W.is_inference() else W._version for W in (self.Wg, self.Wu)))

    def _capturing(self) -> bool:
        return self.Wg.is_cuda and torch.cuda.is_current_stream_capturing()

    def weights_changed(self) -> None:
        """Ends the codes and the input gradients of older forwards, as :meth:`step` does.

        For changes that are not noticed: by other calls of the library, by captured torch operations, through ``.data``.
        A replayed step is noticed on the device alone: answers from older codes and dx of older forwards are NaN."""
        self._changes += 1
        self._scales.fill_(float("nan"))
        if self._capturing():
            self._replays.add_(1)
            self._captured = True

    def _flat(self, x: torch.Tensor) -> torch.Tensor:
        if x.dim() != 2 or x.shape[1] != self.Wg.shape[1]:
            raise ValueError(f"x must be [tokens, {self.Wg.shape[1]}]")
        return _rows(x)

    def forward(self, x: torch.Tensor, train: bool = True):
        """(h, saved) for x [tokens, in] in bf16; ``saved`` (None unless ``train``) goes to backward and holds x itself."""
        x = self._flat(x)
        shape = (x.shape[0], self.Wg.shape[0])
        h = torch.empty(shape, dtype=x.dtype, device=x.device)
        g, u = (torch.empty_like(h), torch.empty_like(h)) if train else (None, None)
        _abi.glu_forward(x, self.Wg, self.Wu, h, g, u, act=self.act)
        if not train:
            return h, None
        mark = self._replays.clone() if self._captured and not self._capturing() else None
        return h, (x, g, u, self._state(), mark)

    def backward(self, dh: torch.Tensor, saved, need_dx: bool = True) -> Optional[torch.Tensor]:
        """Adds both weight gradients to the momenta (decayed by beta once per step) and returns dx.

        dx needs the weights of the forward: after a change of them in between it raises (is NaN, after a replayed step)."""
        x, g, u, state, mark = saved
        if dh.shape != g.shape:
            raise ValueError(f"dh must be [{g.shape[0]}, {g.shape[1]}], as the forward's h")
        if need_dx and state != self._state():
            raise RuntimeError("the weights changed after this forward: dx needs those that it used "
                               "(run backward before step(), or without the input gradient)")
        dh = _rows(dh)
        dg, du = torch.empty_like(g), torch.empty_like(u)
        dx = torch.empty_like(x, memory_format=torch.contiguous_format) if need_dx else None
        _abi.glu_backward(dh, g, u, dg, du, *((self.Wg, self.Wu, dx) if need_dx else ()), act=self.act)
        if need_dx and mark is not None:
            dx.masked_fill_(mark != self._replays, float("nan"))
        _abi.glu_weight_grad(dg, du, x, self.Mg, self.Mu, alpha=self.alpha, beta=1.0 if self._accumulating else self.beta)
        self._accumulating = True
        return dx

    def step(self) -> None:
        """The update of both weights from their momenta, each orthogonalised as a whole."""
        if self.Wg.numel() > 0:
            U = [torch.empty_like(W) for W in (self.Wg, self.Wu)]
            _abi.ns_orthogonalize([(self.Mg, U[0], None), (self.Mu, U[1], None)], *self.coeffs, self.ns_steps)
            for W, direction in zip((self.Wg, self.Wu), U):
                _abi.apply_update_dense(W, direction, self.eta)
        self.weights_changed()
        self._accumulating = False

    def quantize(self) -> None:
        """int8 codes of the current weights, for :meth:`answer`, over the former ones: what still reads those on another
        stream has to be done, or to be waited for, as with any tensor that is written to."""
        if self._codes is None:
            self._codes = [_abi.int8_buffers(*W.shape, device=W.device)[0] for W in (self.Wg, self.Wu)]
        for W, q, s in zip((self.Wg, self.Wu), self._codes, self._scales):
            _abi.int8_quantize(W, q, s)
        self._quantized = self._state()

    def answer(self, x: torch.Tensor) -> torch.Tensor:
        """h for x [tokens, in] (bf16 or fp32) on int8 codes of the tokens and of the weights as of :meth:`quantize`; no gradients."""
        if self._quantized != self._state():
            raise RuntimeError("the weights have no codes, or changed after quantize()")
        _no_tangent(x)
        x = self._flat(x)
        q, s = _abi.int8_buffers(*x.shape, device=x.device)
        _abi.int8_quantize(x, q, s)
        h = torch.empty((x.shape[0], self.Wg.shape[0]), dtype=x.dtype, device=x.device)
        _abi.int8_glu(q, s, self._codes[0], self._scales[0], self._codes[1], self._scales[1], h, act=self.act)
        return h

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        """h for x [..., in], differentiable: backward goes through :meth:`backward`."""
        if x.dim() == 0 or x.shape[-1] != self.Wg.shape[1]:
            raise ValueError(f"x must be [..., {self.Wg.shape[1]}]")
        flat = x.reshape(x.shape[:-1].numel(), x.shape[-1])
        if torch.is_grad_enabled():
            # the weights are no leaves of autograd (their gradients go into the momenta), so the node hangs on x or on an empty anchor
            anchor = torch.empty(0, device=x.device, requires_grad=True)
            h = _GatedLinearFn.apply(flat, anchor, self)
        else:
            _no_tangent(flat)
            h = self.forward(flat, train=False)[0]
        return h.view(*x.shape[:-1], self.Wg.shape[0])


class _GatedLinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, anchor, block):
        h, saved = block.forward(x.detach())
        ctx.block, ctx.rest = block, saved[3:]
        ctx.save_for_backward(*saved[:3])
        return h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh):
        dx = ctx.block.backward(dh, (*ctx.saved_tensors, *ctx.rest), ctx.needs_input_grad[0])
        return dx, None, None
