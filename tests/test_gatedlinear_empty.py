"""A gated block without inputs or without outputs: every call has its (empty or zero) result."""
import pytest
import torch

from test_gatedlinear import block, host, ones  # noqa: F401


def forward_and_backward(lin, device, tokens=7):
    out, inp = lin.Wg.shape
    x = ones(tokens, inp, device=device).requires_grad_()
    h = lin(x)
    assert h.shape == (tokens, out) and (h == 0).all()
    h.backward(torch.ones_like(h))
    assert x.grad.shape == x.shape and (x.grad == 0).all()
    return x


def whole_step(lin, device, tokens=7):
    x, out = forward_and_backward(lin, device, tokens), lin.Wg.shape[0]
    lin.step()
    lin.quantize()
    h = lin.answer(x.detach())
    assert h.shape == (tokens, out) and (h == 0).all()


SIZES = [(40, 0), (0, 40), (0, 0)]


@pytest.mark.parametrize("out,inp", SIZES)
def test_gradients_of_empty_blocks(host, out, inp):
    forward_and_backward(block(out, inp), "cpu")


@pytest.mark.gpu
@pytest.mark.parametrize("out,inp", SIZES)
def test_gradients_of_empty_blocks_on_the_gpu(out, inp):
    forward_and_backward(block(out, inp, device="cuda"), "cuda")


@pytest.mark.parametrize("out,inp", SIZES)
def test_empty_blocks(host, out, inp):
    whole_step(block(out, inp), "cpu")
    assert not [name for name, _, _ in host if name in ("ns_orthogonalize", "apply_update_dense")]     # they refuse empty matrices


@pytest.mark.gpu
@pytest.mark.parametrize("out,inp", SIZES)
def test_empty_blocks_on_the_gpu(out, inp):
    whole_step(block(out, inp, device="cuda"), "cuda")
