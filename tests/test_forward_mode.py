"""Tangents of forward-mode differentiation, which the layers have no rule for, are refused and never dropped."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import matrix_aware_optimizer_amd as mao
from matrix_aware_optimizer_amd import _abi
from test_gatedlinear import block, host, ones  # noqa: F401


def projection(device):
    return mao.BlockLinear(torch.ones(64, 96, dtype=torch.bfloat16, device=device), head_dim=16)


@pytest.fixture
def quiet(host, monkeypatch):
    """The fp8 kernels left out too."""
    for name in ("fp8_quantize", "fp8_gemm"):
        monkeypatch.setattr(_abi, name, lambda *args, **how: None)
    monkeypatch.setattr(_abi, "PreparedNSBlocks", lambda *args, **how: lambda: None)


def refuses(lin, x, grad):
    with fwd.dual_level():
        dual = fwd.make_dual(x, torch.ones_like(x))
        with torch.set_grad_enabled(grad), pytest.raises(RuntimeError, match="forward|jvp"):
            lin(dual)
        with torch.set_grad_enabled(grad):
            assert lin(x).shape == (5, 64)          # without a tangent, inside of a dual level
    with torch.set_grad_enabled(grad):
        assert lin(x).shape == (5, 64)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("make", [block, projection])
def test_tangents_are_refused(quiet, make, grad):
    refuses(make(device="cpu"), ones(5, 96), grad)


def test_answers_refuse_tangents(quiet):
    lin = block()
    lin.quantize()
    with fwd.dual_level(), pytest.raises(RuntimeError, match="forward"):
        lin.answer(fwd.make_dual(ones(5, 96), ones(5, 96)))
    with torch.inference_mode():
        assert lin.answer(ones(5, 96)).shape == (5, 64) and lin(ones(5, 96)).shape == (5, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("make", [block, projection])
def test_tangents_are_refused_on_the_gpu(make):
    for grad in (False, True):
        refuses(make(device="cuda"), ones(5, 96, device="cuda"), grad)
