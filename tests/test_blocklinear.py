"""BlockLinear: the fp8 products, their gradients and the head-wise update as one layer."""
import numpy as np
import pytest
import torch

import matrix_aware_optimizer_amd as mao
import oracle.fp8_oracle as F
import oracle.muon_oracle as O
from workloads import QUINTIC


def test_refusals():
    with pytest.raises(ValueError):
        mao.BlockLinear(torch.zeros(8, 8), head_dim=4, heads="both")
    with pytest.raises(ValueError):
        mao.BlockLinear(torch.zeros(8, 8), head_dim=3)
    with pytest.raises(ValueError):
        mao.BlockLinear(torch.zeros(512, 8), head_dim=256)
    with pytest.raises(ValueError):
        mao.BlockLinear(torch.zeros(8, 16)[:, ::2], head_dim=4)


def ints(shape, seed, top=3):
    return torch.from_numpy(np.random.default_rng(seed).integers(-top, top + 1, shape).astype(np.float32)).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,out,inp", [(1, 64, 64), (5, 96, 160), (130, 128, 72), (300, 192, 256)])
def test_gradients_are_the_formulas_and_the_differences(tokens, out, inp):
    """Small integers are their own codes (scales are powers of two, at most three bits), so the layer is exactly the
    bilinear map, and differences with a step of one are its exact derivatives."""
    W, x, dy = ints((out, inp), 1), ints((tokens, inp), 2), ints((tokens, out), 3, 1)
    layer = mao.BlockLinear(W.clone(), head_dim=32 if out % 32 == 0 else 16, beta=0.5, alpha=1.0)
    layer.M.copy_(ints((out, inp), 4))
    M0 = layer.M.clone()
    xg = x.clone().requires_grad_()
    y = layer(xg)
    assert torch.equal(y.detach().double(), x.double() @ W.double().t())
    y.backward(dy)
    assert torch.equal(xg.grad.double(), dy.double() @ W.double())
    assert torch.equal(layer.M.double(), 0.5 * M0.double() + dy.double().t() @ x.double())
    # differences of f(x, W) = <dy, layer(x)> in single entries
    f = lambda a, w: float((dy.double() * mao.BlockLinear(w, head_dim=layer_dim(w)).forward(a, train=False)[0].double()).sum())  # noqa: E731
    base = f(x, W.clone())
    grad_w = (layer.M - 0.5 * M0).double()
    rng = np.random.default_rng(5)
    for _ in range(3):
        t, i, o = rng.integers(tokens), rng.integers(inp), rng.integers(out)
        moved = x.clone()
        moved[t, i] += 1
        assert f(moved, W.clone()) - base == float(xg.grad[t, i])
        moved = W.clone()
        moved[o, i] += 1
        assert f(x, moved) - base == float(grad_w[o, i])


def layer_dim(w):
    return 32 if w.shape[0] % 32 == 0 else 16


def quantized(t, fmt, block_rows=1):
    q, ex = F.quantize(t.double().cpu().numpy(), fmt, block_rows)
    return q * np.repeat(2.0 ** ex, 128, axis=1)


@pytest.mark.gpu
@pytest.mark.parametrize("heads", ["rows", "cols"])
@pytest.mark.parametrize("w_dtype,m_dtype", [(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
def test_one_training_step(heads, w_dtype, m_dtype):
    """Forward, backward twice (accumulated) and the update against the 64-bit oracles."""
    tokens, out, inp, d = 200, 256, 320, 64
    g = torch.Generator().manual_seed(7)
    W = (0.05 * torch.randn(out, inp, generator=g)).to(w_dtype)
    layer = mao.BlockLinear(W.cuda(), head_dim=d, heads=heads, m_dtype=m_dtype, beta=0.5, alpha=0.25, eta=0.02, decay=0.1,
                            scale=2.0)
    Wv, Wtv = quantized(W, "e4m3", 128)[:, :inp], quantized(W.t(), "e4m3", 128)[:, :out]
    np.testing.assert_array_equal(Wv, Wtv.T)                     # one scale per block: both orientations are the same
    M = np.zeros((out, inp))
    eps_m = torch.finfo(m_dtype).eps / 2
    for k in range(2):
        x = torch.randn(tokens, inp, generator=g).to(torch.bfloat16)
        dy = (0.01 * torch.randn(tokens, out, generator=g)).to(torch.bfloat16)
        y, saved = layer.forward(x.cuda())
        dx = layer.backward(dy.cuda(), saved)
        for got, a, b in ((y, quantized(x, "e4m3")[:, :inp], Wv), (dx, quantized(dy, "e5m2")[:, :out], Wv.T)):
            ref = a @ b.T
            # bf16 result of the fp8 instructions: half a step, and 2^-13 of the largest of eight products, eight times
            assert np.linalg.norm(got.double().cpu().numpy() - ref) <= (2.0 ** -9 + 2.0 ** -10) * np.linalg.norm(ref)
        grad = quantized(dy.t(), "e5m2")[:, :tokens] @ quantized(x.t(), "e4m3")[:, :tokens].T
        M = (0.5 if k == 0 else 1.0) * M + 0.25 * grad
        err = np.linalg.norm(layer.M.double().cpu().numpy() - M)
        assert err <= (k + 1) * (eps_m + 256 * 2.0 ** -23) * np.linalg.norm(M)
    M = layer.M.double().cpu().numpy()                           # the update from the momentum as stored
    cut = (lambda t, h: t[h * d:(h + 1) * d]) if heads == "rows" else (lambda t, h: t[:, h * d:(h + 1) * d])
    layer.step()
    W64 = W.double().numpy()
    eps_w = torch.finfo(w_dtype).eps / 2
    for h in range((out if heads == "rows" else inp) // d):
        U = O.newton_schulz(cut(M, h), *QUINTIC, 5)
        ref = (1 - 0.02 * 0.1) * cut(W64, h) - 0.04 * U
        err = np.linalg.norm(cut(layer.W.double().cpu().numpy(), h) - ref)
        # half a step of W, and the direction's fp32 rounding (sums of 64 and 320 terms, 21 products)
        assert err <= eps_w * np.linalg.norm(ref) + 2 * 8 * 2.0 ** -24 * (18 + 21 * 8) * 0.04 * np.linalg.norm(U)
    # the codes follow the new weights
    q, ex = F.quantize(layer.W.double().cpu().numpy(), "e4m3", 128)
    np.testing.assert_array_equal(F.decode(layer.wq.view(torch.uint8).cpu().numpy(), "e4m3"), q)
    np.testing.assert_array_equal(layer.ws.cpu().numpy(), F.pack_scales(ex))


@pytest.mark.gpu
def test_captured_step_equals_eager_steps():
    """A whole step (forward, backward, update, codes) as a graph, replayed on new tokens, against the same steps run
    eagerly, while an autograd graph over another layer is alive."""
    torch.manual_seed(3)
    W0 = (0.05 * torch.randn(128, 256, device="cuda")).to(torch.bfloat16)
    a, b = (mao.BlockLinear(W0.clone(), head_dim=32, beta=0.9, eta=0.05) for _ in range(2))
    alive = mao.BlockLinear(W0.clone(), head_dim=32)
    xa = torch.randn(64, 256, device="cuda").to(torch.bfloat16).requires_grad_()
    pending = alive(xa).float().square().sum()
    x, dy = torch.zeros(64, 256, device="cuda", dtype=torch.bfloat16), torch.zeros(64, 128, device="cuda", dtype=torch.bfloat16)

    def step(layer):
        _, saved = layer.forward(x)
        layer.backward(dy, saved, need_dx=False)
        layer.step()

    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step(a)
    for k in range(3):
        x.copy_(torch.randn(64, 256, device="cuda"))
        dy.copy_(torch.randn(64, 128, device="cuda"))
        g.replay()
        step(b)
        torch.cuda.synchronize()
        assert torch.equal(a.W, b.W) and torch.equal(a.M, b.M)
        assert torch.equal(a.wq.view(torch.uint8), b.wq.view(torch.uint8))
    assert not torch.equal(a.W, W0)
    pending.backward()
    assert torch.isfinite(xa.grad.float()).all()


@pytest.mark.gpu
def test_example_learns():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_projections_fp8.py")
    spec = importlib.util.spec_from_file_location("attention_projections_fp8", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses = mod.main(["--tokens", "512", "--steps", "20", "--width", "256", "--head-dim", "64"])
    assert np.isfinite(losses).all() and np.mean(losses[-3:]) < 0.8 * losses[0]


@pytest.mark.gpu
def test_leading_dimensions_and_no_input_gradient():
    layer = mao.BlockLinear(ints((64, 128), 1), head_dim=32)
    x = ints((3, 5, 128), 2)
    y = layer(x)                               # x needs no gradient: the momentum still gets its own
    assert y.shape == (3, 5, 64)
    y.backward(torch.ones_like(y))
    assert layer.M.abs().sum() > 0
    with torch.no_grad():
        assert torch.equal(layer(x), y.detach())
