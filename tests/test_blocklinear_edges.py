"""BlockLinear where it is used out of the ordinary: order of calls, empty, strided and mismatched inputs."""
import pytest
import torch

import matrix_aware_optimizer_amd as mao
from matrix_aware_optimizer_amd import _abi


@pytest.fixture
def host(monkeypatch):
    """Layers on the CPU: the kernels are left out and the calls that would be made are recorded."""
    calls = []

    class Plan:
        def __init__(self, *args, **how):
            pass

        def __call__(self):
            calls.append("update")

    monkeypatch.setattr(_abi, "PreparedNSBlocks", Plan)
    monkeypatch.setattr(_abi, "fp8_quantize", lambda x, *rest, **how: calls.append(("quantize", x)))
    monkeypatch.setattr(_abi, "fp8_gemm", lambda a, sa, b, sb, c, **how: (calls.append(("gemm", c)), c.zero_()))
    return calls


def layer(out=64, inp=96, device="cpu", **how):
    return mao.BlockLinear(torch.ones(out, inp, device=device), head_dim=32, **how)


# ---------------------------------------------------------------------------
# a backward after the weights have changed
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("change", ["step", "requantize"])
def test_backward_after_a_change_of_the_weights_raises(host, change):
    lin = layer()
    x = torch.ones(5, 96, requires_grad=True)
    y = lin(x)
    _, saved = lin.forward(x.detach())
    getattr(lin, change)()
    del host[:]
    with pytest.raises(RuntimeError, match="requantised"):
        y.backward(torch.ones_like(y))
    with pytest.raises(RuntimeError, match="requantised"):
        lin.backward(torch.ones(5, 64), saved)
    assert not host and not lin._accumulating            # the momentum was not touched
    assert lin.backward(torch.ones(5, 64), saved, need_dx=False) is None
    lin(torch.ones(5, 96)).backward(torch.ones(5, 64))   # a new forward is free to go back
    y = lin(x)
    y.backward(torch.ones_like(y))
    assert x.grad.shape == x.shape


def test_several_forwards_between_steps(host):
    lin = layer()
    x = [torch.ones(n, 96, requires_grad=True) for n in (2, 3)]
    y = [lin(v) for v in x]
    for v in reversed(y):
        v.backward(torch.ones_like(v))
    lin.step()
    assert all(v.grad is not None for v in x)


def test_a_momentum_gradient_alone_may_come_late(host):
    """Without an input gradient backward reads nothing of the weights."""
    lin = layer()
    y = lin(torch.ones(5, 96))
    lin.step()
    y.backward(torch.ones_like(y))
    assert lin._accumulating


@pytest.mark.gpu
def test_stale_weights_on_the_gpu():
    lin = layer(device="cuda")
    x = torch.ones(5, 96, device="cuda", requires_grad=True)
    y = lin(x)
    y.backward(torch.ones_like(y))
    assert torch.equal(x.grad, torch.full_like(x, 64.0))
    y = lin(x)
    lin.step()
    M = lin.M.clone()
    with pytest.raises(RuntimeError, match="requantised"):
        y.backward(torch.ones_like(y))
    assert torch.equal(lin.M, M)


# ---------------------------------------------------------------------------
# no tokens
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("shape", [(0, 96), (2, 0, 96), (0, 3, 96)])
@pytest.mark.parametrize("grad", [False, True])
def test_no_tokens(host, shape, grad):
    lin = layer()
    x = torch.ones(shape, requires_grad=True)
    with torch.set_grad_enabled(grad):
        y = lin(x)
    assert y.shape == (*shape[:-1], 64)
    if grad:
        y.backward(torch.ones_like(y))
        assert x.grad.shape == shape and lin._accumulating


@pytest.mark.gpu
def test_no_tokens_on_the_gpu():
    """A step without tokens decays the momentum and moves nothing else into it."""
    lin = layer(device="cuda", beta=0.5)
    lin.M.fill_(2.0)
    x = torch.ones(2, 0, 96, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    y = lin(x)
    assert y.shape == (2, 0, 64)
    y.backward(torch.ones_like(y))
    assert x.grad.shape == x.shape and (lin.M == 1.0).all()


# ---------------------------------------------------------------------------
# rows that are not contiguous or not aligned
# ---------------------------------------------------------------------------

def odd_views(device, dtype=torch.float32):
    """Inputs [tokens, 96] as programs have them: transposed, of every other column, repeated rows, an unaligned start."""
    gen = torch.Generator().manual_seed(1)

    def ints(*shape):
        return torch.randint(-3, 4, shape, generator=gen).to(device, dtype)

    return {"transposed": ints(96, 7).t(), "every other": ints(7, 192)[:, ::2], "expanded": ints(96).expand(7, 96),
            "unaligned": ints(7 * 96 + 1)[1:].view(7, 96), "padded": ints(7, 100)[:, 2:98], "aligned": ints(7, 104)[:, 8:],
            "three": ints(3, 96, 7).transpose(1, 2)}


def as_the_kernels_read(t):
    return t.stride(-1) == 1 and t.stride(0) >= t.shape[1] and t.data_ptr() % 16 == 0


@pytest.mark.parametrize("kind", list(odd_views("cpu")))
def test_rows_reach_the_kernels_contiguous_and_aligned(host, kind):
    lin = layer()
    x = odd_views("cpu")[kind].requires_grad_()
    dy = torch.ones(64).expand(*x.shape[:-1], 64)
    y = lin(x)
    y.backward(dy)
    read = [call[1] for call in host if call[0] == "quantize"][1:]      # the first is W
    assert len(read) == 2 and all(as_the_kernels_read(t) for t in read)
    assert torch.equal(read[0], x.detach().reshape(-1, 96)) and torch.equal(read[1], dy.reshape(-1, 64))
    if kind == "aligned":
        assert read[0].data_ptr() == x.data_ptr()                       # nothing is copied without need


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", list(odd_views("cpu")))
def test_odd_rows_on_the_gpu(kind, dtype):
    x = odd_views("cuda", dtype)[kind]
    lin, plain = (layer(device="cuda", alpha=1.0) for _ in range(2))
    got, want = lin(x), plain(x.contiguous().clone())
    assert torch.equal(got, want)
    dy = torch.ones(got.numel() + 1, device="cuda", dtype=dtype)[1:].view(-1, 64)      # unaligned
    got.reshape(-1, 64).backward(dy)
    want.reshape(-1, 64).backward(dy.clone())
    assert torch.equal(lin.M, plain.M) and lin.M.abs().sum() > 0


# ---------------------------------------------------------------------------
# sizes that do not belong together
# ---------------------------------------------------------------------------

def test_sizes_of_inputs_and_gradients(host):
    """Widths are padded to 128 for the products, so that a wrong one within the padding would multiply silently."""
    lin = layer()                                          # [64, 96]
    for x in (torch.ones(5, 95), torch.ones(5, 100), torch.ones(2, 5, 128), torch.ones(96)[:95], torch.ones(5, 0)):
        with pytest.raises(ValueError, match="96"):
            lin(x)
    with pytest.raises(ValueError, match="96"):
        lin.forward(torch.ones(5, 100), train=False)
    _, saved = lin.forward(torch.ones(5, 96))
    del host[:]
    for dy in (torch.ones(5, 65), torch.ones(5, 100), torch.ones(6, 64), torch.ones(100, 64)):
        for need_dx in (False, True):
            with pytest.raises(ValueError):
                lin.backward(dy, saved, need_dx)
    assert not host and not lin._accumulating
    lin.backward(torch.ones(5, 64), saved)


def test_a_single_row(host):
    x = torch.ones(96, requires_grad=True)
    y = layer()(x)
    assert y.shape == (64,)
    y.sum().backward()
    assert x.grad.shape == (96,)
