"""The life of GatedLinear's int8 codes: what a captured answer reads, and what old codes answer."""
import pytest
import torch

import matrix_aware_optimizer_amd as mao
from test_gatedlinear import BF, block, host, ones, randn  # noqa: F401


# ---------------------------------------------------------------------------
# host side
# ---------------------------------------------------------------------------

def test_codes_and_scales_stay_where_they_are(host):
    lin = block(out=66)
    seen = set()
    for _ in range(3):
        lin.quantize()
        lin.answer(ones(5, 96))
        quantized = [args for name, args, _ in host if name == "int8_quantize"][:2]
        answered = [args for name, args, _ in host if name == "int8_glu"][-1]
        places = tuple(t.data_ptr() for args in quantized for t in args[1:3])
        assert places == tuple(t.data_ptr() for t in answered[2:6]) and all(p % 16 == 0 for p in places) and len(set(places)) == 4
        seen.add(places)
        del host[:]
        keep = torch.empty(66, 128, dtype=torch.int8)       # the allocator's next block of that size
        lin.step()
        del keep
    assert len(seen) == 1


@pytest.mark.parametrize("inference", [False, True])
def test_scales_are_nan_until_quantize_and_after_a_change(host, inference):
    with torch.inference_mode(inference):
        lin = block()
        lin.quantize()
    for change in (lin.step, lin.weights_changed):
        scales = [args[2] for name, args, _ in host if name == "int8_quantize"][:2]
        for s in scales:
            s.fill_(1.0)
        change()
        assert all(torch.isnan(s).all() for s in scales)
        with pytest.raises(RuntimeError, match="quantize"):
            lin.answer(ones(5, 96))
        lin.quantize()
        lin.answer(ones(5, 96))


def test_weights_changed_ends_older_forwards(host):
    lin = block()
    x = ones(5, 96).requires_grad_()
    y = lin(x)
    lin.backward(ones(5, 64), lin.forward(x.detach())[1])
    lin.weights_changed()
    assert lin._accumulating                # the gradients so far stay
    with pytest.raises(RuntimeError, match="changed"):
        y.backward(torch.ones_like(y))


# ---------------------------------------------------------------------------
# GPU
# ---------------------------------------------------------------------------

def graph_of(call):
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = call()
    return g, out


def fresh_answer(lin, x):
    """The answer of another block with the same weights."""
    other = mao.GatedLinear(lin.Wg.clone(), lin.Wu.clone(), act=lin.act)
    other.quantize()
    return other.answer(x)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [3, 70])
def test_a_captured_answer_follows_the_weights(tokens):
    """Replays with new codes give the new weights' answers, replays between a step and quantize() give NaN."""
    lin = mao.GatedLinear(*(randn(130, 200, seed=s, size=0.1).cuda() for s in (1, 2)), eta=0.3)
    x = randn(tokens, 200, seed=3).cuda()
    lin.quantize()
    want = lin.answer(x)
    g, h = graph_of(lambda: lin.answer(x))
    for k in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, want) and torch.equal(h, fresh_answer(lin, x))
        _, saved = lin.forward(randn(50, 200, seed=10 + k).cuda())
        lin.backward(randn(50, 130, seed=20 + k).cuda(), saved)
        lin.step()
        taken = [torch.full((130, 256), 77, dtype=torch.int8, device="cuda") for _ in range(4)]     # freed codes would be among them
        g.replay()
        torch.cuda.synchronize()
        assert torch.isnan(h).all()
        lin.quantize()
        before, want = want, lin.answer(x)
        assert not torch.equal(before, want)
        del taken


@pytest.mark.gpu
def test_a_replayed_step_ends_codes_and_older_forwards():
    """A graph's step is not seen by the host: old codes answer NaN, also where they were made after the capture, and so does dx."""
    lin = mao.GatedLinear(*(randn(130, 200, seed=s, size=0.1).cuda() for s in (1, 2)), eta=0.3)
    x, dh = randn(50, 200, seed=3).cuda(), randn(50, 130, seed=4).cuda()

    def step():
        lin.backward(dh, lin.forward(x)[1], need_dx=False)
        lin.step()

    g, _ = graph_of(step)
    for _ in range(3):
        lin.quantize()
        assert torch.equal(lin.answer(x), fresh_answer(lin, x))
        g.replay()
        assert torch.isnan(lin.answer(x)).all()
    xg = x.clone().requires_grad_()
    for replay in (False, True, False):             # dx of a forward before the replay
        xg.grad = None
        y = lin(xg)
        if replay:
            g.replay()
        y.backward(dh)
        assert (torch.isnan(xg.grad).all() if replay else torch.isfinite(xg.grad).all()) and torch.isfinite(lin.Mg).all()
    y = lin(xg)
    g.replay()
    lin.weights_changed()
    with pytest.raises(RuntimeError, match="changed"):
        y.backward(torch.ones_like(y))
    with pytest.raises(RuntimeError, match="quantize"):
        lin.answer(x)
    lin.quantize()
    assert torch.equal(lin.answer(x), fresh_answer(lin, x))


@pytest.mark.gpu
def test_step_quantize_and_answer_in_one_graph():
    lin = mao.GatedLinear(*(randn(130, 200, seed=s, size=0.1).cuda() for s in (1, 2)), eta=0.3)
    x, dh = randn(50, 200, seed=3).cuda(), randn(50, 130, seed=4).cuda()

    def all_of_it():
        lin.backward(dh, lin.forward(x)[1], need_dx=False)
        lin.step()
        lin.quantize()
        return lin.answer(x)

    g, h = graph_of(all_of_it)
    assert torch.isnan(lin.answer(x)).all()         # captured and not run: no codes yet
    seen = []
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, fresh_answer(lin, x)) and torch.equal(h, lin.answer(x))
        seen.append(h.clone())
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2]) and h.dtype == BF
