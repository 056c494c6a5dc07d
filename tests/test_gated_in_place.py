"""glu_backward in place: an output at an operand's address needs that operand's pitch."""
import pytest
import torch

import matrix_aware_optimizer_amd as mao
from test_gated import BF, EINVAL, OK, P, backward_call


@pytest.mark.parametrize("out,ld", [("dG", "ldd"), ("dU", "ldd"), ("H", "ldh")])
@pytest.mark.parametrize("operand,pitch", [("dH", "lddh"), ("G", "ldg"), ("U", "ldg")])
def test_another_pitch_is_refused(out, ld, operand, pitch):
    assert backward_call(**{out: P[9], operand: P[9], ld: 48}) == EINVAL
    assert backward_call(**{out: P[9], operand: P[9], pitch: 48}) == EINVAL
    assert backward_call(**{out: P[9], operand: P[9], ld: 48}, t=0) == OK          # nothing is written


@pytest.mark.gpu
def test_in_place_on_the_gpu():
    wide = torch.randn(30, 50, device="cuda").to(BF)
    dh, g, u = wide[:, :40], torch.randn(30, 40, device="cuda").to(BF), torch.randn(30, 40, device="cuda").to(BF)
    want = [torch.empty(30, 40, dtype=BF, device="cuda") for _ in range(3)]
    mao.glu_backward(dh, g, u, want[0], want[1], h=want[2])
    packed = wide.view(-1)[:1200].view(30, 40)                   # at dh's address, with another pitch
    before = wide.clone()
    with pytest.raises(mao.MuonError):
        mao.glu_backward(dh, g, u, packed, u)
    with pytest.raises(mao.MuonError):
        mao.glu_backward(dh, g, u, g, u, h=packed)
    assert torch.equal(wide, before)
    one = [t[:1].clone() for t in (g, u)]
    first = wide[:1].clone()
    mao.glu_backward(first[:, :40], *one, first.view(-1)[:40].view(1, 40), one[1])      # one row has no pitch
    assert torch.equal(first[:, :40], want[0][:1]) and torch.equal(one[1], want[1][:1])
    mao.glu_backward(dh, g, u, g, u, h=dh)
    assert torch.equal(g, want[0]) and torch.equal(u, want[1]) and torch.equal(dh, want[2]) and torch.equal(wide[:, 40:], before[:, 40:])
