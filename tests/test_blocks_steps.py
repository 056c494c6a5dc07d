"""How many steps ns_blocks takes: rounding in the Gram matrix grows by the square of a step's factor."""
import pytest
import torch

import matrix_aware_optimizer_amd as mao
from workloads import CUBIC, QUINTIC

OK, EINVAL = 0, -1


def status(coeffs, steps, update=False):
    """The numbers alone are looked at in a call without problems."""
    L = mao.lib()
    if update:
        return L.ns_blocks_update(None, 0, *coeffs, steps, 0.1, 0.0, 1.0, None, 0, None)
    return L.ns_blocks(None, 0, *coeffs, steps, None, 0, None)


@pytest.mark.parametrize("update", [False, True])
@pytest.mark.parametrize("coeffs,most", [
    (QUINTIC, 12),                  # 3.4445^12 = 2^21.4
    (CUBIC, 37),                    # 1.5^37 = 2^21.6
    ((2.0, -1.5, 0.5), 22),         # 2^22 exactly
    ((1.0, 7.0, 0.0), 7),           # largest at x = 1: 8^7 = 2^21
    ((1.0, 12.0, -12.0), 11),       # largest inside: 4 at x = 1/2, 4^11 = 2^22
    ((-2.0, 1.5, 0.0), 22),         # sizes count, not signs
])
def test_most_steps(coeffs, most, update):
    assert status(coeffs, 0, update) == OK and status(coeffs, most, update) == OK
    assert status(coeffs, most + 1, update) == EINVAL and status(coeffs, 2 ** 31 - 1, update) == EINVAL


def test_steps_that_do_not_grow():
    assert status((1.0, -0.5, 0.0), 10 ** 6) == OK
    assert status((float("inf"), 0.0, 0.0), 1) == EINVAL and status((float("inf"), 0.0, 0.0), 0) == OK


def test_a_plan_raises_at_once():
    x = torch.zeros(2, 4, 8)
    for how in ({}, dict(eta=0.1)):
        with pytest.raises(Exception, match="ns_blocks"):
            mao.PreparedNSBlocks([(x, x)], *QUINTIC, 13, **how)


@pytest.mark.gpu
def test_padding_of_the_most_steps():
    """The most steps on a short side inside a strip: the padding's part of T stays finite and out of U."""
    import numpy as np
    import oracle.muon_oracle as O
    for coeffs, steps in ((QUINTIC, 12), (CUBIC, 37)):
        M = torch.from_numpy(np.random.default_rng(1).standard_normal((40, 400)).astype(np.float32))
        U = torch.empty((40, 400), device="cuda")
        mao.ns_blocks([(M.cuda(), U)], *coeffs, steps)
        ref = O.newton_schulz(M.double().numpy(), *(float(np.float32(v)) for v in coeffs), steps)
        assert np.linalg.norm(U.double().cpu().numpy() - ref) <= 2.0 ** -23 * np.linalg.norm(ref)
