"""Gates of the int8 block into fp32, entry by entry."""
import pytest
import torch

import matrix_aware_optimizer_amd as mao
from test_int8 import U, activation


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 40, 300])
def test_gates_in_fp32_keep_their_bits(m):
    """silu of gates down to -80 into fp32.

    g = float(code) times the scale, one rounding that is repeated here.  Of silu(g) = g / (1 + exp(-g)): exp is off by
    one step (2 U), the sum by half a step (U), the reciprocal by one step (2 U), a correction of exp's argument by U, the
    product by U: 7 U, and 8 with what their products add.  exp(-g) stays under 2^126, so that nothing underflows."""
    n = 255
    a = torch.zeros(m, 64, dtype=torch.int8, device="cuda")
    a[:, 0] = 1
    bg, bu = torch.zeros(n, 64, dtype=torch.int8, device="cuda"), torch.zeros(n, 64, dtype=torch.int8, device="cuda")
    k = torch.arange(-127, 128, device="cuda")
    bg[:, 0], bu[:, 0] = k.to(torch.int8), 1
    one, sa = torch.ones(n, device="cuda"), torch.ones(m, device="cuda")
    worst = 0.0
    for top in (80.0, 33.3, 7.1):
        sg = torch.full((n,), top / 127, device="cuda")
        h = torch.empty(m, n, device="cuda")
        mao.int8_glu(a, sa, bg, sg, bu, one, h)
        g = (k.float() * sg).double()
        ref = activation(g, "silu")[0]
        err = (h.double() - ref).abs()
        worst = max(worst, (err / (ref.abs() + 1e-300)).max().item() / U)
        assert (err <= 8 * U * ref.abs()).all(), f"off by {worst:.1f} U"
