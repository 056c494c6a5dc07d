"""int8 products over a contraction without terms."""
import pytest
import torch

import matrix_aware_optimizer_amd as mao
from test_int8 import DT


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n", [(1, 1), (5, 40), (50, 43), (300, 40), (2000, 3000)])
def test_no_terms_give_zeros_whatever_the_scales_hold(m, n, dtype):
    """A matrix without columns has no scales (the quantiser launches nothing for it)."""
    a, b = torch.empty(m, 0, dtype=torch.int8, device="cuda"), torch.empty(n, 0, dtype=torch.int8, device="cuda")
    sa, sb = torch.full((m,), float("nan"), device="cuda"), torch.full((n,), float("inf"), device="cuda")
    c = torch.full((m, n + 3), 3.0, dtype=DT[dtype], device="cuda")
    for call in (lambda: mao.int8_gemm(a, sa, b, sb, c[:, :n]), lambda: mao.int8_glu(a, sa, b, sb, b, sb, c[:, :n], act="gelu")):
        c.fill_(3.0)
        call()
        assert (c[:, :n] == 0).all() and (c[:, n:] == 3.0).all()


@pytest.mark.gpu
def test_a_block_without_inputs_answers_zeros():
    lin = mao.GatedLinear(*(torch.empty(40, 0, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    lin.quantize()
    assert (lin.answer(torch.empty(7, 0, dtype=torch.bfloat16, device="cuda")) == 0).all()
