"""The int8 quantiser at every width that it tells apart, bad entries of wide rows, and outputs of more than 2^31 bytes."""
import numpy as np
import pytest
import torch

import matrix_aware_optimizer_amd as mao
from test_int8 import U, check_quantized, codes, exact_sum, quantize64, spread


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(5, 512), (3, 513), (2, 4096), (3, 4097), (2, 6000), (2, 8192), (2, 8193), (2, 16384), (2, 16385)])
def test_widths(rows, cols, dtype):
    check_quantized(spread(rows, cols, 5, dtype).cuda())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [700, 2049, 6000, 14336, 20001])
def test_not_finite_entries_of_wide_rows(cols, dtype):
    """One bad entry in the part of each wave, and at the row's end."""
    places = [p for p in (0, 8 * 64 + 3, 8 * 130 + 7, 8 * 200, 2047, cols - 1) if p < cols]
    x = spread(2 * len(places) + 1, cols, 6, dtype)
    bad = torch.zeros(x.shape[0], dtype=torch.bool)
    for i, p in enumerate(places):
        x[2 * i + 1, p] = (float("nan"), float("inf"), float("-inf"))[i % 3]
        bad[2 * i + 1] = True
    q, s = mao.int8_buffers(*x.shape)
    q.fill_(0x55)
    mao.int8_quantize(x.cuda(), q, s)
    assert torch.equal(torch.isnan(s).cpu(), bad) and (q[bad.cuda()] == 0).all()
    want, scales = quantize64(x[~bad].double().numpy())
    np.testing.assert_array_equal(q[~bad.cuda()][:, :cols].cpu().numpy(), want)
    np.testing.assert_array_equal(s[~bad.cuda()].cpu().numpy(), scales)


@pytest.mark.gpu
def test_outputs_of_more_than_32_bits():
    """C and H of more than 2^31 bytes: the last rows and columns."""
    m, n, K = 70001, 8192, 64
    (a, sa), (b, sb), (bu, su) = codes(m, K, 1), codes(n, K, 2), codes(n, K, 3)
    size = 2.0 ** -9
    c = torch.empty(m, n, device="cuda")
    tail = slice(m - 300, m)
    mao.int8_gemm(a, sa, b, sb, c)
    ref = exact_sum(a[tail], b) * sa[tail].double()[:, None] * sb.double()
    assert ((c[tail].double() - ref).abs() <= ref.abs() * 3.01 * U).all()
    small = torch.empty(300, n, device="cuda")
    mao.int8_gemm(a[tail].clone(), sa[tail].clone(), b, sb, small)
    assert torch.equal(c[tail], small)
    mao.int8_glu(a, sa, b, sb * size, bu, su * size, c, act="gelu_tanh")
    mao.int8_glu(a[tail].clone(), sa[tail].clone(), b, sb * size, bu, su * size, small, act="gelu_tanh")
    assert torch.equal(c[tail], small)      # the sums are exact, so every cut gives the same bits
