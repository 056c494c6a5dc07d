"""The int8 quantiser where a scale lies next to the smallest normal number."""
import numpy as np
import pytest
import torch

from test_int8 import DT, check_quantized, scale32


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ties_under_the_smallest_scales(dtype):
    """Scales in [2^-126, 2^-125): their halves may have no fp32 number, the codes go by the exact quotient all the same."""
    rng = np.random.default_rng(7)
    rows = []
    for _ in range(700):
        top = np.float32(127.0 * 2.0 ** -126 * (1 + rng.random()))
        top = np.float32(torch.tensor(top).to(DT[dtype]).item())
        s = np.float64(scale32(top))
        base = ((rng.integers(-126, 127, 85) + 0.5) * s).astype(np.float32)
        row = np.concatenate([base, np.nextafter(base, np.float32(0)), np.nextafter(base, np.float32(np.inf)), [top]])
        rows.append(np.clip(row, -top, top))
    x = torch.from_numpy(np.array(rows, np.float32)).to(DT[dtype])
    scales = scale32(x.double().abs().amax(dim=1).numpy())
    assert (scales >= 2.0 ** -126).all() and (scales < 2.0 ** -125).mean() > 0.9
    check_quantized(x.cuda())
