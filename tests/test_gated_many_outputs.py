"""Outputs of the gated block whose threads, one for each entry or run of eight, would pass what one launch may have (2^32)."""
import pytest
import torch

import matrix_aware_optimizer_amd as mao
from test_gated import BF, EINVAL, blank, forward_call, randn


def test_more_than_one_launch_covers_is_refused():
    """2^37 entries of h on tiles through registers: refused before anything is launched."""
    t = mao.MUON_GLU_MAX_SIDE
    assert forward_call(t=t, f=40000, d=9, ldx=9, ldw=9, ldh=40000, ldg=40000) == EINVAL


@pytest.mark.gpu
def test_narrow_contractions_of_many_outputs():
    """2^32 + 2^16 entries of h from rows of four."""
    t, f = 65537, 65536
    x, wg, wu = randn((t, 4), 1), randn((f, 4), 2), randn((f, 4), 3)
    h = torch.empty(t, f, dtype=BF, device="cuda")
    mao.glu_forward(x, wg, wu, h, act="gelu")
    for rows in (slice(0, 50), slice(4000, 4100), slice(t - 100, t)):      # around a full stride of the threads, and the last
        part = blank(rows.stop - rows.start, f)
        mao.glu_forward(x[rows].clone(), wg, wu, part, act="gelu")
        assert torch.equal(h[rows], part)


@pytest.mark.gpu
@pytest.mark.parametrize("f", [16384, 16381])
def test_gradients_of_many_entries(f):
    """dg, du and h of more than 2^31 entries, in place."""
    t = 131100
    g = torch.Generator(device="cuda").manual_seed(5)
    dh, gate, up = (torch.randn(t, f, generator=g, device="cuda", dtype=BF) for _ in range(3))
    places = (slice(0, 40), slice(131060, t))
    want = []
    for rows in places:
        a, b, c = (m[rows].clone() for m in (dh, gate, up))
        mao.glu_backward(a, b, c, b, c, h=a, act="silu")
        want.append((a, b, c))
    mao.glu_backward(dh, gate, up, gate, up, h=dh, act="silu")
    for rows, parts in zip(places, want):
        for got, part in zip((dh, gate, up), parts):
            assert torch.equal(got[rows], part)
