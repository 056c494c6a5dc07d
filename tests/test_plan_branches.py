"""Ways of cutting a product that follow from its tiles, for every operand layout, sizes held to the library's own plan."""
import pytest

import tile_plans
from test_gated import ACTS, check_backward, check_forward, check_weights
from test_int8 import check_gemm, check_glu

# (sizes, kind of tiles, parts of the contraction)
INT8 = [((1000, 1280, 4096), "small", 3), ((520, 2200, 2600), "small", 2), ((1100, 960, 7000), "small", 3)]
GLU = [((1000, 640, 4096), "small", 3), ((520, 1100, 2600), "small", 2)]
FORWARD = [((1000, 640, 2048), "small", 3), ((520, 1100, 1304), "small", 2)]
# rows that do not start at 16 bytes
FORWARD_ODD = [((100, 200, 2047), "narrow", 3), ((1500, 768, 2047), "small", 3), ((1500, 768, 299), "small", 1), ((1500, 768, 1301), "small", 2)]
BACKWARD = [((1500, 304, 1536), "small", 1), ((1300, 2056, 1544), "small", 1)]
BACKWARD_ODD = [((100, 1001, 200), "narrow", 3), ((1500, 1001, 1536), "small", 3), ((1500, 301, 1535), "small", 1)]
WEIGHTS = [((1500, 1000, 640), "small", 2), ((3000, 520, 520), "small", 4)]
WEIGHTS_ODD = [((1500, 1001, 640), "small", 2), ((3001, 519, 523), "small", 4), ((100, 1300, 1301), "small", 1)]


@pytest.mark.parametrize("cases,ask,whole", [
    (INT8, tile_plans.int8, None), (GLU, lambda m, n, K: tile_plans.int8(m, n, K, 2), None), (FORWARD, tile_plans.forward, True),
    (FORWARD_ODD, tile_plans.forward, False), (BACKWARD, tile_plans.backward, True), (BACKWARD_ODD, tile_plans.backward, False),
    (WEIGHTS, tile_plans.weights, True), (WEIGHTS_ODD, tile_plans.weights, False)])
def test_sizes_are_cut_as_listed(cases, ask, whole):
    got = [(size, *ask(*size, **({} if whole is None else dict(whole=whole)))[:2]) for size, _, _ in cases]
    assert got == cases


def test_no_split_of_small_tiles_where_narrow_ones_serve():
    """dx on whole rows: at 128 x 128 tiles for no more than half the CUs, twice as many narrow ones are at most the CUs."""
    for t in range(1, 5000, 37):
        for d in range(8, 5000, 88):
            kind, parts, _, _ = tile_plans.backward(t, 65536, d)
            assert kind != "small" or parts == 1


def sizes(cases):
    return [size for size, _, _ in cases]


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,K", sizes(INT8))
def test_int8(m, n, K, out):
    check_gemm(m, n, K, out, seed=41)


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,K", sizes(GLU))
def test_int8_gated(m, n, K, out):
    check_glu(m, n, K, "gelu", out, seed=43)


@pytest.mark.gpu
@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("t,f,d", sizes(FORWARD + FORWARD_ODD))
def test_forward(t, f, d, saved):
    check_forward(t, f, d, ACTS[d % 4], saved=saved, seed=45)


@pytest.mark.gpu
@pytest.mark.parametrize("t,f,d", sizes(BACKWARD + BACKWARD_ODD))
def test_backward(t, f, d):
    check_backward(t, f, d, ACTS[t % 4], seed=47)


@pytest.mark.gpu
@pytest.mark.parametrize("out,beta", [("f32", 0.95), ("bf16", 0.0)])
@pytest.mark.parametrize("t,f,d", sizes(WEIGHTS + WEIGHTS_ODD))
def test_weight_grad(t, f, d, out, beta):
    check_weights(t, f, d, out, beta, seed=49)


@pytest.mark.gpu
@pytest.mark.parametrize("side", [1, 2, 5, 7])
def test_sides_under_eight(side):
    check_forward(90, 70, side, "gelu", seed=51)
    check_backward(90, side, 70, seed=52)
    check_backward(90, 70, side, seed=53)
    for t, f, d in ((90, side, 70), (90, 70, side), (side, 90, 70), (90, side, side)):
        check_weights(t, f, d, "f32", 0.95, seed=54)
        check_weights(t, f, d, "bf16", 0.0, seed=55)
