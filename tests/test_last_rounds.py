"""The last round of large tiles, whole, in halves and in quarters, for every operand layout and output.

The sizes are chosen by their tiles; a CPU test asks the library's own rule that they are cut as their lists say."""
import pytest

import tile_plans
from test_gated import ACTS, check_backward, check_forward, check_weights
from test_int8 import check_gemm, check_glu

# (sizes, tiles, parts of the last round's tiles); fewer tiles than 256: the only round
INT8 = [((1999, 4096, 704), 128, 2), ((2500, 9216, 128), 360, 2), ((2049, 8192, 192), 288, 4), ((1100, 8192, 512), 160, 1), ((4096, 4096, 64), 256, 1)]
GLU = [((1999, 2048, 320), 128, 2), ((2500, 4608, 128), 360, 2), ((1100, 8192, 512), 320, 4), ((2049, 2048, 64), 144, 1)]
# outputs of these pass the caches or not, the cut is the same; 4603 and 1990 columns end inside a tile and a lane's run
FORWARD = [((1999, 2048, 200), 128, 2), ((2500, 4603, 72), 360, 2), ((1100, 8192, 72), 320, 4), ((2049, 4094, 40), 288, 4), ((1999, 1990, 104), 128, 2)]
BACKWARD = [((2040, 296, 4096), 128, 2), ((2500, 104, 9216), 360, 2), ((2049, 200, 8192), 288, 4), ((4100, 72, 4096), 272, 4)]
WEIGHTS = [((200, 2000, 2048), 128, 2), ((40, 2504, 4608), 360, 2), ((264, 2056, 4096), 288, 4), ((96, 4104, 4096), 544, 4)]


@pytest.mark.parametrize("cases,ask", [(INT8, tile_plans.int8), (GLU, lambda m, n, K: tile_plans.int8(m, n, K, 2)), (FORWARD, tile_plans.forward),
                                       (BACKWARD, tile_plans.backward), (WEIGHTS, tile_plans.weights)])
def test_sizes_are_cut_as_listed(cases, ask):
    for size, tiles, parts in cases:
        assert ask(*size) == ("large", 1, tiles, parts), size
    assert {parts for _, _, parts in cases} >= {2, 4}


def sizes(cases):
    return [size for size, _, _ in cases]


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,K", sizes(INT8))
def test_int8(m, n, K, out):
    check_gemm(m, n, K, out, seed=31, more=0)


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,K", sizes(GLU))
def test_int8_gated(m, n, K, out):
    check_glu(m, n, K, "gelu_tanh" if out == "bf16" else "silu", out, seed=33, more=0)


@pytest.mark.gpu
@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("t,f,d", sizes(FORWARD))
def test_forward(t, f, d, saved):
    check_forward(t, f, d, ACTS[f % 4], saved=saved, seed=35)


@pytest.mark.gpu
@pytest.mark.parametrize("t,f,d", sizes(BACKWARD))
def test_backward(t, f, d):
    check_backward(t, f, d, seed=37)


@pytest.mark.gpu
@pytest.mark.parametrize("out,beta", [("f32", 0.95), ("f32", 0.0), ("bf16", 0.95), ("bf16", 0.0)])
@pytest.mark.parametrize("t,f,d", sizes(WEIGHTS))
def test_weight_grad(t, f, d, out, beta):
    check_weights(t, f, d, out, beta, seed=39)
