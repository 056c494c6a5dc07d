"""Head-wise Newton-Schulz of blocks whose singular values decay or vanish, over the range of step counts."""
import numpy as np
import pytest
import torch

import matrix_aware_optimizer_amd as mao
import oracle.muon_oracle as O
from workloads import CUBIC, QUINTIC

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
KINDS = ["rank1", "rank4", "half", "pairs", "tokens", "decades", "power"]


def growth(coeffs):
    """Largest factor by which a step scales a singular value: max of |a + b x + c x x| over x in [0, 1]."""
    a, b, c = coeffs
    x = np.linspace(0, 1, 1001)
    return max(1.0, float(np.abs(a + b * x + c * x * x).max()))


def spectrum(kind, s, l, dtype, seed=0):
    """An s x l momentum: rank 1, 4 or s / 2, equal pairs of rows, the gradient of 3 s / 4 tokens, singular values
    over three decades, and falling as a power."""
    rng = np.random.default_rng([seed, s, l])
    n = rng.standard_normal
    if kind in ("rank1", "rank4", "half", "tokens"):
        r = {"rank1": 1, "rank4": min(4, s), "half": max(1, s // 2), "tokens": max(1, 3 * s // 4)}[kind]
        x = n((s, r)) @ n((r, l))
    elif kind == "pairs":
        x = np.repeat(n((-(-s // 2), l)), 2, axis=0)[:s]
    else:
        sig = np.logspace(0, -3, s) if kind == "decades" else np.arange(1, s + 1) ** -1.5
        x = (np.linalg.qr(n((s, s)))[0] * sig) @ np.linalg.qr(n((l, s)))[0].T
    return torch.from_numpy((0.02 * x).astype(np.float32)).to(DT[dtype])


def directions(M, out_dtype, coeffs, steps):
    """(U of M and of its transpose, as fp64 arrays in M's orientation)."""
    got = []
    for x in (M, M.t().contiguous()):
        U = torch.full(x.shape, float("nan"), dtype=DT[out_dtype], device="cuda")
        mao.ns_blocks([(x.cuda(), U)], *coeffs, steps)
        got.append(U.double().cpu().numpy())
    return got[0], got[1].T


def relative_errors(M, out_dtype, coeffs, steps):
    co = [float(np.float32(v)) for v in coeffs]
    ref = O.newton_schulz(M.double().numpy(), *co, steps)
    return [np.linalg.norm(u - ref) / np.linalg.norm(ref) for u in directions(M, out_dtype, coeffs, steps)]


@pytest.mark.gpu
@pytest.mark.parametrize("m_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("s,l", [(64, 768), (128, 1024), (80, 500)])
def test_as_exact_as_fp32_iterations_on_the_block(s, l, kind, m_dtype):
    """An iteration on X in fp32 puts rounding of 2^-24 into the directions that X lacks, and every step scales it by
    at most the growth g: sqrt(s) 2^-24 g^steps of U.  A recursion on the Gram matrix in fp32 loses the square of that."""
    M = spectrum(kind, s, l, m_dtype)
    for coeffs, steps in ((QUINTIC, 5), (QUINTIC, 6), (QUINTIC, 8), (QUINTIC, 10), (CUBIC, 20), (CUBIC, 30)):
        tol = 2.0 ** -24 * (1 + np.sqrt(s) * growth(coeffs) ** steps)
        errs = relative_errors(M, "f32", coeffs, steps)
        assert max(errs) <= tol, (coeffs, steps, errs, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("m_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("exponent", [-99, -60, 60, 99])
def test_blocks_of_any_size(exponent, m_dtype):
    """The bound holds over the range that the header gives for |M|_F."""
    M = spectrum("power", 48, 300, m_dtype)
    M = M * 2.0 ** (exponent - np.floor(np.log2(float(M.float().norm()))))
    errs = relative_errors(M, "f32", QUINTIC, 5)
    assert max(errs) <= 2.0 ** -24 * (1 + np.sqrt(48) * growth(QUINTIC) ** 5), errs


def tolerance(s, out_dtype, coeffs, steps):
    """Half a step of the output's type and of fp32, and what comes before: the Gram matrix and the iterations in
    fp64, whose rounding grows by g^2 per step, and the product T M, in 24 bits while T is at most g^steps = 512."""
    g = growth(coeffs) ** steps
    before = np.sqrt(s) * (2.0 ** -53 * g * g + (2.0 ** -24 * g if g <= 512 else 0.0))
    return torch.finfo(DT[out_dtype]).eps / 2 + 2.0 ** -24 + before


@pytest.mark.gpu
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("s,l", [(64, 768), (128, 1024), (80, 500)])
def test_little_but_the_output_is_rounded(s, l, kind, m_dtype, out_dtype):
    M = spectrum(kind, s, l, m_dtype, 1)
    for coeffs, steps in ((QUINTIC, 1), (QUINTIC, 3), (QUINTIC, 5), (QUINTIC, 6), (QUINTIC, 8), (QUINTIC, 12), (CUBIC, 5),
                          (CUBIC, 15), (CUBIC, 16), (CUBIC, 30)):
        tol = tolerance(s, out_dtype, coeffs, steps)
        errs = relative_errors(M, out_dtype, coeffs, steps)
        assert max(errs) <= tol, (coeffs, steps, errs, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("w_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("steps", [5, 7])
@pytest.mark.parametrize("kind", ["rank1", "rank4", "power"])
def test_update_of_uneven_spectra(kind, steps, w_dtype):
    """The update takes the same U: its error stays that of the rounding of W."""
    s, l, eta, decay, scale = 64, 768, 0.5, 0.25, 4.0
    M = spectrum(kind, s, l, "f32", 2)
    W = torch.from_numpy(np.random.default_rng(3).standard_normal((s, l)).astype(np.float32) * 0.02).to(DT[w_dtype])
    got = W.cuda()
    mao.ns_blocks_update([(M.cuda(), got)], *QUINTIC, steps, eta=eta, decay=decay, scale=scale)
    U = O.newton_schulz(M.double().numpy(), *(float(np.float32(v)) for v in QUINTIC), steps)
    ref = (1 - eta * decay) * W.double().numpy() - eta * scale * U
    # W's half step; both products and their sum in fp32; U's own error without its rounding to a type
    tol = (torch.finfo(DT[w_dtype]).eps / 2 + 2.0 ** -23) * np.linalg.norm(ref) + eta * scale * np.linalg.norm(U) * (
        tolerance(s, "f32", QUINTIC, steps) + 2.0 ** -24)
    assert np.linalg.norm(got.double().cpu().numpy() - ref) <= tol


@pytest.mark.gpu
@pytest.mark.parametrize("steps", [5, 6])
@pytest.mark.parametrize("s", [1, 2, 15, 16, 17, 33, 48, 63, 65, 79, 81, 96, 97, 111, 112, 113, 127, 128])
def test_every_number_of_strips(s, steps):
    """Short sides at and next to multiples of 16, long sides that end inside a slab, several chunks of the Gram."""
    for l, m_dtype in ((s, "f32"), (s + 1, "bf16"), (3 * s + 131, "bf16"), (4 * s + 1100, "f32")):
        M = torch.from_numpy(np.random.default_rng([s, l]).standard_normal((s, l)).astype(np.float32)).to(DT[m_dtype])
        tol = tolerance(s, "f32", QUINTIC, steps)
        errs = relative_errors(M, "f32", QUINTIC, steps)
        assert max(errs) <= tol, (l, errs, tol)
