"""Newton-Schulz on many small blocks (ns_blocks, ns_blocks_update) against the 64-bit oracle."""
import ctypes

import numpy as np
import pytest
import torch

import matrix_aware_optimizer_amd as mao
import oracle.muon_oracle as O
from matrix_aware_optimizer_amd import _abi
from workloads import CUBIC, QUINTIC

OK, EINVAL, EDTYPE, EALIGN, EWORKSPACE = 0, -1, -2, -3, -4
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# host side
# ---------------------------------------------------------------------------

def problem(**kw):
    good = dict(M=0x100000, out=0x200000, rows=64, cols=768, count=3, ld_m=768, stride_m=64 * 768, ld_out=768,
                stride_out=64 * 768, m_dtype=1, out_dtype=1)
    good.update(kw)
    return _abi.BlockProblem(*[good[f] for f, _ in _abi.BlockProblem._fields_])


def call(probs, steps=5, ws=0x300000, nbytes=None, update=False, n=None):
    L = mao.lib()
    arr = (_abi.BlockProblem * max(len(probs), 1))(*probs)
    ptr = ctypes.cast(arr, ctypes.c_void_p)
    n = len(probs) if n is None else n
    if nbytes is None:
        nbytes = L.ns_blocks_workspace_bytes(ptr, n)
    extra = (0.02, 0.1, 1.0) if update else ()
    f = L.ns_blocks_update if update else L.ns_blocks
    return f(ptr, n, *QUINTIC, steps, *extra, ws, nbytes, None)


@pytest.mark.parametrize("update", [False, True])
def test_refusals(update):
    def one(**kw):
        return call([problem(**kw)], update=update)

    assert one(rows=129, cols=129) == EINVAL                     # both sides over the limit
    assert one(rows=-1) == EINVAL and one(cols=-1) == EINVAL and one(count=-1) == EINVAL
    assert one(cols=(1 << 24) + 1, ld_m=1 << 25, ld_out=1 << 25) == EINVAL
    assert one(count=(1 << 20) + 1) == EINVAL
    assert one(count=1 << 20, cols=1 << 24, ld_m=1 << 24, ld_out=1 << 24) == EINVAL   # too many units
    assert one(M=None) == EINVAL and one(out=None) == EINVAL
    assert one(ld_m=767) == EINVAL and one(ld_out=767) == EINVAL
    assert one(stride_m=0) == EINVAL and one(stride_out=-8) == EINVAL
    assert one(m_dtype=2) == EDTYPE and one(out_dtype=-1) == EDTYPE
    assert one(M=0x100008) == EALIGN and one(out=0x200004) == EALIGN
    good = [problem()]
    assert call(good, steps=-1, update=update) == EINVAL
    assert call(good, n=-1, nbytes=0, update=update) == EINVAL
    need = mao.lib().ns_blocks_workspace_bytes(ctypes.cast((_abi.BlockProblem * 1)(*good), ctypes.c_void_p), 1)
    assert need > 0
    assert call(good, nbytes=need - 1, update=update) == EWORKSPACE
    assert call(good, ws=None, update=update) == EWORKSPACE
    assert call(good, ws=0x300008, update=update) == EALIGN
    # nothing to do: nothing is launched, nothing is asked for
    assert call([], update=update) == OK
    assert call([problem(count=0)], ws=None, update=update) == OK
    assert call([problem(rows=0, M=None, out=None)], ws=None, update=update) == OK
    # one bad problem refuses the whole call
    assert call([problem(), problem(M=None)], update=update) == EINVAL
    assert mao.lib().ns_blocks_workspace_bytes(None, 1) == 0


def test_python_refusals():
    x = torch.zeros(2, 4, 8)
    with pytest.raises(ValueError):
        mao.ns_blocks([(x, x)], *QUINTIC, 5)                     # host tensors
    with pytest.raises(ValueError):
        mao.ns_blocks([(x, x[:1])], *QUINTIC, 5)                 # different shapes
    mao.ns_blocks([], *QUINTIC, 5)
    with pytest.raises(ValueError):
        mao.PreparedNSBlocks([], *QUINTIC, 5)


# ---------------------------------------------------------------------------
# GPU
# ---------------------------------------------------------------------------

def noise(s, l, steps):
    """Relative size of the fp32 rounding in U for a block whose singular values are of one size: sums of l and of
    s terms round like random walks (the Gram, and 17 products of s x s matrices in five steps); eight times that."""
    return 8 * 2.0 ** -24 * (np.sqrt(l) + (4 * steps + 1) * np.sqrt(s))


def check(M, out, got, coeffs=QUINTIC, steps=5, update=None, tol=None):
    """got against U (or the update of `out`) of every block; M, out: 3-D host tensors."""
    eps = torch.finfo(got.dtype).eps / 2
    for i in range(M.shape[0]):
        x = M[i].double().numpy()
        U = O.newton_schulz(x, *coeffs, steps)
        g = got[i].double().cpu().numpy()
        assert np.isfinite(g).all()
        t = noise(min(x.shape), max(x.shape), steps) if tol is None else tol
        if update is None:
            ref, room = U, (eps + t) * np.linalg.norm(U)
        else:
            eta, decay, scale = (float(np.float32(v)) for v in update)
            ref = (1 - eta * decay) * out[i].double().numpy() - eta * scale * U
            # the two factors are rounded to fp32, the sum once more, then to the stored type
            room = (eps + 2 * 2.0 ** -24) * (np.linalg.norm(ref) + eta * scale * np.linalg.norm(U)) + eta * scale * t * np.linalg.norm(U)
        err = np.linalg.norm(g - ref)
        assert err <= room + 1e-30, (i, err, room)


def blocks(count, rows, cols, dtype, seed, layout="rows", pad=0):
    """[count, rows, cols] view into a larger tensor filled with NaN elsewhere, and its values on the host."""
    rng = np.random.default_rng([seed, count, rows, cols])
    x = torch.from_numpy((0.02 * rng.standard_normal((count, rows, cols))).astype(np.float32)).to(DT[dtype])
    if layout == "rows":            # blocks under one another, pad columns at the end
        full = torch.full((count * rows, cols + pad), float("nan"), dtype=DT[dtype], device="cuda")
        view = full[:, :cols].unflatten(0, (count, rows))
    else:                           # blocks side by side
        full = torch.full((rows, count * cols + pad), float("nan"), dtype=DT[dtype], device="cuda")
        view = full[:, :count * cols].view(rows, count, cols) if pad == 0 else full[:, :count * cols].unflatten(1, (count, cols))
        view = view.permute(1, 0, 2)
    view.copy_(x)
    return full, view, x


SHAPES = [(1, 1, 1), (2, 1, 7), (1, 7, 1), (3, 5, 5), (2, 16, 64), (1, 31, 100), (2, 32, 32), (2, 33, 257), (4, 64, 768),
          (2, 64, 65), (1, 80, 1000), (3, 96, 300), (2, 97, 2000), (1, 127, 129), (2, 128, 512), (1, 128, 5000), (1, 40, 9001)]


@pytest.mark.gpu
@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("m_dtype,out_dtype", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("count,s,l", SHAPES)
def test_directions(count, s, l, m_dtype, out_dtype, tall):
    rows, cols = (l, s) if tall else (s, l)
    _, Mv, M = blocks(count, rows, cols, m_dtype, 1, "cols" if tall else "rows")
    full, U, _ = blocks(count, rows, cols, out_dtype, 2, "rows")
    full.fill_(float("nan"))
    mao.ns_blocks([(Mv, U)], *QUINTIC, 5)
    torch.cuda.synchronize()
    tol = None
    if max(s, l) < 4 * min(s, l):   # nearly square: small singular values, see test_hard_spectra
        tol = 2.0 ** -24 * np.sqrt(s) * QUINTIC[0] ** 8 * abs(QUINTIC[1]) / QUINTIC[0]
    check(M, None, U, tol=tol)


@pytest.mark.gpu
@pytest.mark.parametrize("w_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout,pad", [("rows", 0), ("rows", 3), ("rows", 8), ("cols", 0), ("cols", 5), ("cols", 24)])
def test_update_and_strides(layout, pad, m_dtype, w_dtype):
    count, s, l = 3, 40, 333
    rows, cols = (l, s) if layout == "cols" else (s, l)
    _, Mv, M = blocks(count, rows, cols, m_dtype, 3, layout, pad)
    full, Wv, W = blocks(count, rows, cols, w_dtype, 4, layout, pad)
    up = (0.02, 0.1, 4.0)
    mao.ns_blocks_update([(Mv, Wv)], *QUINTIC, 5, eta=up[0], decay=up[1], scale=up[2])
    torch.cuda.synchronize()
    check(M, W, Wv, update=up)
    if pad:
        assert torch.isnan(full[:, -pad:]).all()                # nothing is written between the rows


@pytest.mark.gpu
@pytest.mark.parametrize("coeffs,steps", [(QUINTIC, 0), (QUINTIC, 1), (QUINTIC, 2), (CUBIC, 1), (CUBIC, 6), (QUINTIC, 7)])
def test_coefficients_and_steps(coeffs, steps):
    for rows, cols in ((64, 500), (500, 72)):
        _, Mv, M = blocks(2, rows, cols, "f32", 5)
        U = torch.empty((2, rows, cols), device="cuda")
        mao.ns_blocks([(Mv, U)], *coeffs, steps)
        check(M, None, U, coeffs, steps)


@pytest.mark.gpu
def test_many_problems_of_all_kinds_in_one_call():
    """More problems than one launch holds, of every orientation and type, each as in a call of its own."""
    probs, alone, kept = [], [], []
    for k in range(60):
        s, l = [(16, 200), (64, 256), (128, 600), (100, 400)][k % 4]
        rows, cols = (l, s) if k % 3 == 0 else (s, l)
        md, od = ["bf16", "f32"][k % 2], ["bf16", "f32"][(k // 2) % 2]
        _, Mv, M = blocks(1 + k % 3, rows, cols, md, 10 + k)
        U = torch.full(Mv.shape, float("nan"), dtype=DT[od], device="cuda")
        probs.append((Mv, U))
        kept.append(M)
    mao.ns_blocks(probs, *QUINTIC, 5)
    torch.cuda.synchronize()
    for (Mv, U), M in zip(probs, kept):
        check(M, None, U)


@pytest.mark.gpu
@pytest.mark.parametrize("m_dtype", ["bf16", "f32"])
def test_zero_and_special_blocks(m_dtype):
    """A block of zeros gives zeros (an update only decays); NaN and infinity stay in their block; tiny and large scales."""
    _, Mv, M = blocks(6, 48, 200, m_dtype, 6)
    Mv[1] = 0
    Mv[2, 3, 4] = float("nan")
    Mv[3, 0, 0] = float("inf")
    Mv[4] *= 2.0 ** -30
    Mv[5] *= 2.0 ** 40
    U = torch.empty((6, 48, 200), device="cuda")
    mao.ns_blocks([(Mv, U)], *QUINTIC, 5)
    assert (U[1] == 0).all() and torch.isnan(U[2]).all() and torch.isnan(U[3]).all()
    host = Mv.cpu()
    keep = [0, 4, 5]
    check(host[keep], None, U[keep])
    W = torch.full((6, 48, 200), 2.0, device="cuda")
    mao.ns_blocks_update([(Mv, W)], *QUINTIC, 5, eta=0.5, decay=0.5, scale=1.0)
    assert (W[1] == 1.5).all()


@pytest.mark.gpu
@pytest.mark.parametrize("m_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["decades", "rank", "repeated"])
def test_hard_spectra(kind, m_dtype):
    """Singular values over three decades, half the rank missing, equal rows.  Rounding of A0 (2^-24 sqrt(s) of its
    largest eigenvalue) grows by at most a^2 in each of the four iterations before T's last factor a + b A + ..."""
    rng = np.random.default_rng(7)
    s, l = 96, 700
    q1, _ = np.linalg.qr(rng.standard_normal((s, s)))
    q2, _ = np.linalg.qr(rng.standard_normal((l, s)))
    sig = np.logspace(0, -3, s) if kind == "decades" else np.r_[np.ones(s // 2), np.zeros(s // 2)]
    x = (q1 * sig) @ q2.T
    if kind == "repeated":
        x = rng.standard_normal((s, l))
        x[s // 2:] = x[:s // 2]
    M = torch.from_numpy(x.astype(np.float32)).to(DT[m_dtype])[None]
    for view in (M.cuda(), M.cuda().transpose(1, 2).contiguous()):
        U = torch.empty(view.shape, device="cuda")
        mao.ns_blocks([(view, U)], *QUINTIC, 5)
        check(view.cpu(), None, U, tol=2.0 ** -24 * np.sqrt(s) * QUINTIC[0] ** 8 * abs(QUINTIC[1]) / QUINTIC[0])


@pytest.mark.gpu
def test_repeats_bit_for_bit_and_in_a_graph():
    _, Mv, M = blocks(5, 64, 900, "bf16", 8)
    U = torch.empty((5, 64, 900), device="cuda")
    plan = mao.PreparedNSBlocks([(Mv, U)], *QUINTIC, 5)
    plan()
    first = U.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        U.zero_()
        plan()
    side.synchronize()
    assert torch.equal(U, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan()
    for k in range(3):
        Mv.copy_(M * (1 + k))                  # a power of two or three: the direction is the same up to rounding
        U.zero_()
        plan.workspace.fill_(0xFF)             # what the workspace held does not matter
        g.replay()
        torch.cuda.synchronize()
        eager = torch.empty_like(U)
        mao.ns_blocks([(Mv, eager)], *QUINTIC, 5)
        assert torch.equal(U, eager)
        if k == 0:
            assert torch.equal(U, first)


@pytest.mark.gpu
def test_agrees_with_ns_orthogonalize():
    """Where both apply (a whole matrix with a short side of 128), the two calls compute the same direction; the
    padded one rounds X to bf16 after every product (2e-2 is its own bound)."""
    _, Mv, M = blocks(1, 128, 1024, "bf16", 9)
    U, V = torch.empty((1, 128, 1024), device="cuda"), torch.empty((128, 1024), device="cuda")
    mao.ns_blocks([(Mv, U)], *QUINTIC, 5)
    mao.ns_orthogonalize([(Mv[0].contiguous(), V, None)], *QUINTIC, 5)
    assert torch.linalg.vector_norm(U[0] - V) <= 2e-2 * torch.linalg.vector_norm(U)


@pytest.mark.gpu
@pytest.mark.parametrize("tall", [False, True])
def test_offsets_past_32_bits(tall):
    """Blocks more than 2^31 entries apart, and rows whose pitch takes them there."""
    rows, cols = (300, 64) if tall else (64, 300)
    far = torch.empty(2 ** 31 + 2 ** 20, dtype=torch.bfloat16, device="cuda")
    small = torch.empty(2, rows, cols, device="cuda")
    views = [far.as_strided((2, rows, cols), (2 ** 31 + 8, cols, 1)),
             far.as_strided((1, rows, cols), (1, (2 ** 31 + 2 ** 20 - cols) // (rows - 1), 1))]
    for k, view in enumerate(views):
        M = (0.02 * torch.randn(view.shape, generator=torch.Generator().manual_seed(k))).to(torch.bfloat16)
        view.copy_(M)
        mao.ns_blocks([(view, small[:view.shape[0]])], *QUINTIC, 5)
        check(M, None, small[:view.shape[0]])
        view.copy_(M)
        W = view.clone()
        mao.ns_blocks_update([(M.cuda(), view)], *QUINTIC, 5, eta=0.1, decay=0.5, scale=2.0)
        check(M, W.cpu(), view, update=(0.1, 0.5, 2.0))
