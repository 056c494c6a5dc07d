"""fp8 matrices with a scale for each block of 128: quantiser and product against the 64-bit reference."""
import ctypes

import numpy as np
import pytest
import torch

import matrix_aware_optimizer_amd as mao
import oracle.fp8_oracle as F

OK, EINVAL, EDTYPE, EALIGN, EWORKSPACE = 0, -1, -2, -3, -4
P = [ctypes.c_void_p(0x100000 * (i + 1)) for i in range(6)]
BAD = ctypes.c_void_p(0x100008)
TORCH = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


# ---------------------------------------------------------------------------
# host side
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_oracle_codes_match_the_formats(fmt):
    codes = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(codes.copy()).view(TORCH[fmt]).double().numpy()
    np.testing.assert_array_equal(F.decode(codes, fmt), ref)
    rng = np.random.default_rng(5)
    x = np.concatenate([rng.standard_normal(4000) * s for s in (1e-3, 1.0, 50.0)])
    x = np.clip(x, -F.TOP[fmt], F.TOP[fmt]).astype(np.float32)
    np.testing.assert_array_equal(F.round_to(x, fmt), torch.from_numpy(x).to(TORCH[fmt]).double().numpy())


def test_scale_bytes():
    L = mao.lib()
    assert L.fp8_scale_bytes(1, 1) == 16
    assert L.fp8_scale_bytes(4, 512) == 16
    assert L.fp8_scale_bytes(5, 513) == 2 * 8 * 4
    assert L.fp8_scale_bytes(0, 100) == 0 and L.fp8_scale_bytes(100, 0) == 0
    assert L.fp8_scale_bytes(-1, 5) == 0 and L.fp8_scale_bytes(mao.MUON_FP8_MAX_SIDE + 1, 5) == 0
    for r, c in [(1, 1), (5, 513), (777, 2304)]:
        assert int(np.prod(mao.fp8_scale_shape(r, c))) == L.fp8_scale_bytes(r, c)


def test_quantize_refusals():
    f = mao.lib().fp8_quantize
    x, q, s, qt, st = P[:5]
    good = dict(x=x, dt=1, rows=8, cols=200, ldx=200, fmt=0, br=1, q=q, ldq=256, s=s, qt=qt, ldqt=128, st=st)

    def call(**kw):
        a = {**good, **kw}
        return f(a["x"], a["dt"], a["rows"], a["cols"], a["ldx"], a["fmt"], a["br"], a["q"], a["ldq"], a["s"],
                 a["qt"], a["ldqt"], a["st"], None)

    assert call(rows=-1) == EINVAL and call(cols=-1) == EINVAL
    assert call(rows=mao.MUON_FP8_MAX_SIDE + 1) == EINVAL
    assert call(br=2) == EINVAL and call(ldx=199) == EINVAL and call(x=None) == EINVAL
    assert call(ldq=255) == EINVAL and call(ldq=200) == EINVAL and call(ldqt=64) == EINVAL and call(ldqt=136) == EINVAL
    assert call(q=None) == EINVAL and call(st=None) == EINVAL
    assert call(q=None, s=None, qt=None, st=None) == EINVAL
    assert call(dt=4) == EDTYPE and call(fmt=2) == EDTYPE
    assert call(x=BAD) == EALIGN and call(q=BAD) == EALIGN and call(st=BAD) == EALIGN
    assert call(rows=0) == OK and call(cols=0) == OK      # nothing is launched


def test_gemm_refusals():
    f = mao.lib().fp8_gemm
    A, sa, B, sb, C, W = P
    good = dict(A=A, fa=0, lda=256, sa=sa, B=B, fb=0, ldb=256, sb=sb, C=C, dt=1, ldc=40, m=8, n=40, K=256)

    def call(**kw):
        a = {**good, **kw}
        return f(a["A"], a["fa"], a["lda"], a["sa"], a["B"], a["fb"], a["ldb"], a["sb"], a["C"], a["dt"], a["ldc"],
                 a["m"], a["n"], a["K"], 1.0, 0.0, None, 0, None)

    assert call(m=-1) == EINVAL and call(n=-1) == EINVAL and call(K=-128) == EINVAL
    assert call(K=200) == EINVAL and call(K=384) == EINVAL          # not whole groups; longer than the pitch
    assert call(n=mao.MUON_FP8_MAX_SIDE + 1) == EINVAL
    assert call(lda=264) == EINVAL and call(ldb=128) == EINVAL and call(ldc=39) == EINVAL
    assert call(A=None) == EINVAL and call(sb=None) == EINVAL and call(C=None) == EINVAL
    assert call(fa=2) == EDTYPE and call(fb=1) == EDTYPE and call(dt=2) == EDTYPE
    assert call(A=BAD) == EALIGN and call(sa=BAD) == EALIGN and call(C=BAD) == EALIGN
    assert call(m=0) == OK and call(n=0) == OK                      # nothing is launched


def test_gemm_workspace_refusals():
    """Where a product asks for a workspace, a missing, short or misaligned one is refused."""
    L = mao.lib()
    for m, n, K in [(1, 4096, 4096), (100, 1024, 14336), (300, 512, 65536), (4096, 4096, 4096)]:
        need = L.fp8_gemm_workspace_bytes(m, n, K)
        if need == 0:
            continue
        args = (P[0], 0, K, P[1], P[2], 0, K, P[3], P[4], 1, n, m, n, K, 1.0, 0.0)
        assert L.fp8_gemm(*args, None, 0, None) == EWORKSPACE
        assert L.fp8_gemm(*args, P[5], need - 1, None) == EWORKSPACE
        assert L.fp8_gemm(*args, BAD, need, None) == EALIGN
    assert L.fp8_gemm_workspace_bytes(-1, 5, 128) == 0


def test_python_refusals():
    """The binding checks devices, types and shapes before the library is called."""
    q, s = mao.fp8_buffers(4, 100, device="cpu")
    with pytest.raises(ValueError):
        mao.fp8_quantize(torch.zeros(4, 100), q, s)                  # host tensors
    with pytest.raises(ValueError):
        mao.fp8_quantize(torch.zeros(4, 100), None, None)
    with pytest.raises(ValueError):
        mao.fp8_quantize(torch.zeros(4, 100), q, None)
    with pytest.raises(ValueError):
        mao.fp8_gemm(q, s, q, s, torch.zeros(4, 5))


# ---------------------------------------------------------------------------
# GPU
# ---------------------------------------------------------------------------

def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)


def spread(rows, cols, seed, dtype):
    rng = np.random.default_rng([seed, rows, cols])
    x = rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-6, 7, (rows, 1)) * (1 + 9 * (rng.random((1, cols)) < 0.02))
    t = torch.from_numpy(x.astype(np.float32))
    return t if dtype == "f32" else t.to(torch.bfloat16)


def run_quantize(x, fmt, block_rows, rows_out=True, cols_out=True, q_pad=0):
    rows, cols = x.shape
    bufs = []
    for r, c, want in ((rows, cols, rows_out), (cols, rows, cols_out)):
        if not want:
            bufs += [None, None]
            continue
        q, s = mao.fp8_buffers(r, c, fmt)
        if q_pad:
            q = torch.empty((r, q.shape[1] + q_pad), dtype=torch.uint8, device="cuda").view(q.dtype)
        q.view(torch.uint8).fill_(0x55)      # what was there before must not show
        s.fill_(0x33)
        bufs += [q, s]
    mao.fp8_quantize(x, *bufs, block_rows=block_rows)
    torch.cuda.synchronize()
    return bufs


def check_quantized(x64, fmt, block_rows, q, s):
    rows, cols = x64.shape
    ref, ex = F.quantize(x64, fmt, block_rows)
    codes = q.view(torch.uint8).cpu().numpy()
    np.testing.assert_array_equal(F.decode(codes[:, :ref.shape[1]], fmt), ref)
    np.testing.assert_array_equal(s.cpu().numpy(), F.pack_scales(ex))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 130), (128, 128), (129, 257), (200, 640), (5, 2000), (515, 64)])
def test_quantize(rows, cols, block_rows, fmt, dtype):
    x = spread(rows, cols, 1, dtype)
    q, s, qt, st = run_quantize(x.cuda(), fmt, block_rows)
    check_quantized(x.double().numpy(), fmt, block_rows, q, s)
    check_quantized(x.double().numpy().T, fmt, block_rows, qt, st)


@pytest.mark.gpu
def test_quantize_one_side_and_strides():
    x = spread(150, 300, 2, "bf16")
    wide = torch.full((150, 333), float("nan"), dtype=torch.bfloat16)     # odd pitch, NaN between the rows
    wide[:, :300] = x
    view = wide.cuda()[:, :300]
    for rows_out, cols_out in ((True, False), (False, True)):
        q, s, qt, st = run_quantize(view, "e4m3", 1, rows_out, cols_out, q_pad=32)
        if rows_out:
            check_quantized(x.double().numpy(), "e4m3", 1, q, s)
            assert (q.view(torch.uint8)[:, 384:] == 0x55).all()           # past the padded columns nothing is written
        else:
            check_quantized(x.double().numpy().T, "e4m3", 1, qt, st)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize_borders(fmt):
    """Every tie and every end of the code grid, group maxima at and next to MAX 2^e, the ends of the exponents."""
    top = F.TOP[fmt]
    grid = F.decode(np.arange(128, dtype=np.uint8), fmt)
    grid = np.sort(grid[np.isfinite(grid)])
    mid = (grid[1:] + grid[:-1]) / 2
    rows = []
    for base in (grid, mid, np.nextafter(mid.astype(np.float32), np.float32(0)), np.nextafter(mid.astype(np.float32), np.float32(1e9))):
        row = np.zeros(128)
        row[:base.size] = base
        row[127] = top                       # fixes the scale at 1
        rows.append(row)
    for amax in (top, np.nextafter(np.float32(top), np.float32(1e9)), np.nextafter(np.float32(top), np.float32(0)), 2.0 ** 127,
                 3.3e38, 2.0 ** -126, 2.0 ** -130, 2.0 ** -149, 1e-40, 0.0, 2.0 ** -118, 2.0 ** -111 * 1.75):
        rows.append(np.linspace(-1, 1, 128) * np.float64(amax))
    x = torch.from_numpy(np.array(rows).astype(np.float32))
    q, s, qt, st = run_quantize(x.cuda(), fmt, 1)
    check_quantized(x.double().numpy(), fmt, 1, q, s)
    check_quantized(x.double().numpy().T, fmt, 1, qt, st)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_not_finite(fmt, block_rows):
    x = spread(140, 260, 3, "f32")
    x[0, 0], x[1, 1], x[2, 2], x[139, 259] = float("nan"), float("inf"), float("-inf"), float("nan")
    x[5, :128] = float("inf")                # a group with nothing finite
    q, s, qt, st = run_quantize(x.cuda(), fmt, block_rows)
    check_quantized(x.double().numpy(), fmt, block_rows, q, s)
    check_quantized(x.double().numpy().T, fmt, block_rows, qt, st)


@pytest.mark.gpu
def test_quantize_every_bf16():
    """All finite bf16 patterns, each group of 128 neighbours under its own scale."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).reshape(512, 128)
    q, s, _, _ = run_quantize(bits.cuda(), "e4m3", 1, cols_out=False)
    check_quantized(bits.double().numpy(), "e4m3", 1, q, s)


def operand(rows, cols, fmt, seed, block_rows=1, scale_spread=8, small_ints=False):
    """Codes and scales straight from random bytes (every finite code), or small integers under scale 1."""
    rng = np.random.default_rng([seed, rows, cols])
    K = -(-cols // 128) * 128
    if small_ints:
        codes = torch.from_numpy(rng.integers(-3, 4, (rows, K)).astype(np.float32)).to(TORCH[fmt]).view(torch.uint8).numpy()
        ex = np.zeros((rows, K // 128), np.int64)
    else:
        codes = rng.integers(0, 256, (rows, K), dtype=np.uint8)
        codes = np.where(np.isfinite(F.decode(codes, fmt)), codes, 1).astype(np.uint8)
        ex = rng.integers(-scale_spread, scale_spread + 1, (-(-rows // block_rows), K // 128))
        ex = np.repeat(ex, block_rows, axis=0)[:rows]
    codes[:, cols:] = 0
    s = F.pack_scales(ex)
    q = torch.from_numpy(codes).cuda().view(TORCH[fmt])
    return q, torch.from_numpy(s).cuda(), F.values(codes, s, fmt)


def check_gemm(m, n, K, fa="e4m3", out="f32", alpha=1.0, beta=0.0, seed=0, ldc_pad=0, block_rows=1):
    A, sa, a = operand(m, K, fa, seed + 1)
    B, sb, b = operand(n, K, "e4m3", seed + 2, block_rows)
    dt = torch.float32 if out == "f32" else torch.bfloat16
    rng = np.random.default_rng([seed, 3])
    full = torch.full((m, n + ldc_pad), float("nan"), dtype=dt, device="cuda")
    C = full[:, :n]
    c0 = torch.from_numpy((rng.standard_normal((m, n)) * 1e3).astype(np.float32)).to(dt)
    if beta:
        C.copy_(c0)                          # otherwise C starts as NaN and must not be read
    mao.fp8_gemm(A, sa, B, sb, C, alpha=alpha, beta=beta)
    torch.cuda.synchronize()
    al, be = float(np.float32(alpha)), float(np.float32(beta))
    ref = F.gemm(a, b, c0.double().numpy(), al, be)
    # every fp32 addition is off by at most a step (2^-23) of a partial sum, which is at most the sum of the
    # magnitudes; one more for each of alpha, beta and the last addition; then half a step of the stored type
    mag = abs(al) * (np.abs(a) @ np.abs(b).T) + (abs(be) * np.abs(c0.double().numpy()) if be else 0.0)
    tol = (a.shape[1] + 4) * 2.0 ** -23 * mag + torch.finfo(dt).eps / 2 * np.abs(ref) + 1e-30
    if out == "bf16":
        # the fp8 instructions drop, of each eight neighbouring products, what lies over 13 bits below the
        # largest: eight times 2^-13 of it at most (an fp32 C is computed without that)
        tol += abs(al) * 2.0 ** -10 * sum(np.max(np.abs(a[:, None, k:k + 8] * b[None, :, k:k + 8]), axis=2)
                                          for k in range(0, a.shape[1], 8))
    err = np.abs(C.double().cpu().numpy() - ref)
    assert np.isfinite(err).all() and (err <= tol).all(), float((err / tol).max())
    # and the errors of K additions do not all point one way: the norm stays far below that bound
    rel = np.linalg.norm(err) / max(np.linalg.norm(ref), 1e-300)
    assert rel <= max(torch.finfo(dt).eps, 8 * 2.0 ** -23 * np.sqrt(a.shape[1]))
    if ldc_pad:
        assert torch.isnan(full[:, n:]).all()


GEMM_SIZES = [(1, 1, 1), (1, 16, 128), (1, 2304, 768), (2, 33, 300), (7, 64, 4096), (16, 128, 512), (17, 100, 640), (31, 257, 1000),
              (48, 512, 2048), (64, 130, 129), (65, 64, 128), (100, 300, 1500), (128, 128, 128), (129, 255, 384),
              (255, 256, 512), (256, 256, 256), (257, 513, 640), (300, 1030, 777), (512, 768, 1024), (777, 500, 2304)]


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,K", GEMM_SIZES)
def test_gemm_f32(m, n, K):
    check_gemm(m, n, K)


@pytest.mark.gpu
@pytest.mark.parametrize("fa", ["e4m3", "e5m2"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,K", [(1, 130, 256), (3, 1000, 1024), (40, 75, 600), (130, 260, 512), (300, 513, 1280)])
def test_gemm_types_and_epilogue(m, n, K, out, fa):
    check_gemm(m, n, K, fa, out, alpha=0.05, beta=0.95, seed=10)
    check_gemm(m, n, K, fa, out, alpha=-1.5, beta=0.0, seed=11, ldc_pad=3)
    check_gemm(m, n, K, fa, out, alpha=0.5, beta=1.0, seed=12, ldc_pad=8, block_rows=128)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,K", [(1, 64, 128), (5, 77, 512), (33, 90, 2048), (200, 300, 1024), (600, 520, 384)])
def test_gemm_integers_are_exact(m, n, K):
    """Small integers under scale 1: every partial sum is exact in fp32, so any order gives the same value."""
    A, sa, a = operand(m, K, "e4m3", 21, small_ints=True)
    B, sb, b = operand(n, K, "e4m3", 22, small_ints=True)
    C = torch.empty((m, n), device="cuda")
    mao.fp8_gemm(A, sa, B, sb, C)
    np.testing.assert_array_equal(C.double().cpu().numpy(), a @ b.T)


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,K", [(2100, 4001, 640), (2048, 4096, 128), (5000, 2050, 256), (4097, 2047, 512)])
def test_gemm_large_tiles_are_exact(m, n, K, out):
    """Ragged products of many tiles: entries in -1, 0, 1 under scale 1, sums under 256 are exact in bf16 too."""
    rng = np.random.default_rng([m, n])
    a, b = (rng.integers(-1, 2, (r, K)).astype(np.float32) for r in (m, n))
    A, B = (torch.from_numpy(v).cuda().to(torch.float8_e4m3fn) for v in (a, b))
    sa, sb = (torch.full(mao.fp8_scale_shape(r, K), 127, dtype=torch.uint8, device="cuda") for r in (m, n))
    C = torch.full((m, n), float("nan"), dtype=torch.float32 if out == "f32" else torch.bfloat16, device="cuda")
    mao.fp8_gemm(A, sa, B, sb, C)
    ref = a @ b.T                      # sums of at most 640 ones: exact in fp32
    assert np.abs(ref).max() < 256
    np.testing.assert_array_equal(C.float().cpu().numpy(), ref)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 40, 200, 600])
def test_gemm_repeats_bit_for_bit(m):
    A, sa, _ = operand(m, 4096, "e4m3", 31)
    B, sb, _ = operand(520, 4096, "e4m3", 32)
    got = []
    for _ in range(3):
        C = torch.empty((m, 520), device="cuda")
        mao.fp8_gemm(A, sa, B, sb, C)
        got.append(C)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(1, 64), (40, 200), (300, 520)])
def test_gemm_special_values_stay_in_their_rows(m, n):
    """A NaN code reaches its row (or column) of C only; a NaN or infinite C is not read at beta 0."""
    A, sa, _ = operand(m, 640, "e4m3", 41)
    B, sb, _ = operand(n, 640, "e4m3", 42)
    C = torch.empty((m, n), device="cuda")
    mao.fp8_gemm(A, sa, B, sb, C)
    clean = C.clone()
    A.view(torch.uint8)[m - 1, 130] = 0x7F
    B.view(torch.uint8)[n // 2, 5] = 0xFF
    C.fill_(float("inf"))
    mao.fp8_gemm(A, sa, B, sb, C)
    nan = torch.isnan(C)
    assert nan[m - 1].all() and nan[:, n // 2].all()
    nan[m - 1] = True
    nan[:, n // 2] = True
    assert torch.equal(C[~nan], clean[~nan])


@pytest.mark.gpu
def test_gemm_empty_contraction_and_sides():
    A, B = torch.empty((5, 0), dtype=torch.float8_e4m3fn, device="cuda"), torch.empty((7, 0), dtype=torch.float8_e4m3fn, device="cuda")
    sa, sb = (torch.empty(mao.fp8_scale_shape(r, 0), dtype=torch.uint8, device="cuda") for r in (5, 7))
    C = torch.full((5, 7), 2.0, device="cuda")
    mao.fp8_gemm(A, sa, B, sb, C, beta=0.5)
    assert (C == 1.0).all()
    mao.fp8_gemm(A, sa, B, sb, C)
    assert (C == 0.0).all()
    q, s = mao.fp8_buffers(0, 256)
    qt, st = mao.fp8_buffers(256, 0)
    mao.fp8_quantize(torch.empty((0, 256), device="cuda"), q, s, qt, st)
    B, sb, _ = operand(7, 256, "e4m3", 51)
    mao.fp8_gemm(q, s, B, sb, torch.empty((0, 7), device="cuda"))
    torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 60, 300])
def test_gemm_on_another_stream_and_in_a_graph(m):
    """Work goes to the stream that is current; a captured call replays on new inputs."""
    A, sa, a = operand(m, 1024, "e4m3", 61, small_ints=True)
    B, sb, b = operand(300, 1024, "e4m3", 62, small_ints=True)
    C = torch.zeros((m, 300), device="cuda")
    ws = torch.empty(max(mao.fp8_gemm_workspace_bytes(m, 300, 1024), 16), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mao.fp8_gemm(A, sa, B, sb, C, workspace=ws)
    side.synchronize()
    np.testing.assert_array_equal(C.double().cpu().numpy(), a @ b.T)
    x = torch.zeros((m, 1024), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mao.fp8_quantize(x, A, sa)
        mao.fp8_gemm(A, sa, B, sb, C, workspace=ws)
    for k in range(3):
        x.copy_(torch.randint(-3, 4, x.shape, device="cuda").float())
        C.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(C.double().cpu().numpy(), x.double().cpu().numpy() @ b.T)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """More than 2^31 entries: the last rows of a long matrix, quantised both ways and multiplied, against the reference."""
    rows, cols = 131072 + 130, 16384
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    tail = spread(200, cols, 71, "bf16")
    x[-200:] = tail.cuda()
    q, s = mao.fp8_buffers(rows, cols)
    qt, st = mao.fp8_buffers(cols, rows)
    mao.fp8_quantize(x, q, s, qt, st)
    ref, ex = F.quantize(tail.double().numpy(), "e4m3")
    np.testing.assert_array_equal(F.decode(q[-200:].view(torch.uint8).cpu().numpy(), "e4m3"), ref)
    np.testing.assert_array_equal(s[:, rows - 200:rows].cpu().numpy(), F.pack_scales(ex)[:, :200])
    # a column group of the transpose starts at a multiple of 128 rows: take the rows of its last two groups
    first = (rows // 128 - 1) * 128
    part = x[first:].double().cpu().numpy()[:, :300].T
    ref, ex = F.quantize(part, "e4m3")
    np.testing.assert_array_equal(F.decode(qt[:300, first:first + ref.shape[1]].view(torch.uint8).cpu().numpy(), "e4m3"), ref)
    del x, qt, st
    w = ints_operand(48, cols)
    C = torch.empty((rows, 48), device="cuda")
    mao.fp8_gemm(q, s, w[0], w[1], C)
    a = F.values(q[-200:].view(torch.uint8).cpu().numpy(), F.pack_scales(F.quantize(tail.double().numpy(), "e4m3")[1]), "e4m3")
    want = a @ w[2].T
    mag = np.abs(a) @ np.abs(w[2]).T
    assert (np.abs(C[-200:].double().cpu().numpy() - want) <= (cols + 4) * 2.0 ** -23 * mag + 2.0 ** -24 * np.abs(want)).all()
    assert (C[:rows - 200] == 0).all()


def ints_operand(rows, cols):
    return operand(rows, cols, "e4m3", 72, small_ints=True)


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_output_offsets_past_32_bits(out):
    """A C of more than 2^31 entries: ones and minus ones, so every entry is exact."""
    m, n, K = 262144 + 70, 8200, 128
    rng = np.random.default_rng(73)
    a, b = (rng.integers(-1, 2, (r, K)).astype(np.float32) for r in (256, n))
    A = torch.zeros((m, K), device="cuda")
    A[-256:] = torch.from_numpy(a).cuda()
    A, B = A.to(torch.float8_e4m3fn), torch.from_numpy(b).cuda().to(torch.float8_e4m3fn)
    sa, sb = (torch.full(mao.fp8_scale_shape(r, K), 127, dtype=torch.uint8, device="cuda") for r in (m, n))
    C = torch.full((m, n), 5.0, dtype=torch.float32 if out == "f32" else torch.bfloat16, device="cuda")
    mao.fp8_gemm(A, sa, B, sb, C)
    np.testing.assert_array_equal(C[-256:].float().cpu().numpy(), a @ b.T)
    assert not C[:-256].any()


@pytest.mark.gpu
def test_temporary_workspace_belongs_to_the_stream_of_the_call():
    """A split product on a side stream with a workspace of its own, while the current stream allocates and fills."""
    m, n, K = 100, 512, 14336
    assert mao.fp8_gemm_workspace_bytes(m, n, K) > 0
    A, sa, a = operand(m, K, "e4m3", 81, small_ints=True)
    B, sb, b = operand(n, K, "e4m3", 82, small_ints=True)
    want = torch.from_numpy((a @ b.T).astype(np.float32)).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    words = mao.fp8_gemm_workspace_bytes(m, n, K) // 4
    for handle in (side, side.cuda_stream):
        outs = [torch.zeros((m, n), device="cuda") for _ in range(10)]
        side.wait_stream(torch.cuda.current_stream())
        for C in outs:
            mao.fp8_gemm(A, sa, B, sb, C, stream=handle)
            torch.full((words,), float("nan"), device="cuda")
        torch.cuda.synchronize()
        assert all(torch.equal(C, want) for C in outs)
