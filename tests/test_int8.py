"""8-bit integer matrices with a scale for each row: quantiser, product and gated product against 64-bit values.

Tolerances.  A sum of codes is exact.  int8_gemm rounds it to fp32, multiplies the two
scales, multiplies both and rounds to C: (1 + 2^-24)^3 and, for bf16, 1 + 2^-8.  The gated
product's activation is fp32; its error is counted in `activation_error`.
"""
import ctypes

import numpy as np
import pytest
import torch

import matrix_aware_optimizer_amd as mao

OK, EINVAL, EDTYPE, EALIGN, EWORKSPACE = 0, -1, -2, -3, -4
P = [ctypes.c_void_p(0x100000 * (i + 1)) for i in range(8)]
BAD = ctypes.c_void_p(0x100008)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U = 2.0 ** -24      # half a step of fp32


# ---------------------------------------------------------------------------
# 64-bit values
# ---------------------------------------------------------------------------

def scale32(top):
    """Product of two fp32 factors, rounded to fp32 (in float64 it is exact before)."""
    return (np.asarray(top, np.float64) * np.float64(np.float32(1.0 / 127.0))).astype(np.float32)


def quantize64(x):
    """(codes, scales) of a float64 matrix whose entries are fp32 or bf16 values, from the definition."""
    s = np.maximum(scale32(np.abs(x).max(axis=1)), np.float32(2.0 ** -126))
    return np.rint(x / s.astype(np.float64)[:, None]).astype(np.int8), s


def activation(g, act):
    """(value, slope) in float64."""
    if act == "silu":
        s = torch.special.expit(g)
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        p = torch.special.erfc(-g / 2 ** 0.5) / 2      # ndtr loses its digits below -5: it adds erf to 1
        return g * p, p + g * torch.exp(-g * g / 2) / (2 * np.pi) ** 0.5
    if act == "gelu_tanh":
        w = 2 * (2 / np.pi) ** 0.5 * g * (1 + 0.044715 * g * g)
        s = torch.special.expit(w)
        return g * s, s + g * s * (1 - s) * 2 * (2 / np.pi) ** 0.5 * (1 + 3 * 0.044715 * g * g)
    return torch.relu(g), (g > 0).double()


def activation_error(g, value, act):
    """How far the fp32 activation of an fp32 g may be off.

    silu: exp(-g) is off by 1.5 |g| u for its argument's rounding and 2 u of its own, the reciprocal and
    the two products by 5 u.  gelu_tanh: the same with the argument 1.6 |g| (1 + 0.045 g^2), itself off by
    4 u.  gelu: erfc by 32 u and, for its argument's rounding, 2 g^2 u of itself.  What underflows is
    below 2^-116 (1 + |g|)."""
    if act == "relu":
        return torch.zeros_like(g)
    if act == "gelu":
        rel = 36 + 3 * g * g
    else:
        w = g.abs() if act == "silu" else 1.6 * g.abs() * (1 + 0.045 * g * g)
        rel = 8 + (1.5 if act == "silu" else 6.0) * w
    return value.abs() * rel * U + 2.0 ** -116 * (1 + g.abs())


# ---------------------------------------------------------------------------
# host side
# ---------------------------------------------------------------------------

def test_quantize_refusals():
    f = mao.lib().int8_quantize
    good = dict(x=P[0], dt=1, rows=8, cols=200, ldx=200, q=P[1], ldq=256, s=P[2])

    def call(**kw):
        a = {**good, **kw}
        return f(a["x"], a["dt"], a["rows"], a["cols"], a["ldx"], a["q"], a["ldq"], a["s"], None)

    assert call(rows=-1) == EINVAL and call(cols=-1) == EINVAL and call(rows=mao.MUON_GLU_MAX_SIDE + 1) == EINVAL
    assert call(ldx=199) == EINVAL and call(ldq=255) == EINVAL and call(ldq=192) == EINVAL and call(ldq=264) == EINVAL
    assert call(x=None) == EINVAL and call(q=None) == EINVAL and call(s=None) == EINVAL
    assert call(dt=2) == EDTYPE
    assert call(x=BAD) == EALIGN and call(q=BAD) == EALIGN and call(s=BAD) == EALIGN
    assert call(rows=0) == OK and call(cols=0) == OK      # nothing is launched


def gemm_call(f=None, **kw):
    a = {**dict(A=P[0], lda=256, sa=P[1], B=P[2], ldb=256, sb=P[3], C=P[4], dt=1, ldc=40, m=8, n=40, K=256, ws=None, nb=0), **kw}
    return mao.lib().int8_gemm(a["A"], a["lda"], a["sa"], a["B"], a["ldb"], a["sb"], a["C"], a["dt"], a["ldc"], a["m"], a["n"],
                               a["K"], a["ws"], a["nb"], None)


def glu_call(**kw):
    a = {**dict(A=P[0], lda=256, sa=P[1], Bg=P[2], sg=P[3], Bu=P[4], su=P[5], ldb=256, act=0, H=P[6], dt=1, ldh=40, m=8, n=40, K=256,
                ws=None, nb=0), **kw}
    return mao.lib().int8_glu(a["A"], a["lda"], a["sa"], a["Bg"], a["sg"], a["Bu"], a["su"], a["ldb"], a["act"], a["H"], a["dt"],
                              a["ldh"], a["m"], a["n"], a["K"], a["ws"], a["nb"], None)


@pytest.mark.parametrize("call,b,c,ldc", [(gemm_call, "B", "C", "ldc"), (glu_call, "Bu", "H", "ldh")])
def test_product_refusals(call, b, c, ldc):
    assert call(m=-1) == EINVAL and call(n=-1) == EINVAL and call(K=-64) == EINVAL
    assert call(K=200) == EINVAL and call(K=320) == EINVAL          # not whole steps; longer than the pitch
    assert call(K=mao.MUON_INT8_MAX_K + 64, lda=1 << 20, ldb=1 << 20) == EINVAL
    assert call(n=mao.MUON_GLU_MAX_SIDE + 1) == EINVAL
    assert call(lda=264) == EINVAL and call(ldb=128) == EINVAL and call(lda=1 << 24) == EINVAL and call(**{ldc: 39}) == EINVAL
    assert call(A=None) == EINVAL and call(sa=None) == EINVAL and call(**{b: None}) == EINVAL and call(**{c: None}) == EINVAL
    assert call(dt=2) == EDTYPE
    assert call(A=BAD) == EALIGN and call(sa=BAD) == EALIGN and call(**{b: BAD}) == EALIGN and call(**{c: BAD}) == EALIGN
    assert call(m=0) == OK and call(n=0) == OK                      # nothing is launched


def test_glu_refuses_unknown_activations():
    assert glu_call(act=4) == EINVAL and glu_call(act=-1) == EINVAL


def test_workspace_refusals():
    """Where a product asks for a workspace, a missing, short or misaligned one is refused."""
    L = mao.lib()
    asked = 0
    for query, call in ((L.int8_gemm_workspace_bytes, gemm_call), (L.int8_glu_workspace_bytes, glu_call)):
        for m, n, K in [(1, 4096, 4096), (40, 1024, 14336), (100, 1024, 14336), (300, 512, 65536), (4096, 4096, 4096)]:
            need = query(m, n, K)
            if need == 0:
                continue
            asked += 1
            how = dict(m=m, n=n, K=K, lda=K, ldb=K, ldc=n, ldh=n)
            assert call(**how) == EWORKSPACE and call(**how, ws=P[7], nb=need - 1) == EWORKSPACE
            assert call(**how, ws=BAD, nb=need) == EALIGN
        assert query(-1, 5, 64) == 0 and query(5, 5, mao.MUON_INT8_MAX_K + 64) == 0
    assert asked > 0


def test_python_refusals():
    """The binding checks devices, types and shapes before the library is called."""
    q, s = mao.int8_buffers(4, 100, device="cpu")
    assert q.shape == (4, 128) and s.shape == (4,)
    with pytest.raises(ValueError):
        mao.int8_quantize(torch.zeros(4, 100), q, s)                         # host tensors
    with pytest.raises(ValueError):
        mao.int8_gemm(q, s, q, s, torch.zeros(4, 5))                         # C of another shape
    with pytest.raises(ValueError):
        mao.int8_gemm(q[:, :100], s, q[:, :100], s, torch.zeros(4, 4))       # not whole steps
    with pytest.raises(ValueError):
        mao.int8_glu(q, s, q, s, q[:3], s[:3], torch.zeros(4, 4))            # weights of two shapes


# ---------------------------------------------------------------------------
# GPU
# ---------------------------------------------------------------------------

def spread(rows, cols, seed, dtype):
    rng = np.random.default_rng([seed, rows, cols])
    x = rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-6, 7, (rows, 1)) * (1 + 9 * (rng.random((1, cols)) < 0.02))
    return torch.from_numpy(x.astype(np.float32)).to(DT[dtype])


def check_quantized(x, **pitch):
    rows, cols = x.shape
    q, s = mao.int8_buffers(rows, cols)
    if pitch:
        q = torch.empty((rows, q.shape[1] + pitch["pad"]), dtype=torch.int8, device="cuda")
    q.fill_(0x55)
    s.fill_(-1.0)
    mao.int8_quantize(x, q, s)
    torch.cuda.synchronize()
    want, scales = quantize64(x.double().cpu().numpy())
    padded = -(-cols // 64) * 64
    np.testing.assert_array_equal(s.cpu().numpy(), scales)
    np.testing.assert_array_equal(q[:, :cols].cpu().numpy(), want)
    assert (q[:, cols:padded] == 0).all() and (q[:, padded:] == 0x55).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 64), (3, 65), (4, 2048), (5, 2049), (130, 257), (2, 14336), (3, 20001), (515, 8), (1000, 40)])
def test_quantize(rows, cols, dtype):
    check_quantized(spread(rows, cols, 1, dtype).cuda())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_strides(dtype):
    wide = torch.full((150, 333), float("nan"), dtype=DT[dtype])     # odd pitch, NaN between the rows
    wide[:, :300] = spread(150, 300, 2, dtype)
    check_quantized(wide.cuda()[:, :300], pad=32)
    check_quantized(wide.cuda()[:, :299], pad=16)


@pytest.mark.gpu
def test_quantize_borders():
    """Every tie and its neighbours under scales of all sizes, zeros, the smallest and the largest numbers."""
    rows = []
    ks = np.arange(-127, 128).astype(np.float64)
    for scale in (1.0, 1.5, 2.0 ** -100, 0.7, 1e-3, 3.3, 2.0 ** 100):
        top = np.float32(127.0 * scale)
        s = np.float64(scale32(top))
        for shift in (0.0, 0.5, -0.5):
            base = ((ks + shift) * s).astype(np.float32)
            for to in (None, np.float32(0), np.float32(np.inf)):
                row = base if to is None else np.nextafter(base, to)
                rows.append(np.concatenate([np.clip(row, -top, top), [top]]))
    for amax in (0.0, 1e-45, 1e-40, 2.0 ** -126, 2.0 ** -126 * 127, 1e-36, 3.4e38, float(np.finfo(np.float32).max)):
        rows.append(np.linspace(-1, 1, 256).astype(np.float32) * np.float32(amax))
    check_quantized(torch.from_numpy(np.array(rows).astype(np.float32)).cuda())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_not_finite(dtype):
    x = spread(6, 300, 3, dtype)
    x[1, 17], x[3, 299], x[4, 0] = float("nan"), float("inf"), float("-inf")
    q, s = mao.int8_buffers(6, 300)
    q.fill_(0x55)
    mao.int8_quantize(x.cuda(), q, s)
    bad = torch.tensor([False, True, False, True, True, False])
    assert torch.equal(torch.isnan(s).cpu(), bad) and (q[bad.cuda()] == 0).all()
    want, scales = quantize64(x[~bad].double().numpy())
    np.testing.assert_array_equal(q[~bad.cuda()][:, :300].cpu().numpy(), want)
    np.testing.assert_array_equal(s[~bad.cuda()].cpu().numpy(), scales)


def codes(rows, cols, seed, pad=0, low=-127):
    """Codes of a rows x cols matrix (zero past it), with `pad` more columns of rubbish, and scales over eight octaves."""
    g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + rows * 131 + cols)
    width = -(-cols // 64) * 64
    q = torch.randint(-128, 128, (rows, width + pad), generator=g, device="cuda", dtype=torch.int8)
    q[:, :cols] = torch.randint(low, 128, (rows, cols), generator=g, device="cuda", dtype=torch.int8)
    q[:, cols:width] = 0
    s = torch.exp2(8 * torch.rand(rows, generator=g, device="cuda") - 10)
    return q[:, :width], s


def exact_sum(a, b):
    """Integer sums as float64 (a float64 product of integers this small is exact)."""
    return a.double() @ b.double().t().contiguous()


def check_gemm(m, n, K, out, seed=1, pad=0, low=-127, more=5):
    (a, sa), (b, sb) = codes(m, K, seed, pad, low), codes(n, K, seed + 1, pad, low)
    c = torch.full((m, n + more), 7.0, dtype=DT[out], device="cuda")
    mao.int8_gemm(a, sa, b, sb, c[:, :n])
    ref = exact_sum(a, b) * sa.double()[:, None] * sb.double()
    err = (c[:, :n].double() - ref).abs()
    tol = ref.abs() * ((1 + 3.01 * U) * (1 + HALF_STEP[out]) - 1) + 1e-37
    assert (err <= tol).all(), f"off by {(err / tol).max().item():.2f} of what rounding allows"
    assert (c[:, n:] == 7.0).all()


# one case for each way a product is cut, its borders, and short contractions
SIZES = [(1, 1, 64), (1, 16, 64), (1, 17, 100), (3, 100, 128), (16, 257, 1000), (5, 4096, 14336), (1, 33, 131008),
         (17, 64, 64), (17, 130, 320), (64, 2304, 768), (33, 4096, 4096), (40, 200, 14336), (65, 64, 64), (100, 1000, 640),
         (129, 129, 192), (200, 384, 8192), (777, 2304, 768), (1999, 300, 256), (1100, 8192, 512), (2049, 4100, 704)]


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,K", SIZES)
def test_gemm(m, n, K, out):
    check_gemm(m, n, K, out)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,K", [(7, 50, 500), (60, 300, 500), (300, 300, 500)])
def test_gemm_pitches(m, n, K):
    check_gemm(m, n, K, "f32", seed=5, pad=48)


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,K", [(2049, 4096, 704), (1100, 8192, 512), (3000, 2560, 128)])
def test_outputs_of_whole_lines(m, n, K, out):
    """Large tiles, whose outputs take another way to memory where rows are whole cache lines; last rounds in halves and quarters."""
    check_gemm(m, n, K, out, seed=3, more=0)
    check_glu(m, n // 2, K, "silu", out, seed=4, more=0)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [2, 40, 200])
def test_gemm_largest_sums(m):
    """Codes of -128 throughout over the longest contraction: 2^31 - 2^20 fits."""
    K = mao.MUON_INT8_MAX_K
    a, b = torch.full((m, K), -128, dtype=torch.int8, device="cuda"), torch.full((48, K), -128, dtype=torch.int8, device="cuda")
    one_a, one_b = torch.ones(m, device="cuda"), torch.ones(48, device="cuda")
    c = torch.zeros(m, 48, device="cuda")
    mao.int8_gemm(a, one_a, b, one_b, c)
    assert (c == float(K * 128 * 128)).all()
    b.neg_()        # -(-128) is -128 in int8: the same sums
    b[:, ::2] = 127
    mao.int8_gemm(a, one_a, b, one_b, c)
    assert (c == float(np.float32(K // 2 * 128 * 128 - K // 2 * 128 * 127))).all()


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(5, 40), (50, 40), (300, 40)])
def test_empty_contraction(m, n):
    a, b = torch.empty(m, 0, dtype=torch.int8, device="cuda"), torch.empty(n, 0, dtype=torch.int8, device="cuda")
    c = torch.full((m, n), 3.0, device="cuda")
    mao.int8_gemm(a, torch.ones(m, device="cuda"), b, torch.ones(n, device="cuda"), c)
    assert (c == 0).all()
    c.fill_(3.0)
    mao.int8_glu(a, torch.ones(m, device="cuda"), b, torch.ones(n, device="cuda"), b, torch.ones(n, device="cuda"), c, act="gelu")
    assert (c == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("m", [3, 30, 300])
def test_a_row_that_was_not_finite_stays_visible(m):
    x = spread(m, 200, 4, "bf16").cuda()
    x[m - 1, 5] = float("inf")
    q, s = mao.int8_buffers(m, 200)
    mao.int8_quantize(x, q, s)
    b, sb = codes(70, 200, 9)
    for c in (torch.zeros(m, 70, device="cuda"), torch.zeros(m, 70, device="cuda", dtype=torch.bfloat16)):
        mao.int8_gemm(q, s, b, sb, c)
        assert torch.isnan(c[m - 1]).all() and torch.isfinite(c[:m - 1]).all()
        mao.int8_glu(q, s, b, sb, b, sb, c, act="relu")
        assert torch.isnan(c[m - 1]).all() and torch.isfinite(c[:m - 1]).all()


def check_glu(m, n, K, act, out, seed=2, pad=0, more=3):
    (a, sa), (bg, sg), (bu, su) = codes(m, K, seed, pad), codes(n, K, seed + 1, pad), codes(n, K, seed + 2, pad)
    size = 2.0 / (K ** 0.5 * 5400 * 2.0 ** -12)      # g over a few units
    sg, su = sg * size, su * size
    h = torch.full((m, n + more), 7.0, dtype=DT[out], device="cuda")
    mao.int8_glu(a, sa, bg, sg, bu, su, h[:, :n], act=act)
    g = exact_sum(a, bg) * sa.double()[:, None] * sg.double()
    u = exact_sum(a, bu) * sa.double()[:, None] * su.double()
    v, _ = activation(g, act)
    near = 3.01 * U                                  # of g and u; no slope is over 1.2
    ref = v * u
    err32 = u.abs() * (activation_error(g, v, act) + 1.2 * g.abs() * near) * (1 + near) + ref.abs() * (near + U)
    tol = (err32 + (ref.abs() + err32) * HALF_STEP[out]) * 1.001 + 1e-37
    err = (h[:, :n].double() - ref).abs()
    assert (err <= tol).all(), f"off by {(err / tol).max().item():.2f} of what rounding allows"
    assert (h[:, n:] == 7.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,K", SIZES)
def test_glu(m, n, K):
    check_glu(m, n, K, "silu", "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("m,n,K", [(2, 100, 300), (50, 100, 300), (200, 1000, 300), (40, 200, 14336)])
def test_glu_activations(m, n, K, act, out):
    check_glu(m, n, K, act, out, seed=7, pad=16)


@pytest.mark.gpu
def test_calls_on_streams_and_in_graphs():
    """The same bits from a side stream and from a graph that is replayed with the program's own work between."""
    sizes = [(3, 500, 2048), (40, 512, 14336), (200, 384, 8192), (600, 700, 512)]
    work = []
    for m, n, K in sizes:
        (a, sa), (bg, sg), (bu, su) = codes(m, K, 21), codes(n, K, 22), codes(n, K, 23)
        x = spread(m, K, 24, "bf16").cuda()
        q, s = mao.int8_buffers(m, K)
        work.append(dict(a=a, sa=sa, bg=bg, sg=sg, bu=bu, su=su, x=x, q=q, s=s, c=torch.zeros(m, n, device="cuda"),
                         h=torch.zeros(m, n, device="cuda", dtype=torch.bfloat16),
                         ws=[torch.empty(max(f(m, n, K), 16), dtype=torch.uint8, device="cuda")
                             for f in (mao.int8_gemm_workspace_bytes, mao.int8_glu_workspace_bytes)]))

    def calls(stream=None):
        for w in work:
            mao.int8_quantize(w["x"], w["q"], w["s"], stream=stream)
            mao.int8_gemm(w["q"], w["s"], w["bg"], w["sg"], w["c"], workspace=w["ws"][0], stream=stream)
            mao.int8_glu(w["a"], w["sa"], w["bg"], w["sg"], w["bu"], w["su"], w["h"], workspace=w["ws"][1], stream=stream)

    def outputs():
        torch.cuda.synchronize()
        got = [w[k].clone() for w in work for k in ("q", "s", "c", "h")]
        for w in work:
            for k in ("q", "s", "c", "h"):
                w[k].zero_()
        torch.cuda.synchronize()
        return got

    calls()
    want = outputs()
    side = torch.cuda.Stream()
    calls(side)
    for a, b in zip(outputs(), want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    outputs()
    for _ in range(4):
        graph.replay()
        for a, b in zip(outputs(), want):
            assert torch.equal(a, b)
        calls()
        for a, b in zip(outputs(), want):
            assert torch.equal(a, b)
