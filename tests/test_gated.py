"""The gated feed-forward block in bf16: forward, both backward halves, against 64-bit values.

Tolerances.  A sum of K products of bf16 values in fp32, in any order, is off by at most
K 2^-23 of the sum of their magnitudes (half a step for each addition would be 2^-24; twice
that leaves room for additions that cut).  The activation's own error is counted in
tests/test_int8.py; every stored bf16 value is off by 2^-8 of itself, an fp32 one by 2^-24.
"""
import ctypes

import pytest
import torch

import matrix_aware_optimizer_amd as mao
from test_int8 import DT, HALF_STEP, U, activation, activation_error

OK, EINVAL, EDTYPE, EALIGN, EWORKSPACE = 0, -1, -2, -3, -4
P = [ctypes.c_void_p(0x100000 * (i + 1)) for i in range(12)]
BAD = ctypes.c_void_p(0x100008)
BF = torch.bfloat16
ACTS = ["silu", "gelu", "gelu_tanh", "relu"]


# ---------------------------------------------------------------------------
# host side
# ---------------------------------------------------------------------------

def forward_call(**kw):
    a = {**dict(X=P[0], ldx=64, Wg=P[1], Wu=P[2], ldw=64, act=0, H=P[3], ldh=40, G=P[4], U=P[5], ldg=40, t=20, f=40, d=64, ws=None, nb=0), **kw}
    return mao.lib().glu_forward(a["X"], a["ldx"], a["Wg"], a["Wu"], a["ldw"], a["act"], a["H"], a["ldh"], a["G"], a["U"], a["ldg"],
                                 a["t"], a["f"], a["d"], a["ws"], a["nb"], None)


def backward_call(**kw):
    a = {**dict(dH=P[0], lddh=40, G=P[1], U=P[2], ldg=40, act=0, dG=P[3], dU=P[4], ldd=40, H=P[5], ldh=40, Wg=P[6], Wu=P[7], ldw=64,
                dX=P[8], lddx=64, t=20, f=40, d=64, ws=None, nb=0), **kw}
    return mao.lib().glu_backward(a["dH"], a["lddh"], a["G"], a["U"], a["ldg"], a["act"], a["dG"], a["dU"], a["ldd"], a["H"], a["ldh"],
                                  a["Wg"], a["Wu"], a["ldw"], a["dX"], a["lddx"], a["t"], a["f"], a["d"], a["ws"], a["nb"], None)


def weight_call(**kw):
    a = {**dict(dG=P[0], dU=P[1], ldd=40, X=P[2], ldx=64, Mg=P[3], Mu=P[4], dt=0, ldm=64, t=20, f=40, d=64, ws=None, nb=0), **kw}
    return mao.lib().glu_weight_grad(a["dG"], a["dU"], a["ldd"], a["X"], a["ldx"], a["Mg"], a["Mu"], a["dt"], a["ldm"], a["t"], a["f"],
                                     a["d"], 1.0, 0.0, a["ws"], a["nb"], None)


@pytest.mark.parametrize("call,pointers,pitches", [
    (forward_call, ["X", "Wg", "Wu", "H", "G", "U"], [("ldx", 63), ("ldw", 63), ("ldh", 39), ("ldg", 39), ("ldx", 1 << 23), ("ldw", 1 << 23)]),
    (backward_call, ["dH", "G", "U", "dG", "dU", "Wg", "Wu"], [("lddh", 39), ("ldg", 39), ("ldd", 39), ("ldh", 39), ("ldw", 63), ("lddx", 63),
                                                               ("ldd", 1 << 23), ("ldw", 1 << 23)]),
    (weight_call, ["dG", "dU", "X", "Mg", "Mu"], [("ldd", 39), ("ldx", 63), ("ldm", 63), ("ldd", 1 << 23), ("ldx", 1 << 23)])])
def test_refusals(call, pointers, pitches):
    for side in "tfd":
        assert call(**{side: -1}) == EINVAL and call(**{side: mao.MUON_GLU_MAX_SIDE + 1}) == EINVAL
    for p in pointers:
        assert call(**{p: None}) == EINVAL and call(**{p: BAD}) == EALIGN
    for p, v in pitches:
        assert call(**{p: v}) == EINVAL


def test_other_refusals():
    for call in (forward_call, backward_call):
        assert call(act=4) == EINVAL and call(act=-1) == EINVAL
        assert call(t=0) == OK                                       # nothing is launched
    assert forward_call(f=0) == OK
    assert weight_call(dt=2) == EDTYPE and weight_call(f=0) == OK and weight_call(d=0) == OK
    assert backward_call(H=BAD) == EALIGN and backward_call(dX=BAD) == EALIGN


@pytest.mark.parametrize("call,pairs", [
    (forward_call, ["H G", "H U", "G U"]), (weight_call, ["Mg Mu"]),
    (backward_call, ["dG dU", "H dG", "H dU", "dX dG", "dX dU", "dX H", "dX Wg", "dX Wu"])])
def test_outputs_over_each_other_are_refused(call, pairs):
    for pair in pairs:
        a, b = pair.split()
        assert call(**{a: P[9], b: P[9]}) == EINVAL


def test_more_entries_than_any_memory_are_refused():
    side = mao.MUON_GLU_MAX_SIDE
    assert forward_call(t=side, f=side, ldh=side, ldg=side) == EINVAL
    assert backward_call(t=side, d=side, ldw=side, lddx=side) == EINVAL
    assert weight_call(f=side, d=side, ldd=side, ldx=side, ldm=side) == EINVAL


def test_workspace_refusals():
    L = mao.lib()
    asked = {}
    for name, call, pitch in (("glu_forward", forward_call, dict(ldx="d", ldw="d", ldh="f", ldg="f")),
                              ("glu_backward", backward_call, dict(lddh="f", ldg="f", ldd="f", ldh="f", ldw="d", lddx="d")),
                              ("glu_weight_grad", weight_call, dict(ldd="f", ldx="d", ldm="d"))):
        query = getattr(L, name + "_workspace_bytes")
        for t, f, d in [(1, 4096, 4096), (100, 1024, 8192), (300, 512, 512), (8192, 256, 256), (4096, 4096, 4096)]:
            need = query(t, f, d)
            if need == 0:
                continue
            asked[name] = True
            how = dict(t=t, f=f, d=d, **{k: dict(f=f, d=d)[v] for k, v in pitch.items()})
            assert call(**how) == EWORKSPACE and call(**how, ws=P[9], nb=need - 1) == EWORKSPACE
            assert call(**how, ws=BAD, nb=need) == EALIGN
        assert query(-1, 5, 5) == 0 and query(5, 5, mao.MUON_GLU_MAX_SIDE + 1) == 0
    assert len(asked) == 3


def test_python_refusals():
    """The binding checks devices, types, shapes and pitches before the library is called."""
    def z(*s, dtype=BF):
        return torch.zeros(*s, dtype=dtype)

    x, w, h = z(4, 16), z(8, 16), z(4, 8)
    with pytest.raises(ValueError):
        mao.glu_forward(x, w, w, h)                                   # host tensors
    for bad in ((x.float(), w, w, h), (x, w.float(), w, h), (x, w, w, h.float())):
        with pytest.raises((TypeError, ValueError)):
            mao.glu_forward(*bad)
    with pytest.raises(ValueError):
        mao.glu_forward(x, w, w, h, g=h)                              # g without u
    with pytest.raises(ValueError):
        mao.glu_backward(h, h, h, h, h, dx=x)                         # dx without weights
    with pytest.raises(ValueError):
        mao.glu_weight_grad(h, h, x, w.float(), w.float())


# ---------------------------------------------------------------------------
# GPU
# ---------------------------------------------------------------------------

def randn(shape, seed, pad=0, size=1.0):
    """bf16 normal values in a matrix whose pitch is `pad` longer, NaN between the rows."""
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + shape[0] * 31 + shape[1])
    t = torch.full((shape[0], shape[1] + pad), float("nan"), dtype=BF, device="cuda")
    t[:, :shape[1]] = size * torch.randn(shape, generator=g, device="cuda")
    return t[:, :shape[1]]


def blank(rows, cols, pad=0, dtype=BF):
    return torch.full((rows, cols + pad), 7.0, dtype=dtype, device="cuda")


def product(a, b):
    """(a b, |a| |b|) in float64."""
    a, b = a.double().contiguous(), b.double().contiguous()
    return a @ b, a.abs() @ b.abs()


def within(got, ref, tol, what):
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), f"{what}: off by {(err / tol).max().item():.2f} of what rounding allows"


def check_forward(t, f, d, act="silu", saved=True, pad=0, seed=1):
    x, wg, wu = randn((t, d), seed, pad), randn((f, d), seed + 1, pad, d ** -0.5), randn((f, d), seed + 2, pad, d ** -0.5)
    h = blank(t, f, 3 * pad)
    g, u = (blank(t, f, pad), blank(t, f, pad)) if saved else (None, None)
    mao.glu_forward(x, wg, wu, h[:, :f], *((g[:, :f], u[:, :f]) if saved else ()), act=act)
    (rg, mg), (ru, mu) = product(x, wg.t()), product(x, wu.t())
    eg, eu = d * 2 * U * mg, d * 2 * U * mu
    if saved:
        within(g[:, :f], rg, eg + (rg.abs() + eg) * 2.0 ** -8, "g")
        within(u[:, :f], ru, eu + (ru.abs() + eu) * 2.0 ** -8, "u")
        assert (g[:, f:] == 7.0).all() and (u[:, f:] == 7.0).all()
    v, _ = activation(rg, act)
    ev = activation_error(rg, v, act) + 1.2 * eg
    e32 = ru.abs() * ev + (v.abs() + ev) * eu + (v * ru).abs() * U
    within(h[:, :f], v * ru, 1.001 * (e32 + ((v * ru).abs() + e32) * 2.0 ** -8) + 1e-37, "h")
    assert (h[:, f:] == 7.0).all()


# one case for each way a product is cut, borders of the tiles, odd sides (rows that do not start at 16 bytes)
FORWARD = [(1, 1, 1), (1, 16, 32), (1, 17, 40), (3, 100, 65), (16, 257, 1000), (2, 33, 4096), (5, 4096, 768), (17, 64, 8), (17, 65, 31),
           (40, 200, 8192), (64, 1152, 768), (33, 2304, 100), (65, 64, 32), (100, 1000, 328), (129, 129, 97), (130, 96, 4104), (200, 384, 4096),
           (777, 2304, 768), (300, 301, 303), (1999, 72, 256), (2049, 2052, 360), (1100, 4096, 200), (2100, 4100, 263), (2500, 2304, 1000)]


@pytest.mark.gpu
@pytest.mark.parametrize("t,f,d", FORWARD)
def test_forward(t, f, d):
    check_forward(t, f, d)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("pad", [0, 8, 5])
@pytest.mark.parametrize("t,f,d", [(4, 72, 200), (50, 72, 200), (300, 136, 200)])
def test_forward_activations_and_pitches(t, f, d, pad, act):
    check_forward(t, f, d, act, saved=pad != 8, pad=pad, seed=11)


@pytest.mark.gpu
@pytest.mark.parametrize("t", [3, 40, 300])
def test_forward_extremes(t):
    """Rows that are zero, huge, infinite or NaN stay by themselves; large negative gates give zeros and no NaN."""
    f, d = 72, 64
    x = randn((t, d), 3)
    wg, wu = randn((f, d), 4, size=0.1), randn((f, d), 5, size=0.1)
    h, g, u = blank(t, f), blank(t, f), blank(t, f)
    x[0] = 0.0
    x[1] = 2e4 * x[1].float()
    x[2, 7] = float("inf")
    for act in ACTS:
        mao.glu_forward(x, wg, wu, h, g, u, act=act)
        assert (h[0] == 0).all() and (g[0] == 0).all()
        a, b = x.double() @ wg.double().t(), x.double() @ wu.double().t()
        big = a[1].abs() > 200          # saturated: a(g) is g or 0
        assert big.any()
        v, e = activation(a[1], act)[0], d * 2 * U * (x[1].double().abs() @ wg.double().abs().t())
        eu = d * 2 * U * (x[1].double().abs() @ wu.double().abs().t())
        err = (v.abs() * eu + e * b[1].abs() + (v * b[1]).abs() * 2.0 ** -8) * 1.01 + 1e-30
        within(h[1][big], (v * b[1])[big], err[big], act)
        assert not torch.isfinite(h[2]).any()          # +-inf products, and inf * 0 where the gate closes
        assert torch.isfinite(h[3:]).all()


def check_backward(t, f, d, act="silu", again=True, pad=0, seed=1, input=True):
    dh, g, u = randn((t, f), seed, pad), randn((t, f), seed + 1, pad, 2.0), randn((t, f), seed + 2, pad)
    wg, wu = randn((f, d), seed + 3, pad, f ** -0.5), randn((f, d), seed + 4, pad, f ** -0.5)
    dg, du, dx, h = blank(t, f, pad), blank(t, f, pad), blank(t, d, 2 * pad), blank(t, f, 2 * pad) if again else None
    mao.glu_backward(dh, g, u, dg[:, :f], du[:, :f], *((wg, wu, dx[:, :d]) if input else ()), h=h[:, :f] if again else None, act=act)
    g64, u64, dh64 = g.double(), u.double(), dh.double()
    v, s = activation(g64, act)
    ev = activation_error(g64, v, act)
    # a slope's terms are a few times 1 + g^2 at most, each off by a few u and the argument's rounding
    es = 16 * (1 + g64 * g64) * (1 + g64.abs()) * U if act != "relu" else 0 * g64
    for name, got, ref, e in (("dg", dg, dh64 * u64 * s, (dh64 * u64).abs() * es), ("du", du, dh64 * v, dh64.abs() * ev), ("h", h, v * u64, u64.abs() * ev)):
        if got is None:
            continue
        e = e + ref.abs() * 3 * U
        within(got[:, :f], ref, 1.001 * (e + (ref.abs() + e) * 2.0 ** -8) + 1e-37, name)
        assert (got[:, f:] == 7.0).all()
    if input:
        (r0, m0), (r1, m1) = product(dg[:, :f], wg), product(du[:, :f], wu)      # of dg and du as stored
        e = 2 * f * 2 * U * (m0 + m1)
        within(dx[:, :d], r0 + r1, e + ((r0 + r1).abs() + e) * 2.0 ** -8, "dx")
        assert (dx[:, d:] == 7.0).all()


BACKWARD = [(1, 1, 1), (1, 32, 8), (1, 40, 16), (3, 100, 65), (16, 1000, 256), (17, 31, 64), (40, 4096, 200), (64, 768, 1152), (33, 104, 2304),
            (65, 32, 64), (100, 328, 1000), (129, 97, 129), (200, 4096, 384), (777, 2304, 768), (300, 303, 301), (1999, 256, 72), (2049, 360, 4104),
            (4100, 296, 4096), (2100, 2303, 4096), (2100, 1100, 4095), (2049, 320, 4096)]


@pytest.mark.gpu
@pytest.mark.parametrize("t,f,d", BACKWARD)
def test_backward(t, f, d):
    check_backward(t, f, d)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("pad", [0, 8, 5])
@pytest.mark.parametrize("t,f,d", [(4, 200, 72), (50, 200, 72), (300, 200, 136)])
def test_backward_activations_and_pitches(t, f, d, pad, act):
    check_backward(t, f, d, act, again=pad != 8, pad=pad, seed=13)


@pytest.mark.gpu
@pytest.mark.parametrize("t,f", [(1, 1), (5, 77), (40, 2304)])
def test_backward_without_the_input(t, f):
    check_backward(t, f, 8, input=False)


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [0, 3])
def test_backward_in_place(pad):
    """dg, du and h over dh, g or u give the bits that separate outputs have."""
    t, f = 70, 203
    def inputs():
        return [randn((t, f), s, pad) for s in (31, 32, 33)]
    dh, g, u = inputs()
    want = [blank(t, f) for _ in range(3)]
    mao.glu_backward(dh, g, u, want[0], want[1], h=want[2])
    for order in ((0, 1, 2), (1, 2, 0), (2, 0, 1)):
        held = inputs()
        mao.glu_backward(*held, held[order[0]], held[order[1]], h=held[order[2]])
        for k in range(3):
            assert torch.equal(held[order[k]], want[k])


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
def test_slopes_against_differences(act):
    """dg for dh = u = 1 against central differences of the activation in float64, zero and the ends among the points."""
    g = torch.cat([torch.linspace(-12, 12, 4001), torch.tensor([0.0, -0.0, 1e-3, -1e-3, 60.0, -60.0, 1e4, -1e4])]).to(BF).cuda()[None]
    one = torch.ones_like(g)
    dg, du = torch.empty_like(g), torch.empty_like(g)
    mao.glu_backward(one, g, one, dg, du, act=act)
    x, e = g.double(), 1e-5
    diff = (activation(x + e, act)[0] - activation(x - e, act)[0]) / (2 * e)
    if act == "relu":
        diff = torch.where(x.abs() <= e, (x > 0).double(), diff)      # a difference across the kink is neither slope
    # differences: e^2 / 6 of the third derivative (under 3), and 2^-53 |a| / e of rounding
    within(dg, diff, 1.01 * diff.abs() * 2.0 ** -8 + 16 * (1 + x * x).clamp(max=200) * 13 * U + 1e-10 + x.abs() * 1e-10, act)
    within(du, activation(x, act)[0], 1.01 * activation(x, act)[0].abs() * 2.0 ** -8 + 1e-30, act)


def check_weights(t, f, d, out="f32", beta=0.95, alpha=0.05, pad=0, seed=1):
    dg, du, x = randn((t, f), seed, pad), randn((t, f), seed + 1, pad), randn((t, d), seed + 2, pad)
    m = [blank(f, d, pad, DT[out]) for _ in range(2)]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    for k in m:
        k[:, :d] = torch.randn((f, d), generator=gen, device="cuda") if beta else float("nan")
    was = [k.double()[:, :d] for k in m]
    mao.glu_weight_grad(dg, du, x, m[0][:, :d], m[1][:, :d], alpha=alpha, beta=beta)
    for name, got, old, grad in (("mg", m[0], was[0], dg), ("mu", m[1], was[1], du)):
        r, mag = product(grad.t(), x)
        # alpha and beta cross the interface as fp32
        a, b = float(torch.tensor(alpha)), float(torch.tensor(beta))
        ref = a * r + (b * old if beta else 0.0)
        e = abs(a) * t * 2 * U * mag + 2 * U * (abs(a) * r.abs() + (abs(b) * old.abs() if beta else 0.0)) + 1e-37
        within(got[:, :d], ref, 1.001 * (e + (ref.abs() + e) * HALF_STEP[out]), name)
        assert (got[:, d:] == 7.0).all()


# large tiles with whole lines, without (2056 and 4104 columns), through registers (4095 columns, long sums)
WEIGHTS = [(2100, 2304, 4095), (300, 2304, 4096), (2080, 4096, 2304), (1, 1, 1), (1, 8, 8), (2, 40, 16), (31, 129, 65), (32, 128, 128), (33, 136, 72), (100, 328, 1000), (777, 2304, 768), (777, 301, 303),
           (8192, 256, 136), (5000, 100, 64), (64, 4104, 2056), (200, 4096, 4096)]


@pytest.mark.gpu
@pytest.mark.parametrize("out,beta", [("f32", 0.95), ("bf16", 0.0)])
@pytest.mark.parametrize("t,f,d", WEIGHTS)
def test_weight_grad(t, f, d, out, beta):
    check_weights(t, f, d, out, beta)


@pytest.mark.gpu
@pytest.mark.parametrize("out,beta", [("f32", 0.0), ("bf16", 0.95), ("f32", 1.0)])
@pytest.mark.parametrize("pad", [8, 5])
def test_weight_grad_pitches(pad, out, beta):
    check_weights(90, 200, 136, out, beta, alpha=-1.5, pad=pad, seed=17)


@pytest.mark.gpu
def test_empty_sums():
    """No tokens: the momentum only decays.  No inputs: zeros.  No outputs: a zero input gradient."""
    e = torch.empty
    mg, mu = torch.full((40, 24), 2.0, device="cuda"), torch.full((40, 24), -4.0, device="cuda")
    mao.glu_weight_grad(e(0, 40, dtype=BF, device="cuda"), e(0, 40, dtype=BF, device="cuda"), e(0, 24, dtype=BF, device="cuda"), mg, mu, beta=0.5)
    assert (mg == 1.0).all() and (mu == -2.0).all()
    for t in (4, 40, 200):
        h, w = blank(t, 40), e(40, 0, dtype=BF, device="cuda")
        mao.glu_forward(e(t, 0, dtype=BF, device="cuda"), w, w, h)
        assert (h == 0).all()
        none, w, dx = e(t, 0, dtype=BF, device="cuda"), e(0, 24, dtype=BF, device="cuda"), blank(t, 24)
        mao.glu_backward(none, none, none, none, none, w, w, dx)
        assert (dx == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_the_whole_gradient_against_differences(act):
    """Directional derivatives of sum(r h) over the input and both weights against differences in float64."""
    t, f, d = 48, 72, 40
    x, wg, wu, r = randn((t, d), 41), randn((f, d), 42, size=0.2), randn((f, d), 43, size=0.2), randn((t, f), 44)
    h, g, u, dg, du = (blank(t, f) for _ in range(5))
    dx, mg, mu = blank(t, d), blank(f, d, dtype=torch.float32), blank(f, d, dtype=torch.float32)
    mao.glu_forward(x, wg, wu, h, g, u, act=act)
    mao.glu_backward(r, g, u, dg, du, wg, wu, dx, act=act)
    mao.glu_weight_grad(dg, du, x, mg, mu)

    def value(x, wg, wu):
        return (r.double() * activation(x @ wg.t(), act)[0] * (x @ wu.t())).sum()

    at = [x.double(), wg.double(), wu.double()]
    g64, u64 = at[0] @ at[1].t(), at[0] @ at[2].t()
    v, s = activation(g64, act)
    # g, u, then dg, du are each stored with 2^-8 of themselves; the slope's own slope is under 1.6
    eps = 2.0 ** -8 * 1.05
    edg = r.double().abs() * (u64.abs() * (2 * s.abs() + 1.6 * g64.abs()) + 1e-5) * eps
    edu = r.double().abs() * (v.abs() + 1.2 * g64.abs() + 1e-5) * eps
    errors = [edg @ at[1].abs() + edu @ at[2].abs() + dx.double().abs() * eps, edg.t() @ at[0].abs(), edu.t() @ at[0].abs()]
    for k, (grad, err) in enumerate(zip((dx, mg, mu), errors)):
        step = torch.randn(grad.shape, generator=torch.Generator(device="cuda").manual_seed(50 + k), device="cuda", dtype=torch.float64)
        e = 1e-4
        lo, hi = ([a + sign * e * step if i == k else a for i, a in enumerate(at)] for sign in (-1, 1))
        diff = (value(*hi) - value(*lo)) / (2 * e)
        got = (grad.double() * step).sum()
        assert (got - diff).abs() <= (err * step.abs()).sum() + 1e-3 * diff.abs()
        # and entry by entry against the formula
        ref = [(r.double() * u64 * s) @ at[1] + (r.double() * v) @ at[2], (r.double() * u64 * s).t() @ at[0], (r.double() * v).t() @ at[0]][k]
        within(grad, ref, err * 1.01 + 1e-4, "gradient")


@pytest.mark.gpu
def test_calls_on_streams_and_in_graphs():
    """The same bits from a side stream and from a graph that is replayed with the program's own work between."""
    work = []
    for t, f, d in [(3, 500, 768), (40, 512, 4096), (200, 384, 4096), (300, 301, 303), (1100, 2056, 512)]:
        w = dict(x=randn((t, d), 1), wg=randn((f, d), 2, size=d ** -0.5), wu=randn((f, d), 3, size=d ** -0.5), dh=randn((t, f), 4),
                 h=blank(t, f), g=blank(t, f), u=blank(t, f), dg=blank(t, f), du=blank(t, f), dx=blank(t, d),
                 mg=blank(f, d, dtype=torch.float32), mu=blank(f, d, dtype=torch.float32))
        w["ws"] = [torch.empty(max(q(t, f, d), 16), dtype=torch.uint8, device="cuda")
                   for q in (mao.glu_forward_workspace_bytes, mao.glu_backward_workspace_bytes, mao.glu_weight_grad_workspace_bytes)]
        work.append(w)
    outs = ("h", "g", "u", "dg", "du", "dx", "mg", "mu")

    def calls(stream=None):
        for w in work:
            mao.glu_forward(w["x"], w["wg"], w["wu"], w["h"], w["g"], w["u"], workspace=w["ws"][0], stream=stream)
            mao.glu_backward(w["dh"], w["g"], w["u"], w["dg"], w["du"], w["wg"], w["wu"], w["dx"], workspace=w["ws"][1], stream=stream)
            mao.glu_weight_grad(w["dg"], w["du"], w["x"], w["mg"], w["mu"], workspace=w["ws"][2], stream=stream)

    def outputs():
        torch.cuda.synchronize()
        got = [w[k].clone() for w in work for k in outs]
        for w in work:
            for k in outs:
                w[k].zero_()
        torch.cuda.synchronize()
        return got

    calls()
    want = outputs()
    calls(torch.cuda.Stream())
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
