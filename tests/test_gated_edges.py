"""The gated and int8 calls where they are used out of the ordinary: streams, devices, large offsets, extremes, neighbours."""
import pytest
import torch

import matrix_aware_optimizer_amd as mao
from matrix_aware_optimizer_amd import _abi
from test_gated import ACTS, BF, U, blank, product, randn, within
from test_int8 import activation, codes, exact_sum

NEW = ("int8_gemm", "int8_glu", "glu_forward", "glu_backward", "glu_weight_grad")


# ---------------------------------------------------------------------------
# workspaces
# ---------------------------------------------------------------------------

def stream_of(address):
    """The stream whose pool the memory at an address belongs to."""
    for segment in torch.cuda.memory_snapshot():
        if segment["address"] <= address < segment["address"] + segment["total_size"]:
            return segment["stream"]
    raise AssertionError("not memory of the allocator")


@pytest.mark.gpu
def test_workspaces_come_from_the_stream_of_the_call(monkeypatch):
    seen, L = [], mao.lib()

    class Recording:
        def __getattr__(self, name):
            real = getattr(L, name)
            if name not in NEW:
                return real

            def call(*args):
                if args[-3]:
                    seen.append((name, args[-1], args[-3]))
                return real(*args)
            return call

    (a, sa), (b, sb) = codes(100, 8192, 1), codes(512, 8192, 2)
    x, w, h = randn((100, 4096), 1), randn((256, 4096), 2), blank(100, 256)
    dh, w2, dx = randn((100, 4096), 3), randn((4096, 256), 4), blank(100, 256)
    g, t, m = randn((4096, 256), 5), randn((4096, 128), 6), torch.zeros(256, 128, device="cuda")
    c = torch.empty(100, 512, device="cuda")
    monkeypatch.setattr(_abi, "lib", Recording)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, 0, side, side.cuda_stream):
        with torch.cuda.stream(other):                   # current is another stream than the call's
            mao.int8_gemm(a, sa, b, sb, c, stream=stream)
            mao.int8_glu(a, sa, b, sb, b, sb, c, stream=stream)
            mao.glu_forward(x, w, w, h, stream=stream)
            mao.glu_backward(dh, dh, dh, torch.empty_like(dh), torch.empty_like(dh), w2, w2, dx, stream=stream)
            mao.glu_weight_grad(g, g, t, m, m.clone(), stream=stream)
        want = other.cuda_stream if stream is None else stream if isinstance(stream, int) else stream.cuda_stream
        assert [name for name, _, _ in seen] == list(NEW)
        for _, handle, address in seen:
            assert handle == want and stream_of(address) == want
        del seen[:]
        torch.cuda.synchronize()


@pytest.mark.gpu
def test_a_short_workspace_is_refused():
    x, w, h = randn((100, 4096), 1), randn((256, 4096), 2), blank(100, 256)
    need = mao.glu_forward_workspace_bytes(100, 256, 4096)
    assert need > 0
    with pytest.raises(mao.MuonError):
        mao.glu_forward(x, w, w, h, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    assert (h == 7.0).all()


# ---------------------------------------------------------------------------
# devices
# ---------------------------------------------------------------------------

@pytest.mark.gpu
def test_another_current_device_is_refused(monkeypatch):
    x, w, h = randn((4, 64), 1), randn((8, 64), 2), blank(4, 8)
    q, s = mao.int8_buffers(4, 64)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        mao.glu_forward(x, w, w, h)
    with pytest.raises(ValueError, match="current device"):
        mao.int8_quantize(x, q, s)


@pytest.mark.gpu
def test_tensors_of_two_devices_are_refused():
    x, w, h = randn((4, 64), 1), randn((8, 64), 2), blank(4, 8)
    with pytest.raises(ValueError, match="one device"):
        mao.glu_forward(x, w.cpu(), w, h)
    with pytest.raises(ValueError, match="one device"):
        mao.glu_weight_grad(h, h.cpu(), x, torch.zeros(8, 64, device="cuda"), torch.zeros(8, 64, device="cuda"))


# ---------------------------------------------------------------------------
# offsets past 32 bits, neighbours of the outputs
# ---------------------------------------------------------------------------

@pytest.mark.gpu
def test_offsets_past_32_bits_int8():
    """The last rows of operands and outputs of more than 2^31 bytes, and of 2^32 entries of C."""
    K, m = 2048, (1 << 31) // 2048 + 300
    a = torch.zeros(m, K, dtype=torch.int8, device="cuda")
    tail, _ = codes(400, K, 1)
    a[-400:] = tail
    b, sb = codes(40, K, 2)
    one = torch.ones(m, device="cuda")
    c = torch.empty(m, 40, device="cuda")
    mao.int8_gemm(a, one, b, sb, c)
    assert (c[:-400] == 0).all()
    ref = exact_sum(tail, b) * sb.double()
    assert ((c[-400:].double() - ref).abs() <= ref.abs() * 3.01 * U).all()
    # B in their place, few rows of A: the last columns
    c = torch.empty(3, m, device="cuda")
    mao.int8_gemm(tail[:3], one[:3], a, one, c)
    ref = exact_sum(tail[:3], tail)
    assert (c[:, :-400] == 0).all() and ((c[:, -400:].double() - ref).abs() <= ref.abs() * U).all()
    del a, c
    q, s = mao.int8_buffers(m, K)
    x = torch.zeros(m, K, dtype=BF, device="cuda")
    x[-1] = 127.0
    mao.int8_quantize(x, q, s)
    assert (q[-1] == 127).all() and (q[-2] == 0).all() and s[-1] == s.max()


@pytest.mark.gpu
def test_offsets_past_32_bits_gated():
    f, d = 72, 2048
    t = (1 << 31) // (2 * d) + 300          # x of more than 2^31 bytes
    x = torch.zeros(t, d, dtype=BF, device="cuda")
    tail = randn((300, d), 1)
    x[-300:] = tail
    w = [randn((f, d), s, size=d ** -0.5) for s in (2, 3)]
    h = blank(t, f)
    mao.glu_forward(x, *w, h)
    small = blank(300, f)
    mao.glu_forward(tail, *w, small)
    assert (h[:-300] == 0).all()
    # both are within their rounding of the same values
    assert (h[-300:].double() - small.double()).abs().max() <= 2.0 ** -7 * small.double().abs().max()
    # all tokens summed: only the last ones count
    dg = [torch.ones(t, f, dtype=BF, device="cuda") for _ in range(2)]
    m = [torch.zeros(f, d, device="cuda") for _ in range(2)]
    mao.glu_weight_grad(*dg, x, *m)
    ref = tail.double().sum(0)
    assert all(((k.double() - ref).abs() <= 2 * 300 * U * tail.double().abs().sum(0) + 1e-30).all() for k in m)
    # dx of more than 2^31 bytes
    dx = blank(t, d)
    mao.glu_backward(dg[0], dg[0], dg[0], torch.empty_like(dg[0]), torch.empty_like(dg[0]), *w, dx)
    assert torch.equal(dx[0], dx[-1]) and torch.isfinite(dx[-300:].float()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("t", [5, 40, 150])
@pytest.mark.parametrize("f,d", [(72, 104), (65, 67)])
def test_rows_behind_the_outputs_stay(t, f, d):
    x, w = randn((t, d), 1), [randn((f, d), s, size=0.1) for s in (2, 3)]
    big = {k: blank(r + 3, c, dtype=ty) for k, r, c, ty in (("h", t, f, BF), ("g", t, f, BF), ("u", t, f, BF), ("dg", t, f, BF), ("du", t, f, BF),
                                                          ("dx", t, d, BF), ("mg", f, d, torch.float32), ("mu", f, d, torch.float32))}
    v = {k: b[:-3] for k, b in big.items()}
    mao.glu_forward(x, *w, v["h"], v["g"], v["u"])
    mao.glu_backward(v["h"], v["g"], v["u"], v["dg"], v["du"], *w, v["dx"])
    mao.glu_weight_grad(v["dg"], v["du"], x, v["mg"], v["mu"])
    (a, sa), (b, sb) = codes(t, d, 4), codes(f, d, 5)
    c = blank(t + 3, f)
    mao.int8_gemm(a, sa, b, sb, c[:-3])
    q, s = mao.int8_buffers(t + 3, d)
    q.fill_(9)
    s.fill_(9.0)
    mao.int8_quantize(x, q[:-3], s[:-3])
    torch.cuda.synchronize()
    assert all((k[-3:] == 7.0).all() for k in (*big.values(), c)) and (q[-3:] == 9).all() and (s[-3:] == 9.0).all()


# ---------------------------------------------------------------------------
# extremes
# ---------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
def test_saturated_gates(act):
    """Far from zero the activation is x or 0 and its slope 1 or 0, to the ends of the format."""
    g = torch.tensor([[200.0, 1e4, 1e18, 2e19, 1e25, 3e38, -200.0, -1e4, -1e18, -2e19, -1e25, -3e38]], dtype=BF, device="cuda")
    one = torch.ones_like(g)
    dg, du, h = (torch.empty_like(g) for _ in range(3))
    mao.glu_backward(one, g, one, dg, du, h=h, act=act)
    assert torch.equal(dg, (g > 0).to(BF)) and torch.equal(du, g.clamp(min=0)) and torch.equal(h, g.clamp(min=0))


@pytest.mark.gpu
def test_not_finite_values_stay_in_their_rows():
    """A NaN in one token reaches that token's outputs and the weight gradients, and no other token."""
    t, f, d = 150, 72, 104
    x, w = randn((t, d), 1), [randn((f, d), s, size=0.1) for s in (2, 3)]
    x[77, 3] = float("nan")
    h, g, u, dg, du, dx = blank(t, f), blank(t, f), blank(t, f), blank(t, f), blank(t, f), blank(t, d)
    mao.glu_forward(x, *w, h, g, u)
    mao.glu_backward(torch.ones_like(h), g, u, dg, du, *w, dx)
    rest = torch.arange(t, device="cuda") != 77
    for k in (h, g, u, dg, du, dx):
        assert torch.isnan(k[77]).all() and torch.isfinite(k[rest]).all()


# ---------------------------------------------------------------------------
# two calls at once
# ---------------------------------------------------------------------------

@pytest.mark.gpu
def test_two_streams_at_once():
    """The same products on two streams at once, each with a workspace of its own, give the bits of one at a time."""
    sizes = [(100, 256, 4096), (777, 256, 512)]
    inputs = [(randn((t, d), 1), randn((f, d), 2, size=0.1), randn((f, d), 3, size=0.1)) for t, f, d in sizes]
    want = []
    for x, wg, wu in inputs:
        h = blank(x.shape[0], wg.shape[0])
        mao.glu_forward(x, wg, wu, h)
        want.append(h)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sizes]
    got = [[blank(*h.shape) for _ in range(10)] for h in want]
    torch.cuda.synchronize()
    for k in range(10):
        for (x, wg, wu), st, h in zip(inputs, streams, got):
            mao.glu_forward(x, wg, wu, h[k], stream=st)
    torch.cuda.synchronize()
    for hs, w in zip(got, want):
        assert all(torch.equal(h, w) for h in hs)


@pytest.mark.gpu
def test_one_matrix_as_both_weights():
    """The same matrix twice, and the same gradient twice."""
    t, f, d = 200, 136, 72
    x, w = randn((t, d), 1), randn((f, d), 2, size=0.2)
    h, g, u = blank(t, f), blank(t, f), blank(t, f)
    mao.glu_forward(x, w, w, h, g, u, act="relu")
    assert torch.equal(g, u)
    m = [blank(f, d, dtype=torch.float32) for _ in range(2)]
    mao.glu_weight_grad(g, g, x, *m)
    assert torch.equal(*m)
    r, mag = product(g.t(), x)
    within(m[0], r, 2 * t * U * mag + 2 * U * r.abs(), "m")
    assert torch.equal(activation(g.double(), "relu")[0], g.double().clamp(min=0))
