"""Cases, plain forms and 64-bit values of the fp8 block products and the head-wise orthogonalisation.

``own`` selects between the plain form (elementary torch operations) and the calls that a
program makes of the library.  Formats: an fp8 operand is (codes [rows, K], K a multiple of
128, zero past the matrix; scales [K/128 rounded up to 4, / 4][rows rounded up to 4][4]), each
scale byte s standing for 2^(s - 127) on one row's group of 128 columns.
"""
import math

import torch

own = False

DEV = "cuda"
FMT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
QUINTIC = (3.4445, -4.7750, 2.0315)


def up(n, m):
    return -(-n // m) * m


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # activations of a few tokens on their way into a product (serving: the smallest call)
        dict(name="quantize_tokens", op="quantize", rows=4, cols=4096, dtype="bf16", fmt="e4m3", block=1, rows_out=True, t_out=False),
        # a training step's activations: row groups for the forward product, column groups for the weight gradient
        dict(name="quantize_activations", op="quantize", rows=4096, cols=14336, dtype="bf16", fmt="e4m3", block=1, rows_out=True, t_out=True),
        # weights after an update: 128 x 128 blocks, both orientations; an odd number of rows
        dict(name="quantize_weights", op="quantize", rows=2305, cols=4096, dtype="f32", fmt="e4m3", block=128, rows_out=True, t_out=True),
        # one token through an up projection (decoding)
        dict(name="gemm_token", op="gemm", m=1, n=14336, k=4096, fa="e4m3", out="bf16", beta=0.0),
        # a small batch of tokens through a down projection (batched decoding)
        dict(name="gemm_batch", op="gemm", m=48, n=4096, k=14336, fa="e4m3", out="bf16", beta=0.0),
        # a ragged prompt through a GPT-2-small QKV projection
        dict(name="gemm_ragged", op="gemm", m=777, n=2304, k=768, fa="e4m3", out="bf16", beta=0.0),
        # forward product of a training step at the benchmark's matrix
        dict(name="gemm_forward", op="gemm", m=4096, n=14336, k=4096, fa="e4m3", out="bf16", beta=0.0),
        # its weight gradient accumulated into the fp32 momentum, output gradients in e5m2
        dict(name="gemm_momentum", op="gemm", m=14336, n=4096, k=4096, fa="e5m2", out="f32", beta=0.95),
        # one layer's query, key and value heads of GPT-2 small (12 + 12 + 12 heads of 64 x 768): direction only
        dict(name="heads_layer", op="heads", count=36, s=64, l=768, tall=False, dtype="bf16", out="bf16", update=False),
        # the heads of all layers' output projections: column blocks of 12 weights of 768 x 768
        dict(name="heads_columns", op="heads", count=144, s=64, l=768, tall=True, dtype="bf16", out="bf16", update=True),
        # a wide model's query projection: 32 heads of 128 x 4096, fp32 momentum, bf16 weights updated with decay
        dict(name="heads_wide", op="heads", count=32, s=128, l=4096, tall=False, dtype="f32", out="bf16", update=True),
        # many narrow key/value heads of an odd width, fp32 all through
        dict(name="heads_odd", op="heads", count=50, s=80, l=2309, tall=False, dtype="f32", out="f32", update=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("quantize", "gemm", "gemm", "heads"))
    if op == "quantize":
        rows, cols = _log(rng, 1, 8192), _log(rng, 64, 14336)
        while rows * cols > 4096 * 14336:
            rows //= 2
        both = rng.random() < 0.6
        return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(("bf16", "f32")) if rows * cols < 1 << 24 else "bf16",
                    fmt=rng.choice(("e4m3", "e5m2")), block=rng.choice((1, 128)), rows_out=True, t_out=both)
    if op == "gemm":
        m, n, k = _log(rng, 1, 8192), _log(rng, 64, 14336), _log(rng, 64, 14336)
        while m * n * k > 4096 * 14336 * 4096:
            m = max(1, m // 2)
        return dict(op=op, m=m, n=n, k=k, fa=rng.choice(("e4m3", "e5m2")), out=rng.choice(("bf16", "f32")),
                    beta=rng.choice((0.0, 0.95)))
    s = rng.choice((16, 32, 40, 64, 64, 72, 80, 96, 128, 128, rng.randint(8, 128)))
    l = _log(rng, 4 * s, 8192)
    count = _log(rng, 1, 256)
    while count * s * l > 144 * 128 * 1024:
        count = max(1, count // 2)
    return dict(op=op, count=count, s=s, l=l, tall=rng.random() < 0.4, dtype=rng.choice(("bf16", "f32")),
                out=rng.choice(("bf16", "f32")), update=rng.random() < 0.5)


def work(case):
    if case["op"] == "quantize":
        r, c = case["rows"], case["cols"]
        one = r * c + r * up(c, 128) // 128
        two = r * c + c * up(r, 128) // 128
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": r * c * size + one * case["rows_out"] + two * case["t_out"], "flops": 0}
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        size = 2 if case["out"] == "bf16" else 4
        return {"bytes": (m + n) * (k + k // 128) + m * n * size * (2 if case["beta"] else 1), "flops": 2 * m * n * k}
    s, l, n = case["s"], case["l"], case["count"]
    isz, osz = (2 if case["dtype"] == "bf16" else 4), (2 if case["out"] == "bf16" else 4)
    # the Gram matrix (symmetric), five steps on s x s matrices, one product with the block
    return {"bytes": n * s * l * (isz + osz * (2 if case["update"] else 1)),
            "flops": n * (s * (s + 1) * l + 17 * s * s * (s + 1) + 2 * s * s * l)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _activations(rows, cols, g):
    """Rows of different size and a hundredth of the columns ten times the others, as activations have."""
    x = _randn((rows, cols), g)
    x *= torch.exp2(torch.randint(-3, 4, (rows, 1), generator=g, device=DEV).float())
    x *= 1.0 + 9.0 * (torch.rand((1, cols), generator=g, device=DEV) < 0.01)
    return x


def _momentum(shape, g):
    x = _randn(shape, g)
    x *= 0.02 * (1.0 + 2.0 * (torch.rand(shape[-1], generator=g, device=DEV) < 0.01))
    return x


def _buffers(rows, cols, fmt):
    k = up(cols, 128)
    q = torch.zeros((rows, k), dtype=torch.uint8, device=DEV).view(FMT[fmt])
    s = torch.full((up(k // 128, 4) // 4, up(rows, 4), 4), 127, dtype=torch.uint8, device=DEV)
    return q, s


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    if case["op"] == "quantize":
        r, c = case["rows"], case["cols"]
        st["x"] = _activations(r, c, g).to(DT[case["dtype"]])
        st["q"], st["s"] = _buffers(r, c, case["fmt"]) if case["rows_out"] else (None, None)
        st["qt"], st["st"] = _buffers(c, r, case["fmt"]) if case["t_out"] else (None, None)
    elif case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        st["a"], st["sa"] = _plain_quantize(_activations(m, k, g).to(torch.bfloat16), case["fa"], 1)
        st["b"], st["sb"] = _plain_quantize((0.02 * _randn((n, k), g)).to(torch.bfloat16), "e4m3", 128 if not case["beta"] else 1)
        st["c"] = (_randn((m, n), g) if case["beta"] else torch.zeros((m, n), device=DEV)).to(DT[case["out"]])
        # a gradient's weight in the momentum, else the plain product
        st["alpha"] = 0.05 if case["beta"] else 1.0
        if own:
            import matrix_aware_optimizer_amd as mao
            need = mao.fp8_gemm_workspace_bytes(m, n, up(k, 128))
            st["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    else:
        n, s, l = case["count"], case["s"], case["l"]
        # tall: the blocks are columns of wider matrices, 12 to a matrix where that divides
        per = 12 if n % 12 == 0 else n
        if case["tall"]:
            mats = [_momentum((n // per, l, per * s), g).to(DT[case["dtype"]]),
                    (0.02 * _randn((n // per, l, per * s), g)).to(DT[case["out"]])]
            st["mw"] = mats
            st["blocks"] = [(mats[0][i].view(l, per, s).permute(1, 0, 2), mats[1][i].view(l, per, s).permute(1, 0, 2))
                            for i in range(n // per)]
        else:
            mats = [_momentum((n, s, l), g).to(DT[case["dtype"]]), (0.02 * _randn((n, s, l), g)).to(DT[case["out"]])]
            st["mw"] = mats
            st["blocks"] = [(mats[0], mats[1])]
        if own:
            import matrix_aware_optimizer_amd as mao
            how = dict(eta=ETA, decay=DECAY, scale=_scale(case)) if case["update"] else {}
            st["plan"] = mao.PreparedNSBlocks(st["blocks"], *QUINTIC, 5, **how)
    return st


# the update's step size, decay and scale (the root of the long side over the short one's matches the sizes of the blocks)
ETA, DECAY = 0.02, 0.1


def _scale(case):
    return 0.2 * math.sqrt(case["l"])


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_quantize(x, fmt, block):
    rows, cols = x.shape
    k = up(cols, 128)
    r = up(rows, block)
    p = torch.zeros((r, k), device=x.device)
    p[:rows, :cols] = x
    v = p.view(r // block, block, k // 128, 128)
    finite = torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v))
    amax = finite.amax(dim=(1, 3), keepdim=True)
    mant, e = torch.frexp(amax)                       # amax = mant 2^e, mant in [0.5, 1)
    e = e - (9 if fmt == "e4m3" else 16) + (mant > 0.875)   # 448 = 0.875 2^9, 57344 = 0.875 2^16
    e = torch.where(amax == 0, torch.zeros_like(e), e).clamp(-126, 127)
    q = torch.ldexp(v, -e).reshape(r, k)[:rows].to(FMT[fmt])
    byte = (e + 127).to(torch.uint8).expand(r // block, block, k // 128, 1).reshape(r, k // 128)[:rows]
    s = torch.full((up(k // 128, 4), up(rows, 4)), 127, dtype=torch.uint8, device=x.device)
    s[:k // 128, :rows] = byte.t()
    return q, s.view(-1, 4, up(rows, 4)).permute(0, 2, 1).contiguous()


def _bytes_per_row(s, rows, kb):
    """Scale bytes as [rows, K/128]."""
    return s.permute(0, 2, 1).reshape(-1, s.shape[1])[:kb, :rows].t()


def _values(q, s, dtype):
    rows, k = q.shape
    e = _bytes_per_row(s, rows, k // 128).to(torch.int32) - 127
    v = q.to(dtype).view(rows, k // 128, 128)
    return torch.ldexp(v, e.unsqueeze(2)).view(rows, k)


def _plain_gemm(st):
    a, b = _values(st["a"], st["sa"], torch.float32), _values(st["b"], st["sb"], torch.float32)
    out = st["alpha"] * torch.matmul(a, b.t())
    if st["case"]["beta"]:
        out = out + st["case"]["beta"] * st["c"].float()
    st["c"].copy_(out)
    return st["c"]


def _plain_heads(st):
    case = st["case"]
    a, b, c = QUINTIC
    m, w = st["mw"]
    x = m.float()
    if case["tall"]:                                  # [matrices, l, blocks * s] -> [matrices, blocks, s, l]
        x = x.view(*x.shape[:2], -1, case["s"]).permute(0, 2, 3, 1).contiguous()
    x = x / x.square().sum(dim=(-2, -1), keepdim=True).sqrt()
    for _ in range(5):
        gram = torch.matmul(x, x.transpose(-2, -1))
        x = a * x + torch.matmul(b * gram + c * torch.matmul(gram, gram), x)
    if case["tall"]:
        x = x.permute(0, 3, 1, 2).reshape(w.shape)
    if case["update"]:
        x = (1.0 - ETA * DECAY) * w.float() - (ETA * _scale(case)) * x
    w.copy_(x)
    return w


def run(st):
    case = st["case"]
    if own:
        import matrix_aware_optimizer_amd as mao
        if case["op"] == "quantize":
            mao.fp8_quantize(st["x"], st["q"], st["s"], st["qt"], st["st"], block_rows=case["block"])
            return {k: st[k] for k in ("q", "s", "qt", "st") if st[k] is not None}
        if case["op"] == "gemm":
            mao.fp8_gemm(st["a"], st["sa"], st["b"], st["sb"], st["c"], alpha=st["alpha"], beta=case["beta"], workspace=st["ws"])
            return st["c"]
        st["plan"]()
        return st["mw"][1]
    if case["op"] == "quantize":
        got = {}
        if case["rows_out"]:
            got["q"], got["s"] = _plain_quantize(st["x"], case["fmt"], case["block"])
        if case["t_out"]:
            got["qt"], got["st"] = _plain_quantize(st["x"].t(), case["fmt"], case["block"])
        return got
    return _plain_gemm(st) if case["op"] == "gemm" else _plain_heads(st)


# ---------------------------------------------------------------------------
# 64-bit values, from the definitions
# ---------------------------------------------------------------------------

def _exact_codes(x, fmt, block):
    """Values of the fp8 codes: each group's entries over its scale, rounded to the format's grid."""
    x = x.double()
    rows, cols = x.shape
    out = torch.zeros((rows, up(cols, 128)), dtype=torch.float64, device=x.device)
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    for j in range(0, cols, 128):
        part = x[:, j:j + 128]
        top = part.abs().amax(dim=1)
        if block > 1:
            top = torch.cat([top[i:i + block].max().expand(min(block, rows - i)) for i in range(0, rows, block)])
        e = torch.ceil(torch.log2(top / TOP[fmt])).clamp(min=-126)
        scale = torch.where(top == 0, torch.ones_like(top), torch.exp2(e)).unsqueeze(1)
        v = part / scale
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** low))) - bits)
        out[:, j:j + part.shape[1]] = torch.round(v / step) * step
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quantize":
        got = {}
        if case["rows_out"]:
            got.update(q=_exact_codes(st["x"], case["fmt"], case["block"]), s=None)
        if case["t_out"]:
            got.update(qt=_exact_codes(st["x"].t().contiguous(), case["fmt"], case["block"]), st=None)
        return got
    if case["op"] == "gemm":
        a, b = st["a"].double(), st["b"].double()
        kb = a.shape[1] // 128
        for v, s in ((a, st["sa"]), (b, st["sb"])):
            for j in range(kb):
                v[:, j * 128:(j + 1) * 128] *= 2.0 ** (s[j // 4, :v.shape[0], j % 4].double() - 127.0).unsqueeze(1)
        return st["alpha"] * (a @ b.t()) + case["beta"] * st["c"].double()
    a, b, c = QUINTIC
    eye = torch.eye(case["s"], dtype=torch.float64, device=DEV)
    outs = []
    for m, w in st["blocks"]:
        # y has the long side first; (a I + b G + c G G) from the right, G = y^T y
        y = m.double() if case["tall"] else m.double().transpose(1, 2).contiguous()
        y = y / torch.linalg.vector_norm(y, dim=(1, 2), keepdim=True)
        for _ in range(5):
            gram = y.transpose(1, 2).contiguous() @ y
            y = y @ (a * eye + gram @ (b * eye + c * gram))
        y = y if case["tall"] else y.transpose(1, 2)
        outs.append((1.0 - ETA * DECAY) * w.double() - ETA * _scale(case) * y if case["update"] else y)
    if not case["tall"]:
        return outs[0].contiguous()
    n, l, s = outs[0].shape
    return torch.stack([o.permute(1, 0, 2).reshape(l, n * s) for o in outs])
