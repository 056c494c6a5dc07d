"""ctypes binding of libmuon's C ABI (argument marshalling only).

Every function here has the name of the C entry point it calls, converts
torch tensors to (device pointer, dtype code, size) and the current HIP
stream, and raises :class:`MuonError` on a non-zero status.  No arithmetic
of the method happens in Python, and there is no fallback: if libmuon.so is
missing the first call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from typing import Optional, Sequence, Tuple, Union

import torch  # imported first so libmuon binds to the HIP runtime torch loaded

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG_DIR, "libmuon.so")

MUON_F32, MUON_BF16 = 0, 1
MUON_NS_PAD = 256
MUON_MAX_VOTERS = 1023
MUON_MAX_NUMEL = 1 << 38   # largest element count of the elementwise calls

_c_void_p, _c_int, _c_i64, _c_size, _c_float = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                                 ctypes.c_size_t, ctypes.c_float)


class MuonError(RuntimeError):
    """A libmuon call returned a non-zero status."""

    def __init__(self, name: str, status: int, text: str):
        super().__init__(f"{name} failed with status {status}: {text}")
        self.status = status


class NSProblem(ctypes.Structure):
    """Mirror of ``struct muon_ns_problem``."""

    _fields_ = [("M", _c_void_p), ("U", _c_void_p), ("sumsq", _c_void_p),
                ("rows", _c_i64), ("cols", _c_i64), ("m_dtype", ctypes.c_int32),
                ("u_dtype", ctypes.c_int32), ("bits", _c_void_p)]


# (name, restype, argtypes) of every exported symbol declared in include/muon.h
SIGNATURES = {
    "muon_status_string": (ctypes.c_char_p, [_c_int]),
    "muon_version": (_c_int, []),
    "muon_time_next_launch": (_c_int, [_c_void_p, _c_void_p]),
    "muon_momentum_workspace_bytes": (_c_size, [_c_i64, _c_int]),
    "muon_momentum": (_c_int, [_c_void_p, _c_int, _c_void_p, _c_int, _c_i64, _c_void_p, _c_int,
                               _c_float, _c_float, _c_void_p, _c_void_p, _c_size, _c_void_p]),
    "muon_momentum_noalloc": (_c_int, [_c_void_p, _c_int, _c_void_p, _c_int, _c_i64, _c_void_p, _c_int,
                                       _c_float, _c_float, _c_void_p, _c_void_p]),
    "ns_workspace_bytes": (_c_size, [ctypes.POINTER(NSProblem), _c_int, _c_int]),
    "ns_orthogonalize": (_c_int, [ctypes.POINTER(NSProblem), _c_int, _c_float, _c_float, _c_float,
                                  _c_int, _c_int, _c_void_p, _c_size, _c_void_p]),
    "ns_normalize": (_c_int, [_c_void_p, _c_int, _c_i64, _c_i64, _c_i64, _c_void_p, _c_void_p,
                              _c_int, _c_void_p]),
    "ns_stage_workspace_bytes": (_c_size, [_c_i64, _c_i64, _c_i64, _c_int]),
    "ns_gram": (_c_int, [_c_void_p, _c_void_p, _c_i64, _c_i64, _c_i64, _c_int, _c_void_p,
                         _c_void_p, _c_size, _c_void_p]),
    "ns_poly": (_c_int, [_c_void_p, _c_void_p, _c_i64, _c_i64, _c_float, _c_float, _c_int,
                         _c_void_p, _c_size, _c_void_p]),
    "ns_apply": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_i64, _c_i64, _c_i64,
                          _c_float, _c_float, _c_int, _c_void_p, _c_void_p, _c_size, _c_void_p]),
    "ns_apply_signs": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_i64, _c_i64,
                                _c_i64, _c_float, _c_float, _c_int, _c_void_p, _c_void_p, _c_size,
                                _c_void_p]),
    "ns_workspace_status": (_c_int, [_c_void_p, _c_size, _c_void_p]),
    "ns_residual_iterations": (_c_int, [_c_i64, _c_i64, _c_float, _c_float, _c_float, _c_int, _c_int]),
    "ns_bf16_min_side": (_c_int, []),
    "muon_set_split_wait_limit": (_c_int, [_c_int]),
    "muon_get_split_wait_limit": (_c_int, []),
    "sign_pack": (_c_int, [_c_void_p, _c_int, _c_i64, _c_void_p, _c_void_p]),
    "majority_vote": (_c_int, [_c_void_p, _c_int, _c_i64, _c_void_p, _c_void_p]),
    "apply_update": (_c_int, [_c_void_p, _c_int, _c_i64, _c_void_p, _c_float, _c_void_p]),
    "vote_and_update": (_c_int, [_c_void_p, _c_int, _c_i64, _c_void_p, _c_int, _c_float,
                                 _c_void_p]),
    "sign_int8": (_c_int, [_c_void_p, _c_int, _c_i64, _c_void_p, _c_void_p]),
    "sum_int8": (_c_int, [_c_void_p, _c_int, _c_i64, _c_void_p, _c_void_p]),
    "threshold_pack": (_c_int, [_c_void_p, _c_i64, _c_void_p, _c_void_p]),
    "unpack_signs": (_c_int, [_c_void_p, _c_i64, _c_void_p, _c_int, _c_void_p]),
    "apply_update_dense": (_c_int, [_c_void_p, _c_int, _c_i64, _c_void_p, _c_int, _c_float, _c_void_p]),
    "dion_workspace_bytes": (_c_size, [ctypes.c_void_p, _c_int, _c_int]),
    "dion_step": (_c_int, [ctypes.c_void_p, _c_int, _c_int, _c_float, _c_float, _c_void_p, _c_size,
                           _c_void_p]),
    "fp8_scale_bytes": (_c_size, [_c_i64, _c_i64]),
    "fp8_quantize": (_c_int, [_c_void_p, _c_int, _c_i64, _c_i64, _c_i64, _c_int, _c_int, _c_void_p, _c_i64,
                              _c_void_p, _c_void_p, _c_i64, _c_void_p, _c_void_p]),
    "fp8_gemm_workspace_bytes": (_c_size, [_c_i64, _c_i64, _c_i64]),
    "fp8_gemm": (_c_int, [_c_void_p, _c_int, _c_i64, _c_void_p, _c_void_p, _c_int, _c_i64, _c_void_p, _c_void_p,
                          _c_int, _c_i64, _c_i64, _c_i64, _c_i64, _c_float, _c_float, _c_void_p, _c_size,
                          _c_void_p]),
    "ns_blocks_workspace_bytes": (_c_size, [_c_void_p, _c_int]),
    "ns_blocks": (_c_int, [_c_void_p, _c_int, _c_float, _c_float, _c_float, _c_int, _c_void_p, _c_size, _c_void_p]),
    "ns_blocks_update": (_c_int, [_c_void_p, _c_int, _c_float, _c_float, _c_float, _c_int, _c_float, _c_float,
                                  _c_float, _c_void_p, _c_size, _c_void_p]),
    "int8_quantize": (_c_int, [_c_void_p, _c_int, _c_i64, _c_i64, _c_i64, _c_void_p, _c_i64, _c_void_p, _c_void_p]),
    "int8_gemm_workspace_bytes": (_c_size, [_c_i64, _c_i64, _c_i64]),
    "int8_gemm": (_c_int, [_c_void_p, _c_i64, _c_void_p, _c_void_p, _c_i64, _c_void_p, _c_void_p, _c_int, _c_i64,
                           _c_i64, _c_i64, _c_i64, _c_void_p, _c_size, _c_void_p]),
    "int8_glu_workspace_bytes": (_c_size, [_c_i64, _c_i64, _c_i64]),
    "int8_glu": (_c_int, [_c_void_p, _c_i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_i64, _c_int,
                          _c_void_p, _c_int, _c_i64, _c_i64, _c_i64, _c_i64, _c_void_p, _c_size, _c_void_p]),
    "glu_forward_workspace_bytes": (_c_size, [_c_i64, _c_i64, _c_i64]),
    "glu_forward": (_c_int, [_c_void_p, _c_i64, _c_void_p, _c_void_p, _c_i64, _c_int, _c_void_p, _c_i64, _c_void_p,
                             _c_void_p, _c_i64, _c_i64, _c_i64, _c_i64, _c_void_p, _c_size, _c_void_p]),
    "glu_backward_workspace_bytes": (_c_size, [_c_i64, _c_i64, _c_i64]),
    "glu_backward": (_c_int, [_c_void_p, _c_i64, _c_void_p, _c_void_p, _c_i64, _c_int, _c_void_p, _c_void_p, _c_i64,
                              _c_void_p, _c_i64, _c_void_p, _c_void_p, _c_i64, _c_void_p, _c_i64, _c_i64, _c_i64,
                              _c_i64, _c_void_p, _c_size, _c_void_p]),
    "glu_weight_grad_workspace_bytes": (_c_size, [_c_i64, _c_i64, _c_i64]),
    "glu_weight_grad": (_c_int, [_c_void_p, _c_void_p, _c_i64, _c_void_p, _c_i64, _c_void_p, _c_void_p, _c_int, _c_i64,
                                 _c_i64, _c_i64, _c_i64, _c_float, _c_float, _c_void_p, _c_size, _c_void_p]),
}

_LIB: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """Load libmuon.so (once).  Raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m matrix_aware_optimizer_amd.build` "
                "(there is no fallback implementation)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = handle
    return _LIB


def status_string(status: int) -> str:
    return lib().muon_status_string(status).decode()


def _check(name: str, status: int) -> None:
    if status != 0:
        raise MuonError(name, status, status_string(status))


def dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MUON_F32
    if t.dtype == torch.bfloat16:
        return MUON_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def precision_code(p: Union[str, int]) -> int:
    if isinstance(p, int):
        return p
    return {"f32": MUON_F32, "fp32": MUON_F32, "float32": MUON_F32,
            "bf16": MUON_BF16, "bfloat16": MUON_BF16}[p]


def _dev(t: Optional[torch.Tensor], name: str) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


# the current stream's handle without building a Stream object (2 us of a call's host time)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _workspace(nbytes: int, like: torch.Tensor, workspace: Optional[torch.Tensor]) -> torch.Tensor:
    if workspace is not None:
        return workspace
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=like.device)


def _allocating_on(stream, like: torch.Tensor):
    """Context in which torch allocates from ``stream``'s own pool (None: the current stream's) and fills memory on it."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        # handle 0 is the default stream; an ExternalStream of 0 would be a new stream of torch's
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle, device=like.device) if handle else torch.cuda.default_stream(like.device)
    return torch.cuda.stream(stream)


def _workspace_on(nbytes: int, like: torch.Tensor, workspace: Optional[torch.Tensor], stream) -> torch.Tensor:
    """As _workspace, for a call that goes to ``stream``: memory of that stream's own pool, so that it is free
    when the call begins there and is not given to another stream's work while the call runs."""
    if workspace is not None or stream is None:
        return _workspace(nbytes, like, workspace)
    with _allocating_on(stream, like):
        return _workspace(nbytes, like, None)


# ---------------------------------------------------------------------------
# a1
# ---------------------------------------------------------------------------

def muon_momentum_workspace_bytes(numel: int, nseg: int) -> int:
    return int(lib().muon_momentum_workspace_bytes(numel, nseg))


def muon_momentum(M: torch.Tensor, G: torch.Tensor, beta: float, alpha: float,
                  seg_offsets: Optional[torch.Tensor] = None,
                  sumsq_out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """``M <- beta*M + alpha*G`` in place; optional per-matrix sum of squares."""
    if M.numel() != G.numel():
        raise ValueError("M and G must have the same number of entries")
    nseg, ws_ptr, ws_bytes = 0, None, 0
    if sumsq_out is not None:
        if seg_offsets is None:
            raise ValueError("seg_offsets is required with sumsq_out")
        nseg = seg_offsets.numel() - 1
        need = muon_momentum_workspace_bytes(M.numel(), nseg)
        workspace = _workspace_on(need, M, workspace, stream)
        ws_ptr, ws_bytes = _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()
    _check("muon_momentum", lib().muon_momentum(
        _dev(M, "M"), dtype_code(M), _dev(G, "G"), dtype_code(G), M.numel(),
        _dev(seg_offsets, "seg_offsets") if sumsq_out is not None else None, nseg,
        float(beta), float(alpha), _dev(sumsq_out, "sumsq_out"), ws_ptr, ws_bytes, _stream(stream)))


def muon_momentum_noalloc(M: torch.Tensor, G: torch.Tensor, beta: float, alpha: float,
                          seg_offsets: Optional[torch.Tensor] = None,
                          sumsq_out: Optional[torch.Tensor] = None, stream=None) -> None:
    """muon_momentum without a workspace: the library's fixed per-device scratch holds
    the partial sums (nothing is allocated here or in the library).  Calls that overlap
    on one device race."""
    if M.numel() != G.numel():
        raise ValueError("M and G must have the same number of entries")
    nseg = 0
    if sumsq_out is not None:
        if seg_offsets is None:
            raise ValueError("seg_offsets is required with sumsq_out")
        nseg = seg_offsets.numel() - 1
    _check("muon_momentum_noalloc", lib().muon_momentum_noalloc(
        _dev(M, "M"), dtype_code(M), _dev(G, "G"), dtype_code(G), M.numel(),
        _dev(seg_offsets, "seg_offsets") if sumsq_out is not None else None, nseg,
        float(beta), float(alpha), _dev(sumsq_out, "sumsq_out"), _stream(stream)))


# ---------------------------------------------------------------------------
# a2-a5
# ---------------------------------------------------------------------------

# (M, U, sumsq) or (M, U, sumsq, bits); U may be None when bits are given and
# the signs are fused (bf16, wide, cols % 64 == 0, steps > 0)
ProblemLike = Tuple[torch.Tensor, ...]


def _problems(problems: Sequence[ProblemLike]):
    arr = (NSProblem * len(problems))()
    for i, prob in enumerate(problems):
        M, U, sumsq = prob[:3]
        bits = prob[3] if len(prob) > 3 else None
        if M.dim() != 2 or (U is not None and U.shape != M.shape):
            raise ValueError("each problem needs a 2-D M and a U of the same shape")
        if bits is not None and (bits.element_size() != 8 or bits.numel() < packed_words(M.numel())):
            raise ValueError("bits must hold ceil(rows * cols / 64) 64-bit words")
        arr[i].M = _dev(M, "M")
        arr[i].U = _dev(U, "U")
        arr[i].sumsq = _dev(sumsq, "sumsq") if sumsq is not None else None
        arr[i].bits = _dev(bits, "bits")
        arr[i].rows, arr[i].cols = M.shape
        arr[i].m_dtype = dtype_code(M)
        arr[i].u_dtype = dtype_code(U) if U is not None else dtype_code(M)
    return arr


def ns_workspace_bytes(problems: Sequence[ProblemLike], precision="bf16") -> int:
    arr = _problems(problems)
    return int(lib().ns_workspace_bytes(arr, len(problems), precision_code(precision)))


def ns_orthogonalize(problems: Sequence[ProblemLike], a: float, b: float, c: float, steps: int,
                     precision="bf16", workspace: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    """Polar directions of every (M, U, sumsq-or-None) problem, written into U."""
    if len(problems) == 0:
        return
    arr = _problems(problems)
    prec = precision_code(precision)
    need = int(lib().ns_workspace_bytes(arr, len(problems), prec))
    workspace = _workspace_on(need, problems[0][0], workspace, stream)
    _check("ns_orthogonalize", lib().ns_orthogonalize(
        arr, len(problems), float(a), float(b), float(c), int(steps), prec,
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _stream(stream)))


class PreparedNS:
    """One ns_orthogonalize call whose problem array is marshalled once.

    For a caller that orthogonalises the same device buffers every step (a
    parameter set's momentum, directions and sign words): building the ctypes
    array of a layer set costs the host hundreds of microseconds, long enough
    to leave the GPU idle between the momentum and the first product.  Calling
    the object only enqueues the work, on ``stream`` (default: the current one)."""

    def __init__(self, problems: Sequence[ProblemLike], a: float, b: float, c: float, steps: int,
                 precision="bf16", workspace: Optional[torch.Tensor] = None):
        if len(problems) == 0:
            raise ValueError("no problems")
        self._problems = list(problems)     # keeps the tensors alive
        self._arr = _problems(self._problems)
        self._n = len(self._problems)
        prec = precision_code(precision)
        self._args = (float(a), float(b), float(c), int(steps), prec)
        need = int(lib().ns_workspace_bytes(self._arr, self._n, prec))
        self.workspace = _workspace(need, self._problems[0][0], workspace)
        self._ws = (_dev(self.workspace, "workspace"), self.workspace.numel() * self.workspace.element_size())
        if self._ws[1] < need:
            raise ValueError(f"workspace holds {self._ws[1]} bytes, the call needs {need}")

    def __call__(self, stream=None) -> None:
        _check("ns_orthogonalize", lib().ns_orthogonalize(self._arr, self._n, *self._args, *self._ws,
                                                          _stream(stream)))


def _batch3(t: torch.Tensor) -> Tuple[int, int, int]:
    if t.dim() == 2:
        return 1, t.shape[0], t.shape[1]
    if t.dim() == 3:
        return t.shape[0], t.shape[1], t.shape[2]
    raise ValueError("expected a 2-D or 3-D tensor")


def ns_normalize(M: torch.Tensor, sumsq: torch.Tensor, X0: torch.Tensor, precision="bf16",
                 stream=None) -> None:
    batch, rows, cols = _batch3(M)
    _check("ns_normalize", lib().ns_normalize(
        _dev(M, "M"), dtype_code(M), rows, cols, batch, _dev(sumsq, "sumsq"), _dev(X0, "X0"),
        precision_code(precision), _stream(stream)))


def ns_stage_workspace_bytes(s: int, l: int, batch: int = 1, precision="bf16") -> int:
    return int(lib().ns_stage_workspace_bytes(s, l, batch, precision_code(precision)))


def new_stage_workspace(s: int, l: int, batch: int = 1, precision="bf16", device=None) -> torch.Tensor:
    """Zeroed workspace for the stage calls on [batch][s][l] (its counters start at zero).
    At least the 1024-byte counter block, so that ns_workspace_status can read its
    error word also when nothing splits."""
    n = ns_stage_workspace_bytes(s, l, batch, precision)
    return torch.zeros(max(n, 1024), dtype=torch.uint8, device=device or "cuda")


def _stage_ws(workspace, split: bool, s: int, l: int, batch: int, precision, like: torch.Tensor, stream):
    """(pointer, bytes) of the stage workspace: the caller's, a fresh zeroed one, or none."""
    if not split:
        return None, 0
    if workspace is None:
        with _allocating_on(stream, like):
            workspace = new_stage_workspace(s, l, batch, precision, like.device)
    return _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()


def ns_gram(X: torch.Tensor, A: torch.Tensor, precision="bf16", stream=None,
            sumsq: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
            split: bool = True) -> None:
    """A = X X^T, or M M^T / sumsq with the raw momentum as X.  With split
    (the default) the work is split as ns_orthogonalize splits it, in
    `workspace` (from new_stage_workspace) or a fresh one."""
    batch, s, l = _batch3(X)
    ws, nbytes = _stage_ws(workspace, split, s, l, batch, precision, X, stream)
    _check("ns_gram", lib().ns_gram(_dev(X, "X"), _dev(A, "A"), s, l, batch,
                                    precision_code(precision), _dev(sumsq, "sumsq"), ws, nbytes,
                                    _stream(stream)))


def ns_poly(A: torch.Tensor, B: torch.Tensor, b: float, c: float, precision="bf16",
            stream=None, workspace: Optional[torch.Tensor] = None, split: bool = True) -> None:
    """B = b A + c A A."""
    batch, s, _ = _batch3(A)
    ws, nbytes = _stage_ws(workspace, split, s, s, batch, precision, A, stream)
    _check("ns_poly", lib().ns_poly(_dev(A, "A"), _dev(B, "B"), s, batch, float(b), float(c),
                                    precision_code(precision), ws, nbytes, _stream(stream)))


def ns_apply(B: torch.Tensor, X: torch.Tensor, Xout: torch.Tensor, a: float, alpha: float = 1.0,
             precision="bf16", stream=None, sumsq: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None, split: bool = True,
             X_lo: Optional[torch.Tensor] = None, Xout_lo: Optional[torch.Tensor] = None) -> None:
    """Xout = a X + alpha B X, or (a M + alpha B M) / sqrt(sumsq) with the raw momentum as X.
    With ``X_lo`` the addend is a (X + X_lo); ``Xout_lo`` receives the bf16 rounding
    residual of Xout (bf16 only; the two may be one tensor)."""
    batch, s, l = _batch3(X)
    ws, nbytes = _stage_ws(workspace, split, s, l, batch, precision, X, stream)
    _check("ns_apply", lib().ns_apply(_dev(B, "B"), _dev(X, "X"), _dev(X_lo, "X_lo"), _dev(Xout, "Xout"),
                                      _dev(Xout_lo, "Xout_lo"), s, l, batch, float(a), float(alpha),
                                      precision_code(precision), _dev(sumsq, "sumsq"), ws, nbytes,
                                      _stream(stream)))


def ns_apply_signs(B: torch.Tensor, X: torch.Tensor, Xout: Optional[torch.Tensor], bits: torch.Tensor,
                   a: float, alpha: float = 1.0, precision="bf16", stream=None,
                   sumsq: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   split: bool = True, X_lo: Optional[torch.Tensor] = None) -> None:
    """ns_apply that also packs the signs of Xout into ``bits`` ([batch][s*l/64] words);
    with Xout None only the signs are written."""
    batch, s, l = _batch3(X)
    if bits.element_size() != 8 or bits.numel() < batch * (s * l // 64):
        raise ValueError("bits must hold batch * s * l / 64 64-bit words")
    ws, nbytes = _stage_ws(workspace, split, s, l, batch, precision, X, stream)
    _check("ns_apply_signs", lib().ns_apply_signs(
        _dev(B, "B"), _dev(X, "X"), _dev(X_lo, "X_lo"), _dev(Xout, "Xout"), _dev(bits, "bits"), s, l,
        batch, float(a), float(alpha), precision_code(precision), _dev(sumsq, "sumsq"), ws, nbytes,
        _stream(stream)))


def ns_workspace_status(workspace: torch.Tensor, stream=None) -> None:
    """Synchronise ``stream`` and raise MuonError (MUON_ESPLIT) if a split product that
    used ``workspace`` gave up waiting for its other half (its tile was not written)."""
    _check("ns_workspace_status", lib().ns_workspace_status(
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(), _stream(stream)))


def ns_residual_iterations(rows: int, cols: int, a: float, b: float, c: float, steps: int,
                           precision="bf16") -> int:
    """How many leading iterations of ns_orthogonalize keep the bf16 residual of their output."""
    k = int(lib().ns_residual_iterations(rows, cols, float(a), float(b), float(c), int(steps),
                                         precision_code(precision)))
    if k < 0:
        _check("ns_residual_iterations", k)
    return k


def ns_bf16_min_side() -> int:
    """The shortest short side that ns_orthogonalize runs on bf16 products (smaller
    problems asked for bf16 run on the fp32 products)."""
    return int(lib().ns_bf16_min_side())


def set_split_wait_limit(polls: int) -> int:
    """Set the polls a split product's second half waits for the first (process-wide);
    returns the previous limit."""
    prev = int(lib().muon_get_split_wait_limit())
    _check("muon_set_split_wait_limit", lib().muon_set_split_wait_limit(int(polls)))
    return prev


# ---------------------------------------------------------------------------
# a6-a8
# ---------------------------------------------------------------------------

def packed_words(numel: int) -> int:
    return (numel + 63) // 64


def sign_pack(U: torch.Tensor, bits: torch.Tensor, stream=None) -> None:
    """Pack the signs of U (flat) into ``bits`` (int64/uint64, ceil(numel/64) words)."""
    if bits.numel() < packed_words(U.numel()) or bits.element_size() != 8:
        raise ValueError("bits must hold ceil(numel/64) 64-bit words")
    _check("sign_pack", lib().sign_pack(_dev(U, "U"), dtype_code(U), U.numel(), _dev(bits, "bits"),
                                        _stream(stream)))


def majority_vote(bits: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """Vote over the rows of ``bits`` ([M, nwords] 64-bit words) into ``out`` ([nwords])."""
    if bits.dim() != 2 or bits.element_size() != 8 or out.numel() < bits.shape[1]:
        raise ValueError("bits must be [M, nwords] 64-bit words and out hold nwords")
    _check("majority_vote", lib().majority_vote(_dev(bits, "bits"), bits.shape[0], bits.shape[1],
                                                _dev(out, "out"), _stream(stream)))


def apply_update(W: torch.Tensor, vote_bits: torch.Tensor, eta: float, stream=None) -> None:
    if vote_bits.numel() < packed_words(W.numel()) or vote_bits.element_size() != 8:
        raise ValueError("vote_bits must hold ceil(numel/64) 64-bit words")
    _check("apply_update", lib().apply_update(_dev(W, "W"), dtype_code(W), W.numel(),
                                              _dev(vote_bits, "vote_bits"), float(eta),
                                              _stream(stream)))


def vote_and_update(W: torch.Tensor, bits: torch.Tensor, eta: float, stream=None) -> None:
    if bits.dim() != 2 or bits.element_size() != 8 or bits.shape[1] != packed_words(W.numel()):
        raise ValueError("bits must be [M, ceil(numel/64)] 64-bit words")
    _check("vote_and_update", lib().vote_and_update(_dev(W, "W"), dtype_code(W), W.numel(),
                                                    _dev(bits, "bits"), bits.shape[0], float(eta),
                                                    _stream(stream)))


def muon_version() -> int:
    return int(lib().muon_version())


def time_next_launch(start: Optional[torch.cuda.Event], stop: Optional[torch.cuda.Event]) -> None:
    """Make the next kernel this thread launches through the library record ``start`` and
    ``stop`` (torch timing events) at its own start and end.  Each event must have been
    recorded once already (torch creates the underlying HIP event on its first record)."""
    handles = []
    for ev in (start, stop):
        if ev is None:
            handles.append(None)
            continue
        h = ev.cuda_event
        if not h:
            raise ValueError("record the event once before passing it (the HIP event is created lazily)")
        handles.append(h)
    _check("muon_time_next_launch", lib().muon_time_next_launch(handles[0], handles[1]))


# ---------------------------------------------------------------------------
# int8 exchange format
# ---------------------------------------------------------------------------

MUON_INT8_MAX_VOTERS = 127


def _int8(t: torch.Tensor, name: str) -> int:
    if t.dtype != torch.int8:
        raise TypeError(f"{name} must be an int8 tensor")
    return _dev(t, name)


def sign_int8(U: torch.Tensor, S: torch.Tensor, stream=None) -> None:
    """S[i] = +1 if !(U[i] < 0) else -1 (int8)."""
    if S.numel() < U.numel():
        raise ValueError("S needs one int8 per entry of U")
    _check("sign_int8", lib().sign_int8(_dev(U, "U"), dtype_code(U), U.numel(), _int8(S, "S"),
                                        _stream(stream)))


def sum_int8(S: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """out = sum over the rows of S ([M, n] int8), as the SUM all-reduce delivers it."""
    if S.dim() != 2 or out.numel() < S.shape[1]:
        raise ValueError("S must be [M, n] and out hold n entries")
    _check("sum_int8", lib().sum_int8(_int8(S, "S"), S.shape[0], S.shape[1], _int8(out, "out"),
                                      _stream(stream)))


def threshold_pack(total: torch.Tensor, bits: torch.Tensor, stream=None) -> None:
    """Packed vote bits: bit i = 1 iff total[i] >= 0."""
    if bits.numel() < packed_words(total.numel()):
        raise ValueError("bits too small")
    _check("threshold_pack", lib().threshold_pack(_int8(total, "sum"), total.numel(),
                                                  _dev(bits, "bits"), _stream(stream)))


# ---------------------------------------------------------------------------
# local re-orthogonalisation of the vote
# ---------------------------------------------------------------------------

def unpack_signs(vote_bits: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """out[i] = +1 if vote bit i is set, else -1 (bf16 or fp32)."""
    if vote_bits.numel() < packed_words(out.numel()):
        raise ValueError("vote_bits too small")
    _check("unpack_signs", lib().unpack_signs(_dev(vote_bits, "vote_bits"), out.numel(), _dev(out, "out"),
                                              dtype_code(out), _stream(stream)))


def apply_update_dense(W: torch.Tensor, U: torch.Tensor, eta: float, stream=None) -> None:
    """W <- W - eta * U (one rounding in fp64, then to W's type)."""
    if U.numel() != W.numel():
        raise ValueError("W and U differ in size")
    _check("apply_update_dense", lib().apply_update_dense(_dev(W, "W"), dtype_code(W), W.numel(),
                                                          _dev(U, "U"), dtype_code(U), float(eta),
                                                          _stream(stream)))


# ---------------------------------------------------------------------------
# Dion
# ---------------------------------------------------------------------------

MUON_DION_MAX_RANK = 192


class DionProblem(ctypes.Structure):
    _fields_ = [("M", _c_void_p), ("G", _c_void_p), ("X", _c_void_p), ("Q", _c_void_p),
                ("rows", _c_i64), ("cols", _c_i64)]


def _dion_problems(problems):
    arr = (DionProblem * len(problems))()
    for i, (M, G, X, Q) in enumerate(problems):
        for name, t in (("M", M), ("G", G), ("X", X), ("Q", Q)):
            if t.dtype != torch.float32:
                raise TypeError(f"Dion tensors are fp32 ({name})")
        if M.dim() != 2 or G.shape != M.shape or X.shape != M.shape or Q.dim() != 2 or Q.shape[0] != M.shape[1]:
            raise ValueError("Dion problem shapes: M, G, X m x n and Q n x rank")
        arr[i].M, arr[i].G, arr[i].X, arr[i].Q = (_dev(M, "M"), _dev(G, "G"), _dev(X, "X"), _dev(Q, "Q"))
        arr[i].rows, arr[i].cols = M.shape
    return arr


def dion_workspace_bytes(problems, rank: int) -> int:
    arr = _dion_problems(problems)
    return int(lib().dion_workspace_bytes(ctypes.cast(arr, ctypes.c_void_p), len(problems), int(rank)))


def dion_step(problems, rank: int, mu: float, eta: float, workspace: Optional[torch.Tensor] = None,
              stream=None) -> None:
    """One Dion step on every (M, G, X, Q) problem (fp32 tensors; M, X, Q updated in place)."""
    if not problems:
        return
    arr = _dion_problems(problems)
    nbytes = int(lib().dion_workspace_bytes(ctypes.cast(arr, ctypes.c_void_p), len(problems), int(rank)))
    ws = _workspace_on(nbytes, problems[0][0], workspace, stream)
    _check("dion_step", lib().dion_step(ctypes.cast(arr, ctypes.c_void_p), len(problems), int(rank),
                                        float(mu), float(eta), _dev(ws, "workspace"),
                                        ws.numel() * ws.element_size(), _stream(stream)))


# ---------------------------------------------------------------------------
# fp8 matrices with a scale for each block of 128
# ---------------------------------------------------------------------------

MUON_FP8_GROUP = 128
MUON_FP8_MAX_SIDE = 4194240
_FP8 = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}
_FP8_BY_NAME = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def _ceil_to(n: int, m: int) -> int:
    return -(-n // m) * m


@functools.lru_cache(maxsize=1024)
def fp8_scale_shape(rows: int, cols: int) -> Tuple[int, int, int]:
    """Shape of the scale bytes of a rows x cols matrix: [words of four groups][rows][4]."""
    return _ceil_to(cols, 4 * MUON_FP8_GROUP) // (4 * MUON_FP8_GROUP), _ceil_to(rows, 4), 4


def fp8_buffers(rows: int, cols: int, fmt: str = "e4m3", device="cuda") -> Tuple[torch.Tensor, torch.Tensor]:
    """Uninitialised (codes [rows, cols rounded up to 128], scales) for a rows x cols matrix."""
    q = torch.empty((rows, _ceil_to(cols, MUON_FP8_GROUP)), dtype=_FP8_BY_NAME[fmt], device=device)
    return q, torch.empty(fp8_scale_shape(rows, cols), dtype=torch.uint8, device=device)


def _rows2(t: torch.Tensor, name: str) -> Tuple[int, int]:
    """(pointer, row pitch) of a 2-D device tensor whose rows are contiguous."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D with contiguous rows")
    rows, cols = t.shape
    pitch, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name} must be 2-D with contiguous rows")
    if rows <= 1 or cols == 0:
        return t.data_ptr(), max(cols, 1)
    if pitch < cols:
        raise ValueError(f"{name} must not overlap itself")
    return t.data_ptr(), pitch


def _fp8_operand(q: torch.Tensor, s: torch.Tensor, rows: int, cols: int, name: str):
    """(codes, pitch, scales, format code) of an fp8 matrix that holds rows x cols."""
    fmt = _FP8.get(q.dtype)
    if fmt is None:
        raise TypeError(f"{name} must be float8_e4m3fn or float8_e5m2")
    ptr, ld = _rows2(q, name)
    held, width = q.shape
    if held != rows or width < _ceil_to(cols, MUON_FP8_GROUP):
        raise ValueError(f"{name} must hold {rows} rows of at least {_ceil_to(cols, MUON_FP8_GROUP)} codes")
    if s.dtype != torch.uint8 or s.shape != fp8_scale_shape(rows, cols):
        raise ValueError(f"the scales of {name} must be uint8 of shape {fp8_scale_shape(rows, cols)}")
    if rows <= 1 or cols == 0:      # no second row: the pitch is not used, the library wants a multiple of 16
        ld = _ceil_to(width, 16)
    return ptr, ld, _dev(s, name), fmt


def fp8_quantize(x: torch.Tensor, q: Optional[torch.Tensor], s: Optional[torch.Tensor],
                 qt: Optional[torch.Tensor] = None, st: Optional[torch.Tensor] = None, block_rows: int = 1,
                 stream=None) -> None:
    """Codes and scales of ``x`` into (q, s), and those of its transpose into (qt, st); either may be None.

    ``block_rows`` 1: a scale for each row's group of 128 columns; 128: one for each 128 x 128 block."""
    if (q is None) != (s is None) or (qt is None) != (st is None) or (q is None and qt is None):
        raise ValueError("give (q, s), (qt, st) or both")
    xp, ldx = _rows2(x, "x")
    rows, cols = x.shape
    if q is not None and qt is not None and q.dtype != qt.dtype:
        raise TypeError("q and qt must have one format")
    qp = _fp8_operand(q, s, rows, cols, "q") if q is not None else (None, 0, None, 0)
    tp = _fp8_operand(qt, st, cols, rows, "qt") if qt is not None else (None, 0, None, 0)
    fmt = qp[3] if q is not None else tp[3]
    _check("fp8_quantize", lib().fp8_quantize(xp, dtype_code(x), rows, cols, max(ldx, cols), fmt, int(block_rows),
                                              qp[0], qp[1], qp[2], tp[0], tp[1], tp[2], _stream(stream)))


@functools.lru_cache(maxsize=1024)
def fp8_gemm_workspace_bytes(m: int, n: int, K: int) -> int:
    return int(lib().fp8_gemm_workspace_bytes(m, n, K))


def fp8_gemm(A: torch.Tensor, sa: torch.Tensor, B: torch.Tensor, sb: torch.Tensor, C: torch.Tensor,
             alpha: float = 1.0, beta: float = 0.0, workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """``C <- beta C + alpha A B^T`` for fp8 operands (codes, scales) with K = ``A.shape[1]`` columns."""
    m, K = A.shape
    n, kb = B.shape
    if kb != K or C.shape != (m, n):
        raise ValueError("A is m x K, B n x K and C m x n")
    ap, lda, sap, fa = _fp8_operand(A, sa, m, K, "A")
    bp, ldb, sbp, fb = _fp8_operand(B, sb, n, K, "B")
    cp, ldc = _rows2(C, "C")
    need = fp8_gemm_workspace_bytes(m, n, K)
    ws, nbytes = None, 0
    if need > 0:
        workspace = _workspace_on(need, C, workspace, stream)
        ws, nbytes = _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()
    status = lib().fp8_gemm(ap, fa, lda, sap, bp, fb, ldb, sbp, cp, dtype_code(C), ldc if ldc > n else n, m, n, K,
                            alpha, beta, ws, nbytes, _stream(stream))
    if status:
        _check("fp8_gemm", status)


# ---------------------------------------------------------------------------
# Newton-Schulz on many small blocks (attention heads)
# ---------------------------------------------------------------------------

MUON_BLOCKS_MAX_SHORT = 128


class BlockProblem(ctypes.Structure):
    """Mirror of ``struct muon_block_problem``."""

    _fields_ = [("M", _c_void_p), ("out", _c_void_p), ("rows", _c_i64), ("cols", _c_i64), ("count", _c_i64),
                ("ld_m", _c_i64), ("stride_m", _c_i64), ("ld_out", _c_i64), ("stride_out", _c_i64),
                ("m_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


def _block_view(t: torch.Tensor, name: str):
    """(pointer, count, rows, cols, row pitch, block stride) of a 2-D or 3-D view with contiguous rows."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() == 2:
        t = t.unsqueeze(0)
    if t.dim() != 3 or (t.shape[2] > 1 and t.stride(2) != 1):
        raise ValueError(f"{name} must be [count, rows, cols] (or [rows, cols]) with contiguous rows")
    count, rows, cols = t.shape
    return t.data_ptr(), count, rows, cols, t.stride(1) if rows > 1 else max(cols, 1), t.stride(0) if count > 1 else 0


def _block_problems(problems):
    arr = (BlockProblem * len(problems))()
    for i, (M, out) in enumerate(problems):
        if M.shape != out.shape:
            raise ValueError("each problem needs an M and an output of the same shape")
        mp, count, rows, cols, ld_m, stride_m = _block_view(M, "M")
        op, _, _, _, ld_o, stride_o = _block_view(out, "out")
        arr[i] = BlockProblem(mp, op, rows, cols, count, ld_m, stride_m, ld_o, stride_o, dtype_code(M), dtype_code(out))
    return arr


def ns_blocks_workspace_bytes(problems) -> int:
    arr = _block_problems(problems)
    return int(lib().ns_blocks_workspace_bytes(ctypes.cast(arr, _c_void_p), len(problems)))


class PreparedNSBlocks:
    """One ns_blocks or ns_blocks_update call whose problem array is marshalled once.

    ``problems``: (M, out) pairs of strided views [count, rows, cols] (or [rows, cols]).  Without
    ``eta`` the directions are written to ``out``; with it ``out <- (1 - eta decay) out - eta scale U``.
    Calling the object only enqueues the work, on ``stream`` (default: the current one), with a workspace
    of that stream's own memory, kept for its later calls, or ``workspace`` on every stream.  Steps and
    coefficients that the library refuses (too many steps for fp64) raise at construction."""

    def __init__(self, problems, a: float, b: float, c: float, steps: int, eta: Optional[float] = None,
                 decay: float = 0.0, scale: float = 1.0, workspace: Optional[torch.Tensor] = None):
        if len(problems) == 0:
            raise ValueError("no problems")
        self._name = "ns_blocks" if eta is None else "ns_blocks_update"
        self._fn = getattr(lib(), self._name)
        how = (float(a), float(b), float(c), int(steps))
        if eta is not None:
            how += (float(eta), float(decay), float(scale))
        _check(self._name, self._fn(None, 0, *how, None, 0, None))     # no problems: only the numbers are looked at
        self._problems = list(problems)     # keeps the tensors alive
        self._arr = _block_problems(self._problems)
        self._ptr = ctypes.cast(self._arr, _c_void_p)
        self._need = int(lib().ns_blocks_workspace_bytes(self._ptr, len(self._problems)))
        self.workspace = _workspace(self._need, self._problems[0][0], workspace)
        self._given = workspace is not None
        self._by_stream = {_stream(None): self._entry(self.workspace)}
        self._args = (self._ptr, len(self._problems), *how)

    @staticmethod
    def _entry(ws: torch.Tensor):
        return ws, _dev(ws, "workspace"), ws.numel() * ws.element_size()

    def __call__(self, stream=None) -> None:
        handle = _stream(stream)
        entry = self._by_stream.get(handle)
        if entry is None:
            # the first call on this stream: memory that is free there (another stream's may still be in use)
            entry = self._by_stream[handle] = self._entry(
                self.workspace if self._given else _workspace_on(self._need, self._problems[0][0], None, stream))
        _check(self._name, self._fn(*self._args, entry[1], entry[2], handle))


def ns_blocks(problems, a: float, b: float, c: float, steps: int, workspace: Optional[torch.Tensor] = None,
              stream=None) -> None:
    """Newton-Schulz directions of every block of every (M, U) problem, each block by itself."""
    if len(problems) > 0:
        workspace = _workspace_on(ns_blocks_workspace_bytes(problems), problems[0][0], workspace, stream)
        PreparedNSBlocks(problems, a, b, c, steps, workspace=workspace)(stream)


def ns_blocks_update(problems, a: float, b: float, c: float, steps: int, eta: float, decay: float = 0.0,
                     scale: float = 1.0, workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """``W <- (1 - eta decay) W - eta scale U`` for every block of every (M, W) problem, U as in ns_blocks."""
    if len(problems) > 0:
        workspace = _workspace_on(ns_blocks_workspace_bytes(problems), problems[0][0], workspace, stream)
        PreparedNSBlocks(problems, a, b, c, steps, eta, decay, scale, workspace)(stream)


# ---------------------------------------------------------------------------
# 8-bit integer matrices with a scale for each row
# ---------------------------------------------------------------------------

MUON_INT8_STEP = 64
MUON_INT8_MAX_K = 131008
MUON_GLU_MAX_SIDE = 4194240
_ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}


def _act_code(act: str) -> int:
    code = _ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {', '.join(_ACTS)}")
    return code


def _same_device(first: torch.Tensor, *rest: Optional[torch.Tensor]) -> int:
    """The one device of all tensors: the current one, whose stream and pool the call uses."""
    where = first.get_device()
    for t in rest:
        if t is not None and t.get_device() != where:
            raise ValueError("all tensors must be on one device")
    if where < 0:
        raise ValueError("the tensors must be device tensors")
    if where != torch.cuda.current_device():
        raise ValueError(f"the tensors are on cuda:{where}, which is not the current device (use torch.cuda.device)")
    return where


def _stream_on(stream, where: int) -> int:
    """As _stream, for a call whose device is known to be the current one."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(where)
    return _stream(stream)


def _two_sides(t: torch.Tensor, name: str) -> Tuple[int, int]:
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    return t.shape


def _matrix(t: torch.Tensor, dtype: torch.dtype, rows: int, cols: int, name: str) -> Tuple[int, int]:
    """(pointer, row pitch) of a rows x cols device matrix of one type."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}]")
    if t.is_contiguous():
        return t.data_ptr(), cols
    ptr, ld = _rows2(t, name)
    return ptr, ld if ld > cols else cols


def _pair(a: torch.Tensor, b: torch.Tensor, dtype: torch.dtype, rows: int, cols: int, names: str) -> Tuple[int, int, int]:
    """(pointers, common row pitch) of two rows x cols matrices of one type."""
    ap, lda = _matrix(a, dtype, rows, cols, f"each of {names}")
    bp, ldb = _matrix(b, dtype, rows, cols, f"each of {names}")
    if lda != ldb:
        raise ValueError(f"{names} must have one row pitch")
    return ap, bp, lda


def _space(need: int, like: torch.Tensor, workspace: Optional[torch.Tensor], stream):
    """(workspace that is kept alive, pointer, bytes) for a call that needs ``need`` bytes."""
    if need == 0:
        return None, None, 0
    workspace = _workspace_on(need, like, workspace, stream)
    return workspace, _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()


def int8_buffers(rows: int, cols: int, device="cuda") -> Tuple[torch.Tensor, torch.Tensor]:
    """Uninitialised (codes [rows, cols rounded up to 64], scales [rows]) for a rows x cols matrix."""
    q = torch.empty((rows, _ceil_to(cols, MUON_INT8_STEP)), dtype=torch.int8, device=device)
    return q, torch.empty(rows, dtype=torch.float32, device=device)


def _int8_operand(q: torch.Tensor, s: torch.Tensor, rows: int, cols: int, name: str) -> Tuple[int, int, int]:
    """(codes, pitch, scales) of an int8 matrix that holds rows x cols."""
    if q.dtype != torch.int8:
        raise TypeError(f"{name} must be int8")
    held, width = _two_sides(q, name)
    ptr, ld = (q.data_ptr(), width) if q.is_contiguous() else _rows2(q, name)
    need = _ceil_to(cols, MUON_INT8_STEP)
    if held != rows or width < need:
        raise ValueError(f"{name} must hold {rows} rows of at least {need} codes")
    if s.dtype != torch.float32 or s.shape != (rows,):
        raise ValueError(f"the scales of {name} must be float32 of shape ({rows},)")
    if rows <= 1 or width == 0:     # the pitch is not used, the library wants a multiple of 16
        ld = _ceil_to(max(width, need), 16)
    return ptr, ld, _dev(s, f"the scales of {name}")


def int8_quantize(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor, stream=None) -> None:
    """Codes and scales of ``x`` [rows, cols] into (q, s): ``x / s`` rounded to nearest even, s = max |row| * (1 / 127)."""
    where = _same_device(x, q, s)
    xp, ldx = _rows2(x, "x")
    rows, cols = x.shape
    qp, ldq, sp = _int8_operand(q, s, rows, cols, "q")
    status = lib().int8_quantize(xp, dtype_code(x), rows, cols, ldx if ldx > cols else cols, qp, ldq, sp, _stream_on(stream, where))
    if status:
        _check("int8_quantize", status)


@functools.lru_cache(maxsize=1024)
def int8_gemm_workspace_bytes(m: int, n: int, K: int) -> int:
    return int(lib().int8_gemm_workspace_bytes(m, n, K))


@functools.lru_cache(maxsize=1024)
def int8_glu_workspace_bytes(m: int, n: int, K: int) -> int:
    return int(lib().int8_glu_workspace_bytes(m, n, K))


def int8_gemm(A: torch.Tensor, sa: torch.Tensor, B: torch.Tensor, sb: torch.Tensor, C: torch.Tensor,
              workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """``C = (A B^T) sa sb`` for int8 operands (codes, scales) with K = ``A.shape[1]`` columns; C fp32 or bf16."""
    where = _same_device(C, A, sa, B, sb, workspace)
    m, K = A.shape
    n, kb = B.shape
    if kb != K or K % MUON_INT8_STEP or C.shape != (m, n):
        raise ValueError(f"A is m x K, B n x K and C m x n, K a multiple of {MUON_INT8_STEP}")
    ap, lda, sap = _int8_operand(A, sa, m, K, "A")
    bp, ldb, sbp = _int8_operand(B, sb, n, K, "B")
    cp, ldc = (C.data_ptr(), n) if C.is_contiguous() else _rows2(C, "C")
    workspace, ws, nbytes = _space(int8_gemm_workspace_bytes(m, n, K), C, workspace, stream)
    status = lib().int8_gemm(ap, lda, sap, bp, ldb, sbp, cp, dtype_code(C), ldc if ldc > n else n, m, n, K, ws, nbytes,
                             _stream_on(stream, where))
    if status:
        _check("int8_gemm", status)


def int8_glu(A: torch.Tensor, sa: torch.Tensor, Bg: torch.Tensor, sg: torch.Tensor, Bu: torch.Tensor, su: torch.Tensor,
             H: torch.Tensor, act: str = "silu", workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """``H = act(g) * u``, ``g = (A Bg^T) sa sg`` and ``u = (A Bu^T) sa su``, for int8 operands; H fp32 or bf16."""
    where = _same_device(H, A, sa, Bg, sg, Bu, su, workspace)
    m, K = A.shape
    n, kb = Bg.shape
    if kb != K or K % MUON_INT8_STEP or Bu.shape != (n, K) or H.shape != (m, n):
        raise ValueError(f"A is m x K, Bg and Bu n x K and H m x n, K a multiple of {MUON_INT8_STEP}")
    ap, lda, sap = _int8_operand(A, sa, m, K, "A")
    gp, ldg, sgp = _int8_operand(Bg, sg, n, K, "Bg")
    up, ldu, sup = _int8_operand(Bu, su, n, K, "Bu")
    if ldg != ldu:
        raise ValueError("Bg and Bu must have one row pitch")
    hp, ldh = (H.data_ptr(), n) if H.is_contiguous() else _rows2(H, "H")
    workspace, ws, nbytes = _space(int8_glu_workspace_bytes(m, n, K), H, workspace, stream)
    status = lib().int8_glu(ap, lda, sap, gp, sgp, up, sup, ldg, _act_code(act), hp, dtype_code(H), ldh if ldh > n else n, m, n, K,
                            ws, nbytes, _stream_on(stream, where))
    if status:
        _check("int8_glu", status)


# ---------------------------------------------------------------------------
# The gated feed-forward block in bf16
# ---------------------------------------------------------------------------

@functools.lru_cache(maxsize=1024)
def glu_forward_workspace_bytes(tokens: int, out: int, inp: int) -> int:
    return int(lib().glu_forward_workspace_bytes(tokens, out, inp))


@functools.lru_cache(maxsize=1024)
def glu_backward_workspace_bytes(tokens: int, out: int, inp: int) -> int:
    return int(lib().glu_backward_workspace_bytes(tokens, out, inp))


@functools.lru_cache(maxsize=1024)
def glu_weight_grad_workspace_bytes(tokens: int, out: int, inp: int) -> int:
    return int(lib().glu_weight_grad_workspace_bytes(tokens, out, inp))


def glu_forward(x: torch.Tensor, wg: torch.Tensor, wu: torch.Tensor, h: torch.Tensor, g: Optional[torch.Tensor] = None,
                u: Optional[torch.Tensor] = None, act: str = "silu", workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """``h = act(x wg^T) * (x wu^T)`` in bf16; ``g`` and ``u`` (both or neither) receive the two products for the backward."""
    where = _same_device(h, x, wg, wu, g, u, workspace)
    tokens, inp = _two_sides(x, "x")
    out = _two_sides(wg, "wg")[0]
    if (g is None) != (u is None):
        raise ValueError("give g and u or neither")
    bf = torch.bfloat16
    xp, ldx = _matrix(x, bf, tokens, inp, "x")
    gp, up, ldw = _pair(wg, wu, bf, out, inp, "wg and wu")
    hp, ldh = _matrix(h, bf, tokens, out, "h")
    sg, su, lds = _pair(g, u, bf, tokens, out, "g and u") if g is not None else (None, None, 0)
    workspace, ws, nbytes = _space(glu_forward_workspace_bytes(tokens, out, inp), h, workspace, stream)
    status = lib().glu_forward(xp, ldx, gp, up, ldw, _act_code(act), hp, ldh, sg, su, lds, tokens, out, inp, ws, nbytes,
                               _stream_on(stream, where))
    if status:
        _check("glu_forward", status)


def glu_backward(dh: torch.Tensor, g: torch.Tensor, u: torch.Tensor, dg: torch.Tensor, du: torch.Tensor,
                 wg: Optional[torch.Tensor] = None, wu: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                 h: Optional[torch.Tensor] = None, act: str = "silu", workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """``dg = dh u act'(g)``, ``du = dh act(g)``; ``dx = dg wg + du wu`` where ``dx`` is given, and ``h`` again where it is.

    dg, du and h may each be dh, g or u itself."""
    where = _same_device(dh, g, u, dg, du, wg, wu, dx, h, workspace)
    tokens, out = _two_sides(dh, "dh")
    if (wg is None) != (wu is None) or (dx is not None and wg is None):
        raise ValueError("dx needs wg and wu")
    bf = torch.bfloat16
    dhp, lddh = _matrix(dh, bf, tokens, out, "dh")
    gp, up, ldg = _pair(g, u, bf, tokens, out, "g and u")
    dgp, dup, ldd = _pair(dg, du, bf, tokens, out, "dg and du")
    hp, ldh = _matrix(h, bf, tokens, out, "h") if h is not None else (None, 0)
    inp, wgp, wup, ldw, dxp, lddx, ws, nbytes = 0, None, None, 0, None, 0, None, 0
    if dx is not None:
        inp = _two_sides(dx, "dx")[1]
        wgp, wup, ldw = _pair(wg, wu, bf, out, inp, "wg and wu")
        dxp, lddx = _matrix(dx, bf, tokens, inp, "dx")
        workspace, ws, nbytes = _space(glu_backward_workspace_bytes(tokens, out, inp), dx, workspace, stream)
    status = lib().glu_backward(dhp, lddh, gp, up, ldg, _act_code(act), dgp, dup, ldd, hp, ldh, wgp, wup, ldw, dxp, lddx, tokens,
                                out, inp, ws, nbytes, _stream_on(stream, where))
    if status:
        _check("glu_backward", status)


def glu_weight_grad(dg: torch.Tensor, du: torch.Tensor, x: torch.Tensor, mg: torch.Tensor, mu: torch.Tensor, alpha: float = 1.0,
                    beta: float = 0.0, workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """``mg <- beta mg + alpha dg^T x`` and ``mu <- beta mu + alpha du^T x``, mg and mu fp32 or bf16."""
    where = _same_device(mg, mu, dg, du, x, workspace)
    tokens, out = _two_sides(dg, "dg")
    inp = _two_sides(x, "x")[1]
    bf = torch.bfloat16
    dgp, dup, ldd = _pair(dg, du, bf, tokens, out, "dg and du")
    xp, ldx = _matrix(x, bf, tokens, inp, "x")
    code = dtype_code(mg)
    gp, up, ldm = _pair(mg, mu, mg.dtype, out, inp, "mg and mu")
    workspace, ws, nbytes = _space(glu_weight_grad_workspace_bytes(tokens, out, inp), mg, workspace, stream)
    status = lib().glu_weight_grad(dgp, dup, ldd, xp, ldx, gp, up, code, ldm, tokens, out, inp, alpha, beta, ws, nbytes,
                                   _stream_on(stream, where))
    if status:
        _check("glu_weight_grad", status)
