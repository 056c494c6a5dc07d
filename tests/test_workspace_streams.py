"""Workspaces that a call makes for itself belong to the stream that the call goes to."""
import contextlib

import pytest
import torch

import matrix_aware_optimizer_amd as mao
from matrix_aware_optimizer_amd import _abi
from workloads import QUINTIC


@pytest.mark.parametrize("handle,want", [(0, "default"), (7, ("external", 7))])
def test_the_null_handle_is_the_default_stream(monkeypatch, handle, want):
    """Handle 0 is the default stream; an ExternalStream of 0 would be a new one from the pool."""
    seen = []

    def stream(s):
        seen.append(s)
        return contextlib.nullcontext()

    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: ("external", h))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    ws = _abi._workspace_on(16, torch.empty(1), None, handle)
    assert ws.numel() == 16 and seen == [want]


def stream_of(address):
    """The stream whose pool the memory at an address belongs to."""
    for segment in torch.cuda.memory_snapshot():
        if segment["address"] <= address < segment["address"] + segment["total_size"]:
            return segment["stream"]
    raise AssertionError("not memory of the allocator")


@pytest.fixture
def workspaces(monkeypatch):
    """(stream, workspace address) of every call that takes a workspace, and the calls go on."""
    seen, L = [], mao.lib()

    class Recording:
        def __getattr__(self, name):
            real = getattr(L, name)
            if name not in ("fp8_gemm", "ns_blocks", "ns_blocks_update", "muon_momentum", "ns_orthogonalize", "ns_gram", "dion_step"):
                return real

            def call(*args):
                if args[-3]:
                    seen.append((args[-1], args[-3]))
                return real(*args)
            return call

    monkeypatch.setattr(_abi, "lib", Recording)
    return seen


def blocks(seed=0):
    M = torch.randn(2, 32, 96, generator=torch.Generator().manual_seed(seed)).cuda()
    return M, torch.empty_like(M)


@pytest.mark.gpu
def test_one_shot_calls(workspaces):
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    q, s = mao.fp8_buffers(100, 14336)
    w, ws = mao.fp8_buffers(512, 14336)
    q.view(torch.uint8).zero_()
    w.view(torch.uint8).zero_()
    C = torch.empty(100, 512, device="cuda")
    M, U = blocks()
    torch.cuda.synchronize()
    for stream in (None, 0, side, side.cuda_stream):
        with torch.cuda.stream(other):                   # current is another stream than the call's
            mao.fp8_gemm(q, s, w, ws, C, stream=stream)
            mao.ns_blocks([(M, U)], *QUINTIC, 5, stream=stream)
            mao.ns_blocks_update([(M, U)], *QUINTIC, 5, eta=0.1, stream=stream)
        want = other.cuda_stream if stream is None else stream if isinstance(stream, int) else stream.cuda_stream
        assert len(workspaces) == 3
        for handle, address in workspaces:
            assert handle == want and stream_of(address) == want
        del workspaces[:]
        torch.cuda.synchronize()


def test_a_plan_keeps_a_workspace_for_each_stream(monkeypatch):
    """The memory that a plan runs on comes from the stream it is called on, whatever stream made the plan."""
    made, calls = [], []
    current = [11]

    class Lib:
        ns_blocks_workspace_bytes = staticmethod(lambda *a: 64)
        ns_blocks = staticmethod(lambda *a: calls.append((a[-1], a[-3])) or 0)

    def workspace_on(need, like, given, stream):
        ws = torch.empty(need, dtype=torch.uint8) if given is None else given
        made.append((_abi._stream(stream), ws.data_ptr()))
        return ws

    monkeypatch.setattr(_abi, "lib", Lib)
    monkeypatch.setattr(_abi, "_block_problems", lambda problems: (_abi.BlockProblem * 1)())
    monkeypatch.setattr(_abi, "_dev", lambda t, name: t.data_ptr())
    monkeypatch.setattr(_abi, "_stream", lambda stream: current[0] if stream is None else stream)
    monkeypatch.setattr(_abi, "_workspace_on", workspace_on)
    monkeypatch.setattr(_abi, "_workspace", lambda need, like, given: workspace_on(need, like, given, None))
    x = torch.empty(2, 4, 8)
    plan = mao.PreparedNSBlocks([(x, x)], *QUINTIC, 5)
    del calls[:]                                         # what the plan asked while it was made
    for stream in (None, 22, None, 33, 22):
        plan(stream)
    current[0] = 44
    plan()
    assert [c[0] for c in calls] == [11, 22, 11, 33, 22, 44]
    owner = {address: handle for handle, address in made}
    assert all(owner[address] == handle for handle, address in calls)
    assert len(made) == 4 and plan.workspace.data_ptr() == calls[0][1]
    # a workspace that the caller gave is used on every stream
    mine = torch.empty(64, dtype=torch.uint8)
    plan = mao.PreparedNSBlocks([(x, x)], *QUINTIC, 5, workspace=mine)
    del calls[:]
    plan()
    plan(22)
    assert [c[1] for c in calls] == [mine.data_ptr()] * 2


@pytest.mark.gpu
def test_plans(workspaces):
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    M, U = blocks()
    torch.cuda.synchronize()
    plan = mao.PreparedNSBlocks([(M, U)], *QUINTIC, 5)
    plan()
    want = U.clone()
    default = torch.cuda.current_stream().cuda_stream
    for stream in (side, other.cuda_stream, 0, None):
        torch.cuda.synchronize()
        U.zero_()
        torch.cuda.synchronize()
        plan(stream)
        torch.cuda.synchronize()
        assert torch.equal(U, want)
    handles = [handle for handle, _ in workspaces]
    assert handles == [default, side.cuda_stream, other.cuda_stream, 0, default]
    for handle, address in workspaces:
        assert stream_of(address) == handle


@pytest.mark.gpu
def test_calls_of_the_optimizer_steps(workspaces):
    """muon_momentum, ns_orthogonalize, a stage call (its fresh workspace is cleared on the call's stream) and dion_step."""
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    M, G = (torch.randn(256, 512, device="cuda") for _ in range(2))
    U, sums = torch.empty_like(M), torch.empty(1, device="cuda")
    offsets = torch.tensor([0, M.numel()], device="cuda")
    X = torch.randn(1, 256, 512, device="cuda").to(torch.bfloat16)
    A = torch.empty(1, 256, 256, device="cuda", dtype=torch.bfloat16)
    Q = torch.linalg.qr(torch.randn(512, 16, device="cuda"))[0].contiguous()
    torch.cuda.synchronize()
    for stream in (None, 0, side, side.cuda_stream):
        with torch.cuda.stream(other):
            mao.muon_momentum(M, G, 0.9, 0.1, offsets, sums, stream=stream)
            mao.ns_orthogonalize([(M, U, None)], *QUINTIC, 5, stream=stream)
            mao.ns_gram(X, A, stream=stream)
            mao.dion_step([(M, G, U, Q)], 16, 0.95, 0.01, stream=stream)
        want = other.cuda_stream if stream is None else stream if isinstance(stream, int) else stream.cuda_stream
        assert len(workspaces) == 4
        for handle, address in workspaces:
            assert handle == want and stream_of(address) == want
        del workspaces[:]
        torch.cuda.synchronize()
