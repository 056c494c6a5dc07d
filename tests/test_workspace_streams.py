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
    """(stream, workspace address) of every call of fp8_gemm, ns_blocks and ns_blocks_update, and the calls go on."""
    seen, L = [], mao.lib()

    class Recording:
        def __getattr__(self, name):
            real = getattr(L, name)
            if name not in ("fp8_gemm", "ns_blocks", "ns_blocks_update"):
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
