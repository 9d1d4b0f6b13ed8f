"""Where the optimizers' calls take outputs and workspaces from when a call
names a stream: what is allocated for a call must come from the call's own
stream, since the allocator may give it away as soon as the call returns.
Nothing runs: the library and torch's streams are stood in for."""
import contextlib

import pytest
import torch

import sharded_optimizer_step_adamw_amd as z

DEV = torch.device("cuda:0")
SIDE = 0x200


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Tensor:
    """What the binding asks of a tensor that it passes on."""
    device, shape, dtype = DEV, torch.Size((4, 8)), torch.float32

    def numel(self):
        return 1 << 20

    def data_ptr(self):
        return 256


class Library:
    def __getattr__(self, name):
        return lambda *a: z.ZOPT_OK


@pytest.fixture
def made(monkeypatch):
    """The handles of the streams under which memory was taken."""
    state = {"current": 0}
    taken = []

    @contextlib.contextmanager
    def on(stream):
        before, state["current"] = state["current"], stream.cuda_stream
        yield
        state["current"] = before

    def empty(*a, **k):
        taken.append(state["current"])
        return Tensor()

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: Stream(h or 0xF00))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(state["current"]))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: state["current"], raising=False)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(z, "_lib", Library())
    monkeypatch.setattr(z, "_need", lambda *a, **k: None)
    monkeypatch.setattr(z, "_check_matrices", lambda *a, **k: None)
    return taken


T = Tensor()
CALLS = {
    "grad_sq_norm": lambda s: z.grad_sq_norm(T, 100, 10, 1, 0, stream=s),
    "grad_clip_stats": lambda s: z.grad_clip_stats(T, 1.0, stream=s),
    "muon_step": lambda s: z.muon_step([T], [T], [T], [T], 1e-3, stream=s),
    "muon_step_groups": lambda s: z.muon_step_groups([([T], [T], [T], [T])], 1e-3, stream=s),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("stream", [None, Stream(SIDE), SIDE, Stream(0)])
def test_memory_comes_from_the_stream_of_the_call(made, name, stream):
    CALLS[name](stream)
    want = 0 if stream is None else getattr(stream, "cuda_stream", stream)
    assert made and set(made) == {want}


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["grad_sq_norm", "grad_clip_stats", "muon_step", "muon_step_groups"])
def test_results_on_another_stream_are_the_same(name):
    g = torch.Generator(device=DEV).manual_seed(1)
    grad = torch.randn(100_003, generator=g, device=DEV).to(torch.bfloat16)
    sq = torch.rand(3, generator=g, device=DEV, dtype=torch.float64)
    P, M = (torch.randn((96, 160), generator=g, device=DEV) for _ in range(2))
    G = torch.randn((96, 160), generator=g, device=DEV).to(torch.bfloat16)

    def call(stream):
        if name == "grad_sq_norm":
            return [z.grad_sq_norm(grad, 100_003, 8192, 1, 0, stream=stream)]
        if name == "grad_clip_stats":
            return [z.grad_clip_stats(sq, 1.0, stream=stream)]
        p, m, w = P.clone(), M.clone(), torch.empty_like(G)
        torch.cuda.synchronize()
        if name == "muon_step":
            z.muon_step([p], [m], [G], [w], 1e-3, stream=stream)
        else:
            z.muon_step_groups([([p], [m], [G], [w])], 1e-3, stream=stream)
        torch.cuda.synchronize()
        return [p, m, w]

    want = call(None)
    torch.cuda.synchronize()
    got = call(torch.cuda.Stream())
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
