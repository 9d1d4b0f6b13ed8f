"""Where the gradient operators take outputs and workspaces from when a call
names a stream: torch's allocator must see the call's own stream."""
import contextlib

import pytest
import torch

import sharded_optimizer_step_adamw_amd as z

DEV = torch.device("cuda:0")


class Named:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def taken(monkeypatch):
    """The handles of the streams under which memory was taken, with torch's
    streams stood in for: an ExternalStream of 0 is a new stream, as torch's is."""
    state = {"current": 0, "made": []}

    @contextlib.contextmanager
    def on(stream):
        before, state["current"] = state["current"], stream.cuda_stream
        yield
        state["current"] = before

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: Named(h or 0xF00))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Named(0))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: state["current"], raising=False)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: state["made"].append(state["current"]))
    return state


@pytest.mark.parametrize("current", [0, 0x100])
@pytest.mark.parametrize("stream", [None, Named(0), 0, Named(0x100), Named(0x200), 0x200])
def test_memory_comes_from_the_stream_of_the_call(taken, current, stream):
    taken["current"] = current
    on = z._On(DEV, stream)
    on.empty((3,), torch.uint8)
    want = current if stream is None else getattr(stream, "cuda_stream", stream)
    assert on.handle == want and taken["made"] == [want] and taken["current"] == current


@pytest.mark.gpu
def test_default_stream_named_while_another_is_current():
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn((100, 40), generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randn((60, 40), generator=g, device=DEV).to(torch.bfloat16)
    y = torch.randint(0, 60, (100,), generator=g, device=DEV)
    want = z.linear_xent_grad(x, w, y)
    torch.cuda.synchronize()
    real, seen = torch.empty, []

    def empty(*a, **k):
        seen.append(torch.cuda.current_stream(DEV).cuda_stream)
        return real(*a, **k)

    with pytest.MonkeyPatch.context() as m, torch.cuda.stream(torch.cuda.Stream()):
        m.setattr(torch, "empty", empty)
        for stream in (torch.cuda.default_stream(DEV), 0):
            got = z.linear_xent_grad(x, w, y, stream=stream)
            torch.cuda.synchronize()
            for a, b in zip(want, got):
                assert torch.equal(a, b)
    assert seen and set(seen) == {0}
