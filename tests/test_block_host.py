"""The operators around the routed layer, host side: what needs no GPU."""
import types

import pytest

import sparse_mixture_experts_19_b200 as moe


# ------------------------------------------------------------- streams
@pytest.fixture
def streams(monkeypatch):
    """torch's stream functions replaced by ones that say which was asked for."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: ("external", handle))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: ("on", s))


@pytest.mark.parametrize("stream,want", [
    (0, "default"), (1, "default"), (2, ("external", 2)), (0x7f0000001000, ("external", 0x7f0000001000)),
    (types.SimpleNamespace(cuda_stream=0), "default"),
    (types.SimpleNamespace(cuda_stream=0x7f0000002000), ("external", 0x7f0000002000))])
def test_raw_stream_handles(streams, stream, want):
    """Handle 0 is the default stream, in a call of the convenience forms too,
    and an object needs no more than its handle."""
    assert moe._on(stream) == ("on", want)
