"""The operators around the routed layer, host side: what needs no GPU."""
import os
import re
import types

import pytest

import sparse_mixture_experts_19_b200 as moe
from sparse_mixture_experts_19_b200 import build


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


# --------------------------------------------------- waits of whole warps
@pytest.mark.parametrize("name", ["dense_gemm_sm100.cu", "dense_skinny_sm100.cu"])
def test_collective_waits(name):
    """In the dense kernels only the producer's single lane waits by itself; a
    warp whose next instruction takes all of its lanes (tcgen05.ld among them)
    waits in the form that gives each lane the same answer, and looks at it."""
    code = [line.split("//")[0] for line in open(os.path.join(build.CSRC, name))]
    waits = [line.strip() for line in code if re.search(r"\b(wait_or_abort|wait_sleep_or_abort)(_warp)?\(", line)]
    assert len([w for w in waits if "_warp(" not in w]) == 1 and len(waits) >= 3
    assert all(re.match(r"if \(!?wait_", w) for w in waits), waits
