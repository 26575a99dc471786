"""The operators around the routed layer, host side: what needs no GPU."""
import ctypes
import os
import re
import subprocess
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


# --------------------------------------------------------------- overlaps
# (function, configuration, tensors in argument order with their bytes, which of
# them are written, inputs that the first output may replace, workspace query)
T, K, N, G = 16, 64, 32, 1 << 30
TK, TN, NK, V = T * K * 2, T * N * 2, N * K * 2, N * 4
CALLS = [
    ("moe_norm_forward", moe.norm_config(T, K, eps=1e-5),
     [("x", TK), ("weight", K * 4), ("bias", K * 4), ("y", TK), ("mean_out", T * 4), ("rstd_out", T * 4)],
     ("y", "mean_out", "rstd_out"), ("x",), None),
    ("moe_norm_backward", moe.norm_config(T, K),
     [("dy", TK), ("x", TK), ("weight", K * 4), ("mean", T * 4), ("rstd", T * 4), ("d_residual", TK), ("dx", TK),
      ("d_weight", K * 4), ("d_bias", K * 4)],
     ("dx", "d_weight", "d_bias"), ("dy", "x", "d_residual"), "moe_norm_workspace_size"),
    ("moe_linear_forward", moe.dense_config(T, K, N, "silu"),
     [("x", TK), ("w", NK), ("bias", V), ("residual", TN), ("y", TN), ("z_out", TN)], ("y", "z_out"), ("residual",),
     "moe_linear_workspace_size"),
    ("moe_linear_backward", moe.dense_config(T, K, N, "silu"),
     [("dy", TN), ("x", TK), ("w", NK), ("z", TN), ("dx", TK), ("d_w", 2 * NK), ("d_bias", V)],
     ("dx", "d_w", "d_bias"), (), "moe_linear_backward_workspace_size"),
    ("moe_gated_forward", moe.dense_config(T, K, N, "silu"),
     [("x", TK), ("w_gate", NK), ("w_up", NK), ("b_gate", V), ("b_up", V), ("h", TN), ("g_out", TN), ("u_out", TN)],
     ("h", "g_out", "u_out"), (), "moe_gated_workspace_size"),
    ("moe_gated_backward", moe.dense_config(T, K, N, "silu", grad_dtype="bf16"),
     [("dh", TN), ("x", TK), ("w_gate", NK), ("w_up", NK), ("g", TN), ("u", TN), ("dx", TK), ("d_w_gate", NK),
      ("d_w_up", NK), ("d_b_gate", V), ("d_b_up", V)],
     ("dx", "d_w_gate", "d_w_up", "d_b_gate", "d_b_up"), (), "moe_gated_backward_workspace_size"),
]


@pytest.mark.parametrize("fn,cfg,tensors,written,in_place,ws_query", CALLS, ids=[c[0] for c in CALLS])
def test_overlapping_tensors(fn, cfg, tensors, written, in_place, ws_query):
    """A written tensor that shares its first, its last or all bytes with
    another one of the call, and a tensor inside the workspace, are refused; each
    call here has one such pair, so none gets as far as a launch."""
    build.build()
    lib = moe.load()
    at = {name: (i + 1) * G for i, (name, _) in enumerate(tensors)}
    size = dict(tensors)
    ws = (len(tensors) + 1) * G
    ws_bytes = getattr(lib, ws_query)(ctypes.byref(cfg)) if ws_query else 0

    def refused(moved, by):
        where = dict(at, **{moved: by})
        extra = [ws, ws_bytes] if ws_query else []
        assert getattr(lib, fn)(ctypes.byref(cfg), *(where[n] for n, _ in tensors), *extra, None) == 1, (moved, by)
        message = lib.moe_last_error().decode()
        assert moved in message and ("overlaps" in message or "the same tensor" in message), message

    for w in written:
        for other, n in tensors:
            if other == w:
                continue
            if not (w == written[0] and other in in_place):
                refused(w, at[other])
            refused(w, at[other] + n - 16)
            refused(w, at[other] - size[w] + 16)
    for name, n in tensors if ws_query else []:
        refused(name, ws)
        refused(name, ws + ws_bytes - 16)
        refused(name, ws - n + 16)


def test_overlap_without_rows():
    """T = 0: the weight gradients are written (zeros), so not over a weight."""
    build.build()
    lib, cfg = moe.load(), moe.dense_config(0, K, N)
    a = [None, None, G, None, None, G, None]
    assert lib.moe_linear_backward(ctypes.byref(cfg), *a, 2 * G, 1 << 40, None) == 1


# ------------------------------------------------- kernels' shared memory
SMEM_ATTR = r"""
#include <cuda_runtime.h>
#include <stdio.h>
static int device = 0, sets = 0, last = 0;
static cudaError_t get_device(int* d) { *d = device; return cudaSuccess; }
template <typename F> static cudaError_t set_attribute(F, cudaFuncAttribute, int bytes) {
    ++sets;
    last = bytes;
    return cudaSuccess;
}
#define cudaGetDevice get_device
#define cudaFuncSetAttribute set_attribute
#include "tma_host.cuh"
template <int I> void kernel(int* p) { *p = I; }
template <int I> struct Each {
    static void run(size_t bytes) {
        moe::ensure_smem_attr(kernel<I>, bytes);
        Each<I - 1>::run(bytes);
    }
};
template <> struct Each<-1> { static void run(size_t) {} };
int main() {
    for (int round = 0; round < 3; ++round)
        for (device = 0; device < 3; ++device) Each<55>::run(1000);
    printf("%d ", sets);
    device = 1;
    Each<0>::run(2000);  // more: set anew, on each device
    Each<0>::run(1500);
    device = 2;
    Each<0>::run(1500);
    Each<0>::run(2000);
    printf("%d %d\n", sets, last);
}
"""


def test_shared_memory_attribute_on_several_devices(tmp_path):
    """56 kernels of one type on three devices: the attribute is set once for
    each, and the largest size asked for is what later devices get."""
    src = tmp_path / "attr.cpp"
    src.write_text(SMEM_ATTR)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(build._nvcc())))
    subprocess.run(["g++", "-std=c++17", "-O0", "-w", f"-I{cuda}/include", f"-I{build.CSRC}", str(src), "-o",
                    str(tmp_path / "attr"), f"-L{cuda}/lib64", "-lcudart", f"-Wl,-rpath,{cuda}/lib64"], check=True)
    assert subprocess.check_output([str(tmp_path / "attr")], text=True).split() == ["168", "170", "2000"]
