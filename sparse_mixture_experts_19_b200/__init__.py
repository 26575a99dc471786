"""Routed MoE FFN layer for B200 (sm_100a): Python binding of ``libmoe.so``.

Every entry point of the C ABI (``include/moe.h``) has a function of the
same name here.  This module only marshals arguments (torch tensors ->
device pointers, the current CUDA stream); every step of the layer runs in
the library's CUDA kernels.  There is no CPU fallback: if the library is
missing or cannot load, calls raise ``MoeError``.

``forward(...)`` is the convenience form of ``moe_forward`` that allocates
the output and the workspace with torch; ``norm``, ``linear`` and ``gated``
are those of the operators around the layer, and ``ffn_block`` /
``ffn_block_backward`` run them together as a dense pre-norm FFN block.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_F32, MOE_BF16 = 0, 1
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE",
          4: "MOE_ERR_CUDA", 5: "MOE_ERR_DEVICE_CHECK"}
DEVFLAG_BAD_EXPERT_INDEX = 0x1
DEVFLAG_WAIT_TIMEOUT = 0x2
ACTS = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu": 4}
DENSE_WS_HEADER = 5120  # MOE_DENSE_WS_HEADER
NORMS = {"layer": 0, "rms": 1}


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class moe_config_t(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("top_k", ctypes.c_int32), ("I_shared", ctypes.c_int32),
                ("capacity_factor", ctypes.c_float), ("dtype", ctypes.c_int32)]


class moe_norm_config_t(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("kind", ctypes.c_int32), ("eps", ctypes.c_float),
                ("dtype", ctypes.c_int32), ("dy_dtype", ctypes.c_int32)]


class moe_dense_config_t(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("K", ctypes.c_int32), ("N", ctypes.c_int32), ("act", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32)]


class moe_trace_record_t(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("ms", ctypes.c_float)]


_P = ctypes.c_void_p
_SIGS = {
    "moe_workspace_size": ([ctypes.POINTER(moe_config_t)], ctypes.c_size_t),
    "moe_mxfp4_workspace_size": ([ctypes.POINTER(moe_config_t)], ctypes.c_size_t),
    "moe_capacity": ([ctypes.POINTER(moe_config_t)], ctypes.c_int64),
    "moe_route": ([ctypes.POINTER(moe_config_t), _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "moe_route_importance": ([ctypes.POINTER(moe_config_t), _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
                             ctypes.c_int),
    "moe_permute": ([ctypes.POINTER(moe_config_t), _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P],
                    ctypes.c_int),
    "moe_permute_noalloc": ([ctypes.POINTER(moe_config_t), _P, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "moe_grouped_ffn": ([ctypes.POINTER(moe_config_t)] + [_P] * 11 + [ctypes.c_size_t, _P], ctypes.c_int),
    "moe_combine": ([ctypes.POINTER(moe_config_t), _P, _P, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "moe_forward": ([ctypes.POINTER(moe_config_t)] + [_P] * 14 + [ctypes.c_size_t, _P], ctypes.c_int),
    "moe_forward_routed": ([ctypes.POINTER(moe_config_t)] + [_P] * 14 + [ctypes.c_size_t, _P], ctypes.c_int),
    "moe_shard_capacity_left": ([ctypes.POINTER(moe_config_t), _P, ctypes.c_int32, ctypes.c_int32, _P, _P],
                                ctypes.c_int),
    "moe_shard_capacity_left_host": ([ctypes.POINTER(moe_config_t), _P, ctypes.c_int32, ctypes.c_int32, _P],
                                     ctypes.c_int),
    "moe_balance_losses": ([ctypes.c_int32, ctypes.c_int64, _P, _P, ctypes.POINTER(ctypes.c_double)],
                           ctypes.c_int),
    "moe_forward_expert_shard": ([ctypes.POINTER(moe_config_t), _P, _P, _P, ctypes.c_int32, ctypes.c_int32]
                                 + [_P] * 10 + [ctypes.c_size_t, _P], ctypes.c_int),
    "moe_forward_mxfp4": ([ctypes.POINTER(moe_config_t)] + [_P] * 14 + [ctypes.c_size_t, _P], ctypes.c_int),
    "moe_backward_workspace_size": ([ctypes.POINTER(moe_config_t)], ctypes.c_size_t),
    "moe_backward": ([ctypes.POINTER(moe_config_t)] + [_P] * 21 + [ctypes.c_size_t, _P], ctypes.c_int),
    "moe_reduce_partials": ([ctypes.POINTER(moe_config_t), _P, ctypes.c_int32, _P, _P], ctypes.c_int),
    "moe_norm_forward": ([ctypes.POINTER(moe_norm_config_t)] + [_P] * 7, ctypes.c_int),
    "moe_norm_workspace_size": ([ctypes.POINTER(moe_norm_config_t)], ctypes.c_size_t),
    "moe_norm_backward": ([ctypes.POINTER(moe_norm_config_t)] + [_P] * 10 + [ctypes.c_size_t, _P], ctypes.c_int),
    "moe_linear_workspace_size": ([ctypes.POINTER(moe_dense_config_t)], ctypes.c_size_t),
    "moe_linear_backward_workspace_size": ([ctypes.POINTER(moe_dense_config_t)], ctypes.c_size_t),
    "moe_gated_workspace_size": ([ctypes.POINTER(moe_dense_config_t)], ctypes.c_size_t),
    "moe_gated_backward_workspace_size": ([ctypes.POINTER(moe_dense_config_t)], ctypes.c_size_t),
    "moe_linear_forward": ([ctypes.POINTER(moe_dense_config_t)] + [_P] * 7 + [ctypes.c_size_t, _P], ctypes.c_int),
    "moe_linear_backward": ([ctypes.POINTER(moe_dense_config_t)] + [_P] * 8 + [ctypes.c_size_t, _P], ctypes.c_int),
    "moe_gated_forward": ([ctypes.POINTER(moe_dense_config_t)] + [_P] * 9 + [ctypes.c_size_t, _P], ctypes.c_int),
    "moe_gated_backward": ([ctypes.POINTER(moe_dense_config_t)] + [_P] * 12 + [ctypes.c_size_t, _P], ctypes.c_int),
    "moe_dense_get_device_status": ([_P, ctypes.c_size_t, _P, ctypes.POINTER(ctypes.c_int32)], ctypes.c_int),
    "moe_get_device_status": ([ctypes.POINTER(moe_config_t), _P, ctypes.c_size_t, _P,
                               ctypes.POINTER(ctypes.c_int32)], ctypes.c_int),
    "moe_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "moe_last_error": ([], ctypes.c_char_p),
    "moe_trace_begin": ([ctypes.c_int32, ctypes.c_char_p], ctypes.c_int),
    "moe_trace_end": ([ctypes.POINTER(moe_trace_record_t), ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)],
                      ctypes.c_int),
}

_lib = None


def load(path: str | None = None):
    """Load libmoe.so (built by ``sparse_mixture_experts_19_b200.build``)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise MoeError(4, f"{p} is missing; build it with `python -m sparse_mixture_experts_19_b200.build`")
    lib = ctypes.CDLL(p)
    for name, (args, res) in _SIGS.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    if path is None:
        _lib = lib
    return lib


def exported_symbols() -> list[str]:
    return list(_SIGS)


def _check(status: int):
    if status != 0:
        raise MoeError(status, load().moe_last_error().decode())


def config(T: int, H: int, I: int, E: int, top_k: int, I_shared: int = 0,
           capacity_factor: float = 0.0, dtype: str = "bf16") -> moe_config_t:
    return moe_config_t(T, H, I, E, top_k, I_shared, capacity_factor,
                        MOE_BF16 if dtype == "bf16" else MOE_F32)


def workspace_size(cfg: moe_config_t) -> int:
    n = load().moe_workspace_size(ctypes.byref(cfg))
    if n == 0:
        raise MoeError(1, load().moe_last_error().decode())
    return n


def capacity(cfg: moe_config_t) -> int:
    return load().moe_capacity(ctypes.byref(cfg))


def _host(a):
    """A host numpy view of a tensor or array (device tensors are copied)."""
    if hasattr(a, "is_cuda"):
        return a.detach().cpu().numpy()
    return a


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise MoeError(1, "tensor is not on a CUDA device")
    if not t.is_contiguous():
        raise MoeError(1, "tensor is not contiguous")
    return t.data_ptr()


def _ws(ws):
    return _ptr(ws), (ws.numel() * ws.element_size() if ws is not None and not isinstance(ws, int) else 0)


def _stream(stream):
    if stream is None:
        import torch

        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _on(stream):
    """Makes `stream` current for a convenience form's own allocations and
    fills, so that they are ordered with the kernels it enqueues.  A torch
    stream, a raw handle, or an object that has one as `cuda_stream`."""
    import contextlib

    import torch

    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.Stream):
        handle = stream if isinstance(stream, int) else stream.cuda_stream
        # 0 and 1 are the default stream's handles (none, cudaStreamLegacy); as an
        # external stream's, 0 would mean "none given": a stream of torch's own
        stream = torch.cuda.default_stream() if handle in (0, 1) else torch.cuda.ExternalStream(handle)
    return torch.cuda.stream(stream)


def workspace(cfg: moe_config_t, device="cuda"):
    """A zeroed torch byte tensor big enough for cfg (torch allocations are
    256-byte aligned; zeroed so the device check flags start clear)."""
    import torch

    return torch.zeros(workspace_size(cfg), dtype=torch.uint8, device=device)


def moe_route(cfg, x, router_w, router_b, topk_idx, topk_w, ws, stream=None):
    p, n = _ws(ws)
    _check(load().moe_route(ctypes.byref(cfg), _ptr(x), _ptr(router_w), _ptr(router_b), _ptr(topk_idx),
                            _ptr(topk_w), p, n, _stream(stream)))


def moe_route_importance(cfg, x, router_w, router_b, topk_idx, topk_w, importance, ws, stream=None):
    """moe_route, and the softmax over all E scores of each token added to
    importance [E] float32 (the caller zeroes it)."""
    _check(load().moe_route_importance(ctypes.byref(cfg), _ptr(x), _ptr(router_w), _ptr(router_b),
                                       _ptr(topk_idx), _ptr(topk_w), _ptr(importance), *_ws(ws), _stream(stream)))


def moe_balance_losses(importance, counts, T: int) -> dict:
    """The library's load-balance penalties (kl, std, switch; fp64) from the
    per-expert importance (moe_route_importance) and load (the top-k counts
    from moe_permute or moe_forward) covering T tokens.  Tensors on a device
    are copied to the host first (the C function reads host arrays)."""
    import numpy as np

    imp = np.ascontiguousarray(_host(importance), dtype=np.float32).ravel()
    ld = np.ascontiguousarray(_host(counts), dtype=np.int32).ravel()
    if ld.size != imp.size:
        raise MoeError(1, f"importance has {imp.size} experts, load {ld.size}")
    out = (ctypes.c_double * 3)()
    _check(load().moe_balance_losses(imp.size, int(T), imp.ctypes.data, ld.ctypes.data, out))
    return dict(kl=out[0], std=out[1], switch=out[2])


balance_losses = moe_balance_losses


def moe_permute(cfg, topk_idx, counts, offsets, perm_rows, row_of, dropped, ws, stream=None):
    p, n = _ws(ws)
    _check(load().moe_permute(ctypes.byref(cfg), _ptr(topk_idx), _ptr(counts), _ptr(offsets),
                              _ptr(perm_rows), _ptr(row_of), _ptr(dropped), p, n, _stream(stream)))


def moe_permute_noalloc(cfg, topk_idx, counts, offsets, perm_rows, row_of, dropped, stream=None):
    """moe_permute without a workspace, for callers that cannot allocate device
    memory (allocator callbacks, host-owned memory, allocation-free serving
    loops): the scratch is a fixed static array inside the library.  Limit
    T*top_k <= 1048576; concurrent calls on one device race."""
    _check(load().moe_permute_noalloc(ctypes.byref(cfg), _ptr(topk_idx), _ptr(counts), _ptr(offsets),
                                      _ptr(perm_rows), _ptr(row_of), _ptr(dropped), _stream(stream)))


def moe_grouped_ffn(cfg, x, perm_rows, offsets, w_gate, w_up, w_down, ws_gate, ws_up, ws_down,
                    expert_out, ws, stream=None):
    p, n = _ws(ws)
    _check(load().moe_grouped_ffn(ctypes.byref(cfg), _ptr(x), _ptr(perm_rows), _ptr(offsets), _ptr(w_gate),
                                  _ptr(w_up), _ptr(w_down), _ptr(ws_gate), _ptr(ws_up), _ptr(ws_down),
                                  _ptr(expert_out), p, n, _stream(stream)))


def moe_combine(cfg, expert_out, row_of, topk_w, y, ws, stream=None):
    p, n = _ws(ws)
    _check(load().moe_combine(ctypes.byref(cfg), _ptr(expert_out), _ptr(row_of), _ptr(topk_w), _ptr(y),
                              p, n, _stream(stream)))


def moe_forward(cfg, x, router_w, router_b, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, y,
                topk_idx_out=None, counts_out=None, dropped_out=None, ws=None, stream=None):
    p, n = _ws(ws)
    _check(load().moe_forward(ctypes.byref(cfg), _ptr(x), _ptr(router_w), _ptr(router_b), _ptr(w_gate),
                              _ptr(w_up), _ptr(w_down), _ptr(ws_gate), _ptr(ws_up), _ptr(ws_down), _ptr(y),
                              _ptr(topk_idx_out), _ptr(counts_out), _ptr(dropped_out), p, n,
                              _stream(stream)))


def moe_forward_routed(cfg, x, topk_idx, topk_w, capacity_left, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, y,
                       counts_out=None, dropped_out=None, ws=None, stream=None):
    p, n = _ws(ws)
    _check(load().moe_forward_routed(ctypes.byref(cfg), _ptr(x), _ptr(topk_idx), _ptr(topk_w), _ptr(capacity_left),
                                     _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(ws_gate), _ptr(ws_up),
                                     _ptr(ws_down), _ptr(y), _ptr(counts_out), _ptr(dropped_out), p, n,
                                     _stream(stream)))


def moe_shard_capacity_left(cfg, counts_per_shard, shard: int, capacity_left, stream=None):
    """capacity_left [E] int32 for token shard `shard` of the batch cfg
    describes (cfg.T = tokens of all shards), from every shard's counts
    counts_per_shard [n_shards, E] int32, both on the device."""
    n = counts_per_shard.shape[0]
    _check(load().moe_shard_capacity_left(ctypes.byref(cfg), _ptr(counts_per_shard), n, shard, _ptr(capacity_left),
                                          _stream(stream)))


def moe_shard_capacity_left_host(cfg, counts_per_shard, shard: int):
    """moe_shard_capacity_left on host arrays (counts gathered on the host);
    returns an int32 numpy array [E]."""
    import numpy as np

    c = np.ascontiguousarray(counts_per_shard, dtype=np.int32)
    if c.ndim != 2 or c.shape[1] != cfg.E:
        raise MoeError(1, f"counts_per_shard must be [n_shards, {cfg.E}]")
    out = np.empty(cfg.E, np.int32)
    _check(load().moe_shard_capacity_left_host(ctypes.byref(cfg), c.ctypes.data, c.shape[0], shard,
                                               out.ctypes.data))
    return out


def moe_forward_expert_shard(cfg, x, topk_idx, topk_w, expert_begin: int, expert_count: int, w_gate, w_up, w_down,
                             ws_gate, ws_up, ws_down, y_partial, counts_out=None, dropped_out=None, ws=None,
                             stream=None):
    """This shard's float32 partial output of the layer cfg describes (experts
    [expert_begin, expert_begin + expert_count) held here)."""
    p, n = _ws(ws)
    _check(load().moe_forward_expert_shard(ctypes.byref(cfg), _ptr(x), _ptr(topk_idx), _ptr(topk_w), expert_begin,
                                           expert_count, _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(ws_gate),
                                           _ptr(ws_up), _ptr(ws_down), _ptr(y_partial), _ptr(counts_out),
                                           _ptr(dropped_out), p, n, _stream(stream)))


def moe_forward_mxfp4(cfg, x, router_w, router_b, w_gate_blocks, w_gate_scales, w_up_blocks, w_up_scales,
                      w_down_blocks, w_down_scales, y, topk_idx_out=None, counts_out=None, dropped_out=None, ws=None,
                      stream=None):
    """moe_forward with MXFP4 routed experts (uint8 blocks [E, rows, K/32, 16]
    and scales [E, rows, K/32]).  ws: moe_mxfp4_workspace_size(cfg) bytes
    (mxfp4_workspace); up to 32 routed slots that is moe_workspace_size."""
    p, n = _ws(ws)
    _check(load().moe_forward_mxfp4(ctypes.byref(cfg), _ptr(x), _ptr(router_w), _ptr(router_b), _ptr(w_gate_blocks),
                                    _ptr(w_gate_scales), _ptr(w_up_blocks), _ptr(w_up_scales), _ptr(w_down_blocks),
                                    _ptr(w_down_scales), _ptr(y), _ptr(topk_idx_out), _ptr(counts_out),
                                    _ptr(dropped_out), p, n, _stream(stream)))


def moe_mxfp4_workspace_size(cfg) -> int:
    n = load().moe_mxfp4_workspace_size(ctypes.byref(cfg))
    if n == 0:
        raise MoeError(1, load().moe_last_error().decode())
    return n


def mxfp4_workspace(cfg: moe_config_t, device="cuda"):
    """A zeroed workspace for moe_forward_mxfp4 (see workspace)."""
    import torch

    return torch.zeros(moe_mxfp4_workspace_size(cfg), dtype=torch.uint8, device=device)


def moe_backward_workspace_size(cfg) -> int:
    n = load().moe_backward_workspace_size(ctypes.byref(cfg))
    if n == 0:
        raise MoeError(1, load().moe_last_error().decode())
    return n


def moe_backward(cfg, x, dy, topk_idx, topk_w, router_w, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, dx,
                 d_router_w, d_router_b, d_w_gate, d_w_up, d_w_down, d_ws_gate=None, d_ws_up=None, d_ws_down=None,
                 ws=None, stream=None):
    """Every gradient of the layer (float32 outputs, written) for upstream dy."""
    p, n = _ws(ws)
    _check(load().moe_backward(ctypes.byref(cfg), _ptr(x), _ptr(dy), _ptr(topk_idx), _ptr(topk_w), _ptr(router_w),
                               _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(ws_gate), _ptr(ws_up), _ptr(ws_down),
                               _ptr(dx), _ptr(d_router_w), _ptr(d_router_b), _ptr(d_w_gate), _ptr(d_w_up),
                               _ptr(d_w_down), _ptr(d_ws_gate), _ptr(d_ws_up), _ptr(d_ws_down), p, n,
                               _stream(stream)))


def moe_reduce_partials(cfg, partials, y, stream=None):
    """y = the float32 sum of partials [n, T, H] in order, rounded once."""
    n = 1 if partials.dim() == 2 else partials.shape[0]
    _check(load().moe_reduce_partials(ctypes.byref(cfg), _ptr(partials), n, _ptr(y), _stream(stream)))


def forward_expert_parallel(cfg, x, topk_idx, topk_w, expert_begin: int, expert_count: int, w_gate, w_up, w_down,
                            ws_gate=None, ws_up=None, ws_down=None, group=None, ws=None, stream=None):
    """y on every rank of `group` (torch.distributed, NCCL over NVLink): this
    rank's shard of the experts, an all-reduce of the float32 partial outputs,
    one rounding to the layer dtype."""
    import torch
    import torch.distributed as dist

    T, H = x.shape
    y32 = torch.empty((T, H), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = workspace(cfg, x.device)
    moe_forward_expert_shard(cfg, x, topk_idx, topk_w, expert_begin, expert_count, w_gate, w_up, w_down, ws_gate,
                             ws_up, ws_down, y32, ws=ws, stream=stream)
    dist.all_reduce(y32, group=group)  # the exchange step
    y = torch.empty_like(x)
    moe_reduce_partials(cfg, y32, y, stream)
    return y


def moe_get_device_status(cfg, ws, stream=None) -> int:
    """Waits for the stream; returns the device check flags (and clears them)."""
    p, n = _ws(ws)
    flags = ctypes.c_int32(0)
    st = load().moe_get_device_status(ctypes.byref(cfg), p, n, _stream(stream), ctypes.byref(flags))
    if st not in (0, 5):
        _check(st)
    return flags.value


def moe_status_string(status: int) -> str:
    return load().moe_status_string(status).decode()


def moe_last_error() -> str:
    return load().moe_last_error().decode()


def moe_trace_begin(max_launches: int, only: str | None = None):
    """Trace the next launches (only kernels whose name contains `only`)."""
    _check(load().moe_trace_begin(max_launches, None if only is None else only.encode()))


def moe_trace_end(max_records: int = 4096) -> list[tuple[str, float]]:
    recs = (moe_trace_record_t * max_records)()
    n = ctypes.c_int32(0)
    _check(load().moe_trace_end(recs, max_records, ctypes.byref(n)))
    return [(recs[i].name.decode(), recs[i].ms) for i in range(n.value)]


# ------------------------------------------------ the operators around the layer
def _code(table: dict, name: str, what: str) -> int:
    if name not in table:
        raise MoeError(1, f"{what} {name!r} unknown: one of {', '.join(table)}")
    return table[name]


_DTYPES = {"f32": MOE_F32, "bf16": MOE_BF16}


def norm_config(T: int, H: int, kind: str = "layer", eps: float = 1e-5, dtype: str = "bf16",
                dy_dtype: str | None = None) -> moe_norm_config_t:
    """kind "layer" or "rms"; dtype of the rows; dy_dtype (default: dtype) of
    the backward's upstream gradient."""
    d = _code(_DTYPES, dtype, "dtype")
    return moe_norm_config_t(T, H, _code(NORMS, kind, "norm kind"), eps, d,
                             d if dy_dtype is None else _code(_DTYPES, dy_dtype, "dy_dtype"))


def dense_config(T: int, K: int, N: int, act: str = "none", dtype: str = "bf16",
                 grad_dtype: str = "f32") -> moe_dense_config_t:
    """T rows of K inputs to N outputs; act one of ACTS; grad_dtype of the
    weight gradients."""
    return moe_dense_config_t(T, K, N, _code(ACTS, act, "act"), _code(_DTYPES, dtype, "dtype"),
                              _code(_DTYPES, grad_dtype, "grad_dtype"))


class _Call:
    """Argument marshalling of one call: the current device and its stream are
    looked up once, each tensor's type, shape, layout and device checked."""

    __slots__ = ("dev",)

    def __init__(self):
        import torch

        try:
            self.dev = torch.cuda.current_device()
        except (RuntimeError, AssertionError):  # no CUDA device: every tensor is refused below
            self.dev = -2

    def arg(self, t, name: str, shape: tuple, dtype, optional: bool = False):
        """Device pointer of a contiguous tensor of this shape and dtype on the
        current device (ints pass through as raw pointers)."""
        if t is None:
            if optional:
                return None
            raise MoeError(1, f"{name} is None")
        if isinstance(t, int):
            return t
        if t.dtype is dtype and t.shape == shape and t.get_device() == self.dev and t.is_contiguous():
            return t.data_ptr()
        if t.dtype is not dtype:
            raise MoeError(1, f"{name} is {t.dtype}, not {dtype}")
        if t.shape != shape:
            raise MoeError(1, f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
        _ptr(t)
        raise MoeError(1, f"{name} is on {t.device}, not on the current device")

    def ws(self, ws):
        """(pointer, bytes) of a workspace on the current device."""
        if ws is None or isinstance(ws, int):
            return _ws(ws)
        if ws.get_device() == self.dev and ws.is_contiguous():
            return ws.data_ptr(), ws.nbytes
        if ws.is_cuda and ws.get_device() != self.dev:
            raise MoeError(1, f"ws is on {ws.device}, not on the current device")
        return _ptr(ws), ws.nbytes

    def stream(self, stream):
        if stream is None:
            import torch

            return torch._C._cuda_getCurrentRawStream(self.dev)
        return stream if isinstance(stream, int) else stream.cuda_stream


_torch_types: dict = {}


def _torch_type(code: int):
    """The torch dtype of a MOE_* dtype."""
    if not _torch_types:
        import torch

        _torch_types.update({MOE_F32: torch.float32, MOE_BF16: torch.bfloat16})
    if code not in _torch_types:
        raise MoeError(1, f"dtype = {code} unknown")
    return _torch_types[code]


def _sized(size_fn, cfg) -> int:
    n = size_fn(ctypes.byref(cfg))
    if n == 0:
        raise MoeError(1, load().moe_last_error().decode())
    return n


def _new_ws(nbytes: int, device):
    """A workspace whose header (device check flags, counters) is clear."""
    import torch

    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    ws[:DENSE_WS_HEADER].zero_()
    return ws


def moe_norm_workspace_size(cfg) -> int:
    return _sized(load().moe_norm_workspace_size, cfg)


def moe_linear_workspace_size(cfg) -> int:
    return _sized(load().moe_linear_workspace_size, cfg)


def moe_linear_backward_workspace_size(cfg) -> int:
    return _sized(load().moe_linear_backward_workspace_size, cfg)


def moe_gated_workspace_size(cfg) -> int:
    return _sized(load().moe_gated_workspace_size, cfg)


def moe_gated_backward_workspace_size(cfg) -> int:
    return _sized(load().moe_gated_backward_workspace_size, cfg)


def norm_workspace(cfg, device="cuda"):
    return _new_ws(moe_norm_workspace_size(cfg), device)


def linear_workspace(cfg, device="cuda"):
    return _new_ws(moe_linear_workspace_size(cfg), device)


def linear_backward_workspace(cfg, device="cuda"):
    return _new_ws(moe_linear_backward_workspace_size(cfg), device)


def gated_workspace(cfg, device="cuda"):
    return _new_ws(moe_gated_workspace_size(cfg), device)


def gated_backward_workspace(cfg, device="cuda"):
    return _new_ws(moe_gated_backward_workspace_size(cfg), device)


def moe_norm_forward(cfg, x, weight, bias, y, mean_out=None, rstd_out=None, stream=None):
    """y = norm(x); mean_out, rstd_out [T] float32 keep the statistics."""
    T, H = cfg.T, cfg.H
    c, d, f32 = _Call(), _torch_type(cfg.dtype), _torch_type(MOE_F32)
    arg = c.arg
    _check(load().moe_norm_forward(ctypes.byref(cfg), arg(x, "x", (T, H), d),
                                   arg(weight, "weight", (H,), f32, True),
                                   arg(bias, "bias", (H,), f32, True), arg(y, "y", (T, H), d),
                                   arg(mean_out, "mean_out", (T,), f32, True),
                                   arg(rstd_out, "rstd_out", (T,), f32, True), c.stream(stream)))


def moe_norm_backward(cfg, dy, x, weight, mean, rstd, d_residual, dx, d_weight, d_bias, ws, stream=None):
    """dx (+ d_residual), d_weight and d_bias (each may be None) of the norm."""
    T, H = cfg.T, cfg.H
    c, d, f32 = _Call(), _torch_type(cfg.dtype), _torch_type(MOE_F32)
    arg = c.arg
    p, n = c.ws(ws)
    _check(load().moe_norm_backward(ctypes.byref(cfg), arg(dy, "dy", (T, H), _torch_type(cfg.dy_dtype)),
                                    arg(x, "x", (T, H), d), arg(weight, "weight", (H,), f32, True),
                                    arg(mean, "mean", (T,), f32, True), arg(rstd, "rstd", (T,), f32),
                                    arg(d_residual, "d_residual", (T, H), d, True), arg(dx, "dx", (T, H), d),
                                    arg(d_weight, "d_weight", (H,), f32, True),
                                    arg(d_bias, "d_bias", (H,), f32, True), p, n, c.stream(stream)))


def moe_linear_forward(cfg, x, w, bias, residual, y, z_out=None, ws=None, stream=None):
    """y = act(x w^T + bias) + residual; z_out keeps the pre-activations."""
    T, K, N = cfg.T, cfg.K, cfg.N
    c, d, f32 = _Call(), _torch_type(cfg.dtype), _torch_type(MOE_F32)
    arg = c.arg
    _check(load().moe_linear_forward(ctypes.byref(cfg), arg(x, "x", (T, K), d), arg(w, "w", (N, K), d),
                                     arg(bias, "bias", (N,), f32, True),
                                     arg(residual, "residual", (T, N), d, True), arg(y, "y", (T, N), d),
                                     arg(z_out, "z_out", (T, N), d, True), *c.ws(ws), c.stream(stream)))


def moe_linear_backward(cfg, dy, x, w, z, dx, d_w, d_bias, ws=None, stream=None):
    """dx, d_w, d_bias (each may be None) of the linear layer."""
    T, K, N = cfg.T, cfg.K, cfg.N
    c, d, f32, gt = _Call(), _torch_type(cfg.dtype), _torch_type(MOE_F32), _torch_type(cfg.grad_dtype)
    arg = c.arg
    _check(load().moe_linear_backward(ctypes.byref(cfg), arg(dy, "dy", (T, N), d),
                                      arg(x, "x", (T, K), d, d_w is None), arg(w, "w", (N, K), d, dx is None),
                                      arg(z, "z", (T, N), d, True), arg(dx, "dx", (T, K), d, True),
                                      arg(d_w, "d_w", (N, K), gt, True),
                                      arg(d_bias, "d_bias", (N,), f32, True), *c.ws(ws), c.stream(stream)))


def moe_gated_forward(cfg, x, w_gate, w_up, b_gate, b_up, h, g_out=None, u_out=None, ws=None, stream=None):
    """h = act(x w_gate^T + b_gate) * (x w_up^T + b_up); g_out, u_out keep the
    two projections."""
    T, K, N = cfg.T, cfg.K, cfg.N
    c, d, f32 = _Call(), _torch_type(cfg.dtype), _torch_type(MOE_F32)
    arg = c.arg
    _check(load().moe_gated_forward(ctypes.byref(cfg), arg(x, "x", (T, K), d), arg(w_gate, "w_gate", (N, K), d),
                                    arg(w_up, "w_up", (N, K), d), arg(b_gate, "b_gate", (N,), f32, True),
                                    arg(b_up, "b_up", (N,), f32, True), arg(h, "h", (T, N), d),
                                    arg(g_out, "g_out", (T, N), d, True), arg(u_out, "u_out", (T, N), d, True),
                                    *c.ws(ws), c.stream(stream)))


def moe_gated_backward(cfg, dh, x, w_gate, w_up, g, u, dx, d_w_gate, d_w_up, d_b_gate=None, d_b_up=None, ws=None,
                       stream=None):
    """dx, the two weight gradients and the two bias gradients (each may be
    None) of the gate/up projections."""
    T, K, N = cfg.T, cfg.K, cfg.N
    c, d, f32, gt = _Call(), _torch_type(cfg.dtype), _torch_type(MOE_F32), _torch_type(cfg.grad_dtype)
    arg = c.arg
    no_dw = d_w_gate is None and d_w_up is None
    _check(load().moe_gated_backward(
        ctypes.byref(cfg), arg(dh, "dh", (T, N), d), arg(x, "x", (T, K), d, no_dw),
        arg(w_gate, "w_gate", (N, K), d, dx is None), arg(w_up, "w_up", (N, K), d, dx is None),
        arg(g, "g", (T, N), d), arg(u, "u", (T, N), d), arg(dx, "dx", (T, K), d, True),
        arg(d_w_gate, "d_w_gate", (N, K), gt, True), arg(d_w_up, "d_w_up", (N, K), gt, True),
        arg(d_b_gate, "d_b_gate", (N,), f32, True), arg(d_b_up, "d_b_up", (N,), f32, True), *c.ws(ws),
        c.stream(stream)))


def moe_dense_get_device_status(ws, stream=None) -> int:
    """moe_get_device_status for a workspace of the linear and gated calls."""
    flags = ctypes.c_int32(0)
    st = load().moe_dense_get_device_status(*_ws(ws), _stream(stream), ctypes.byref(flags))
    if st not in (0, 5):
        _check(st)
    return flags.value


def _dtype_name(t) -> str:
    import torch

    if t.dtype not in (torch.bfloat16, torch.float32):
        raise MoeError(1, f"{t.dtype} tensors are not supported")
    return "bf16" if t.dtype == torch.bfloat16 else "f32"


def norm(x, weight=None, bias=None, eps: float = 1e-5, kind: str = "layer", mean_out=None, rstd_out=None,
         stream=None):
    """moe_norm_forward into a new tensor."""
    import torch

    T, H = x.shape
    with _on(stream):
        y = torch.empty_like(x)
        moe_norm_forward(norm_config(T, H, kind, eps, _dtype_name(x)), x, weight, bias, y, mean_out, rstd_out)
    return y


def linear(x, w, bias=None, residual=None, act: str = "none", z_out=None, ws=None, stream=None):
    """moe_linear_forward into a new tensor."""
    import torch

    cfg = dense_config(x.shape[0], x.shape[1], w.shape[0], act, _dtype_name(x))
    with _on(stream):
        ws = linear_workspace(cfg, x.device) if ws is None else ws
        y = torch.empty((cfg.T, cfg.N), dtype=x.dtype, device=x.device)
        moe_linear_forward(cfg, x, w, bias, residual, y, z_out, ws)
    return y


def gated(x, w_gate, w_up, b_gate=None, b_up=None, act: str = "silu", g_out=None, u_out=None, ws=None, stream=None):
    """moe_gated_forward into a new tensor."""
    import torch

    cfg = dense_config(x.shape[0], x.shape[1], w_gate.shape[0], act, _dtype_name(x))
    with _on(stream):
        ws = gated_workspace(cfg, x.device) if ws is None else ws
        h = torch.empty((cfg.T, cfg.N), dtype=x.dtype, device=x.device)
        moe_gated_forward(cfg, x, w_gate, w_up, b_gate, b_up, h, g_out, u_out, ws)
    return h


def ffn_block(x, norm_w, w_gate, w_up, w_down, norm_b=None, kind: str = "rms", eps: float = 1e-5, act: str = "silu",
              keep: bool = False, stream=None):
    """A dense pre-norm FFN block, y = x + (act(n w_gate^T) * (n w_up^T)) w_down^T
    with n = norm(x): the dense layers between routed ones.  x [T, H] bf16,
    w_gate, w_up [I, H], w_down [H, I], norm_w, norm_b [H] float32 or None.
    keep: returns (y, kept), kept being what ffn_block_backward reads."""
    import torch

    T, H = x.shape
    I = w_gate.shape[0]
    dev = x.device
    mean = rstd = g = u = None
    with _on(stream):
        if keep:
            mean, rstd = torch.empty((2, (T + 3) // 4 * 4), dtype=torch.float32, device=dev)[:, :T].unbind()
            g, u = (torch.empty((T, I), dtype=x.dtype, device=dev) for _ in range(2))
        n = norm(x, norm_w, norm_b, eps, kind, mean, rstd)
        h = gated(n, w_gate, w_up, act=act, g_out=g, u_out=u)
        y = linear(h, w_down, residual=x)
    if not keep:
        return y
    return y, dict(x=x, n=n, g=g, u=u, h=h, mean=mean, rstd=rstd, norm_w=norm_w, has_norm_b=norm_b is not None,
                   w_gate=w_gate, w_up=w_up, w_down=w_down, kind=kind, eps=eps, act=act)


def ffn_block_backward(dy, kept, grad_dtype: str = "f32", stream=None) -> dict:
    """Every gradient of ffn_block for the upstream gradient dy [T, H] bf16:
    dx, d_norm_w, d_norm_b (None without the bias), d_w_gate, d_w_up, d_w_down
    (in grad_dtype)."""
    import torch

    k = kept
    x, h, n = k["x"], k["h"], k["n"]
    (T, H), I, dev = x.shape, h.shape[1], x.device
    gt = torch.float32 if grad_dtype == "f32" else torch.bfloat16
    with _on(stream):
        dh, dn, dx = torch.empty_like(h), torch.empty_like(n), torch.empty_like(x)
        out = dict(dx=dx, d_norm_w=None, d_norm_b=None, d_w_gate=torch.empty((I, H), dtype=gt, device=dev),
                   d_w_up=torch.empty((I, H), dtype=gt, device=dev), d_w_down=torch.empty((H, I), dtype=gt, device=dev))
        for name, has in (("d_norm_w", k["norm_w"] is not None), ("d_norm_b", k["has_norm_b"])):
            if has:
                out[name] = torch.empty(H, dtype=torch.float32, device=dev)
        cfg = dense_config(T, I, H, "none", "bf16", grad_dtype)
        moe_linear_backward(cfg, dy, h, k["w_down"], None, dh, out["d_w_down"], None,
                            linear_backward_workspace(cfg, dev))
        cfg = dense_config(T, H, I, k["act"], "bf16", grad_dtype)
        moe_gated_backward(cfg, dh, n, k["w_gate"], k["w_up"], k["g"], k["u"], dn, out["d_w_gate"], out["d_w_up"],
                           ws=gated_backward_workspace(cfg, dev))
        cfg = norm_config(T, H, k["kind"], k["eps"], "bf16")
        moe_norm_backward(cfg, dn, x, k["norm_w"], k["mean"] if k["kind"] == "layer" else None, k["rstd"], dy, dx,
                          out["d_norm_w"], out["d_norm_b"], norm_workspace(cfg, dev))
    return out


def forward(x, router_w, w_gate, w_up, w_down, top_k: int, router_b=None, ws_gate=None, ws_up=None,
            ws_down=None, capacity_factor: float = 0.0, ws=None, topk_idx_out=None, counts_out=None,
            dropped_out=None, stream=None, norm_w=None, norm_b=None, norm_kind: str | None = None,
            norm_eps: float = 1e-5):
    """y = MoE(x): the pages' moe_forward(x, experts, router, top_k) on the GPU.
    norm_kind "layer" or "rms": y = MoE(norm(x)), the layer behind its
    pre-norm (moe_norm_forward with norm_w, norm_b, norm_eps)."""
    import torch

    if norm_kind is None and (norm_w is not None or norm_b is not None):
        raise MoeError(1, "norm_w and norm_b need norm_kind")

    T, H = x.shape
    E, I, _ = w_gate.shape
    Is = 0 if ws_gate is None else ws_gate.shape[0]
    dtype = "bf16" if x.dtype == torch.bfloat16 else "f32"
    cfg = config(T, H, I, E, top_k, Is, capacity_factor, dtype)
    with _on(stream):
        if norm_kind is not None:
            x = norm(x, norm_w, norm_b, norm_eps, norm_kind)
        if ws is None:
            ws = workspace(cfg, x.device)
        y = torch.empty_like(x)
        moe_forward(cfg, x, router_w, router_b, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, y,
                    topk_idx_out, counts_out, dropped_out, ws)
    return y
