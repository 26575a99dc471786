"""Refusals of the operators around the routed layer: bad arguments return a
status before anything is enqueued (no GPU needed: no call here gets as far as
a launch)."""
import ctypes

import pytest

import sparse_mixture_experts_19_b200 as moe
from sparse_mixture_experts_19_b200 import build

P = 1 << 20  # a 256-byte aligned address that no refused call reads
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return moe.load()


def dense(**kw):
    c = moe.dense_config(16, 64, 32, "silu")
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def norm(**kw):
    c = moe.norm_config(16, 64)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(K=0), 1), (dict(K=12), 1), (dict(N=-8), 1), (dict(N=20), 1), (dict(act=5), 1),
    (dict(act=-1), 1), (dict(dtype=7), 1), (dict(grad_dtype=2), 1), (dict(dtype=0), 2)])
def test_dense_configurations(lib, kw, status):
    c = dense(**kw)
    r = ctypes.byref(c)
    for fn in (lib.moe_linear_workspace_size, lib.moe_linear_backward_workspace_size, lib.moe_gated_workspace_size,
               lib.moe_gated_backward_workspace_size):
        assert fn(r) == 0 and lib.moe_last_error()
    assert lib.moe_linear_forward(r, P, P, None, None, 2 * P, None, P, BIG, None) == status
    assert lib.moe_linear_backward(r, P, P, P, P, 2 * P, 3 * P, None, P, BIG, None) == status
    assert lib.moe_gated_forward(r, P, P, P, None, None, 2 * P, None, None, P, BIG, None) == status
    assert lib.moe_gated_backward(r, P, P, P, P, P, P, 2 * P, 3 * P, 4 * P, None, None, P, BIG, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(H=12), 1), (dict(H=16392), 2), (dict(kind=2), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(dtype=3), 1), (dict(dy_dtype=3), 1),
    (dict(dtype=0, dy_dtype=1), 2)])
def test_norm_configurations(lib, kw, status):
    r = ctypes.byref(norm(**kw))
    assert lib.moe_norm_workspace_size(r) == 0
    assert lib.moe_norm_forward(r, P, None, None, P, None, None, None) == status
    assert lib.moe_norm_backward(r, P, P, None, P, P, None, 2 * P, None, None, P, BIG, None) == status


def test_null_configuration(lib):
    assert lib.moe_norm_forward(None, P, None, None, P, None, None, None) == 1
    assert lib.moe_linear_forward(None, P, P, None, None, P, None, P, BIG, None) == 1
    assert lib.moe_gated_backward_workspace_size(None) == 0


def test_workspaces(lib):
    r = ctypes.byref(dense())
    n = lib.moe_gated_backward_workspace_size(r)
    assert n > lib.moe_gated_workspace_size(r) >= moe.DENSE_WS_HEADER
    args = [P, P, P, P, P, P, 2 * P, 3 * P, 4 * P, None, None]
    assert lib.moe_gated_backward(r, *args, None, n, None) == 3
    assert lib.moe_gated_backward(r, *args, P + 16, n, None) == 3
    assert lib.moe_gated_backward(r, *args, P, n - 1, None) == 3
    nr = ctypes.byref(norm())
    m = lib.moe_norm_workspace_size(nr)
    assert lib.moe_norm_backward(nr, P, P, None, P, P, None, 2 * P, P, None, P, m - 1, None) == 3
    assert lib.moe_dense_get_device_status(None, 256, None, None) == 3
    assert lib.moe_dense_get_device_status(P, moe.DENSE_WS_HEADER - 1, None, None) == 3
    # the workspace grows with T only as its contents do
    sizes = [moe.moe_linear_backward_workspace_size(moe.dense_config(t, 64, 32, "silu")) for t in (0, 1, 64, 4096)]
    assert sizes == sorted(sizes) and sizes[0] == moe.DENSE_WS_HEADER


def test_linear_pointers(lib):
    r = ctypes.byref(dense())
    ok = [P, P, None, None, 2 * P, None]
    for i in (0, 1, 4):
        assert lib.moe_linear_forward(r, *[None if j == i else a for j, a in enumerate(ok)], P, BIG, None) == 1
    for i in range(6):
        assert lib.moe_linear_forward(r, *[P + 8 if j == i else a for j, a in enumerate(ok)], P, BIG, None) == 1
    assert lib.moe_linear_forward(r, P, P, None, None, P, None, P, BIG, None) == 1  # y is x
    assert lib.moe_linear_forward(r, P, P, None, 3 * P, 2 * P, 3 * P, P, BIG, None) == 1  # z_out is residual
    # backward: z is needed with an activation, x with d_w, w with dx
    assert lib.moe_linear_backward(r, P, P, P, None, 2 * P, 3 * P, None, P, BIG, None) == 1
    assert lib.moe_linear_backward(r, P, None, P, P, 2 * P, 3 * P, None, P, BIG, None) == 1
    assert lib.moe_linear_backward(r, P, P, None, P, 2 * P, 3 * P, None, P, BIG, None) == 1
    assert lib.moe_linear_backward(r, P, P, P, P, P, 3 * P, None, P, BIG, None) == 1  # dx is dy
    # dx is w, d_w is x, w or dx
    assert lib.moe_linear_backward(r, P, 2 * P, 3 * P, P, 3 * P, 4 * P, None, P, BIG, None) == 1
    for d_w in (2 * P, 3 * P, 5 * P):
        assert lib.moe_linear_backward(r, P, 2 * P, 3 * P, P, 5 * P, d_w, None, P, BIG, None) == 1


def test_gated_pointers(lib):
    r = ctypes.byref(dense())
    ok = [P, P, P, None, None, 2 * P, None, None]
    for i in (0, 1, 2, 5):
        assert lib.moe_gated_forward(r, *[None if j == i else a for j, a in enumerate(ok)], P, BIG, None) == 1
    for i in range(8):
        assert lib.moe_gated_forward(r, *[P + 4 if j == i else a for j, a in enumerate(ok)], P, BIG, None) == 1
    assert lib.moe_gated_forward(r, P, P, P, None, None, 2 * P, 3 * P, 3 * P, P, BIG, None) == 1  # g is u
    args = [P, P, P, P, P, P, 2 * P, 3 * P, None, None, None]
    assert lib.moe_gated_backward(r, *args, P, BIG, None) == 1  # one weight gradient alone
    assert b"go together" in lib.moe_last_error()
    # dx is w_gate; d_w_up is x, w_gate, w_up or dx
    back = [P, 2 * P, 3 * P, 4 * P, P, P, 5 * P, 6 * P, 7 * P, None, None]
    for i, v in ((6, 3 * P), (8, 2 * P), (8, 3 * P), (8, 4 * P), (8, 5 * P)):
        assert lib.moe_gated_backward(r, *[v if j == i else a for j, a in enumerate(back)], P, BIG, None) == 1
        assert b"the same tensor" in lib.moe_last_error()


def test_norm_pointers(lib):
    r = ctypes.byref(norm())
    assert lib.moe_norm_forward(r, None, None, None, P, None, None, None) == 1
    assert lib.moe_norm_forward(r, P, P + 4, None, P, None, None, None) == 1
    assert lib.moe_norm_backward(r, P, P, None, None, P, None, 2 * P, None, None, P, BIG, None) == 1  # layer: mean
    assert lib.moe_norm_backward(r, P, P, None, P, None, None, 2 * P, None, None, P, BIG, None) == 1
    mixed = ctypes.byref(norm(dy_dtype=0))
    assert lib.moe_norm_backward(mixed, P, P, None, P, P, None, P, None, None, P, BIG, None) == 1  # dx in a float32 dy


def test_python_refusals():
    torch = pytest.importorskip("torch")
    with pytest.raises(moe.MoeError):
        moe.dense_config(1, 8, 8, act="swish")
    with pytest.raises(moe.MoeError):
        moe.norm_config(1, 8, kind="batch")
    with pytest.raises(moe.MoeError):
        moe.dense_config(1, 8, 8, grad_dtype="f16")
    cfg = moe.dense_config(2, 8, 8)
    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    with pytest.raises(moe.MoeError, match="unknown"):
        moe.moe_linear_forward(dense(dtype=7), x, x, None, None, x)
    with pytest.raises(moe.MoeError, match="CUDA"):
        moe.moe_linear_forward(cfg, x, torch.zeros(8, 8, dtype=torch.bfloat16), None, None, x)
    with pytest.raises(moe.MoeError, match="shape"):
        moe.moe_linear_forward(cfg, torch.zeros(3, 8, dtype=torch.bfloat16), x, None, None, x)
    with pytest.raises(moe.MoeError, match="not torch.bfloat16"):
        moe.moe_linear_forward(cfg, torch.zeros(2, 8), x, None, None, x)
    with pytest.raises(moe.MoeError, match="None"):
        moe.moe_linear_forward(cfg, None, x, None, None, x)
    with pytest.raises(moe.MoeError, match="norm_kind"):
        moe.forward(x, x, x, x, x, 1, norm_w=x)
