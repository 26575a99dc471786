"""The operators around the routed layer on the GPU: raw stream handles, rings
and split tiles that are used again and again, the forms a product takes, far
activations and the largest sizes.  References are the formulas in float64;
the tolerances are those of test_block_ops.py, from which the checks come, and
what a test adds is derived where it stands."""
import math

import pytest
import torch

from test_block_ops import (ACTS, BF, F32, U8, acc_tol, gen_of, rnd,
                            test_gated_backward as check_gated_backward, test_gated_forward as check_gated_forward,
                            test_linear_backward as check_linear_backward,
                            test_linear_forward as check_linear_forward, test_norm_backward as check_norm_backward,
                            test_norm_forward as check_norm_forward, within)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- streams
class Handle:
    """A stream object of another library: a handle, nothing else."""

    def __init__(self, cuda_stream):
        self.cuda_stream = cuda_stream


def block_operands(g, T=70, H=256, I=128, E=8):
    x, dy, rw = rnd(g, T, H), rnd(g, T, H), rnd(g, E, H, scale=H ** -0.5)
    nw = rnd(g, H, scale=0.1, dtype=F32, shift=1.0)
    wg, wu, wd = rnd(g, I, H, scale=H ** -0.5), rnd(g, I, H, scale=H ** -0.5), rnd(g, H, I, scale=I ** -0.5)
    return x, dy, rw, nw, wg, wu, wd


@pytest.mark.parametrize("handle", [0, 1, Handle(0)])
def test_default_stream_by_its_handle(gpu_lib, handle):
    """stream=0 is the default stream: a call there from within another stream
    waits for an input that the default stream writes late."""
    moe = gpu_lib
    x, dy, rw, nw, wg, wu, wd = block_operands(gen_of(21))
    ew = [w.unsqueeze(0).repeat(8, 1, 1) for w in (wg, wu, wd)]
    late, late_dy = torch.empty_like(x), torch.empty_like(dy)

    def calls(x, dy, stream):
        y, kept = moe.ffn_block(x, nw, wg, wu, wd, keep=True, stream=stream)
        return [moe.forward(x, rw, *ew, 2, stream=stream), moe.norm(x, nw, stream=stream),
                moe.linear(x, wg, stream=stream), moe.gated(x, wg, wu, stream=stream), y,
                *(t for t in moe.ffn_block_backward(dy, kept, stream=stream).values() if t is not None)]

    want = calls(x, dy, None)
    late.zero_()
    late_dy.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(100_000_000)  # about 60 ms of the default stream
    late.copy_(x)
    late_dy.copy_(dy)
    with torch.cuda.stream(side):
        got = calls(late, late_dy, handle)
    torch.cuda.default_stream().synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_stream_handles_of_torch_streams(gpu_lib):
    """A torch stream, its handle and an object that holds the handle are one
    stream; 2 (the calling thread's default stream) is passed on."""
    moe = gpu_lib
    st = torch.cuda.Stream()
    for s in (st, st.cuda_stream, Handle(st.cuda_stream)):
        with moe._on(s):
            assert torch.cuda.current_stream().cuda_stream == st.cuda_stream
    plain = torch.Stream(device="cuda")  # torch's stream of any device
    with moe._on(plain):
        assert torch.cuda.current_stream().stream_id == plain.stream_id
    with torch.cuda.stream(st), moe._on(0):
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
    with moe._on(2):
        assert torch.cuda.current_stream().cuda_stream == 2
    g = gen_of(22)
    x, w = rnd(g, 40, 64), rnd(g, 72, 64)
    want = moe.linear(x, w)
    torch.cuda.synchronize()
    y = moe.linear(x, w, stream=2)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


# ------------------------------------------------- activations, far tails
def test_gelu_lower_tail(gpu_lib):
    """GELU and its slope keep their relative accuracy where both fall off to
    zero: one rounding to bf16 (of the slope as an operand; dx repeats it), and
    2^-13 for the function: 5.6e-5 for the polynomial, 1.6e-5 for the exponential,
    whose argument is at most 122 and off by 3 * 2^-24 of itself (times ln 2), and
    a few 1e-7 for the special function unit.  The slope's terms cancel by
    1 / (z^2 - 1): below -3 that at most doubles their error."""
    moe = gpu_lib
    z = torch.linspace(-12.75, -3.0, 1280, device="cuda").to(BF).view(160, 8)
    eye = torch.eye(8, device="cuda").to(BF)
    z64 = z.double()
    cdf = torch.special.erfc(-z64 / math.sqrt(2)) / 2  # torch's ndtr is 0 below about -6 on this device
    val, slope = z64 * cdf, cdf + z64 * torch.exp(-z64 * z64 / 2) / math.sqrt(2 * math.pi)
    within(moe.linear(z, eye, act="gelu"), val, (U8 + (1 + U8) * 2.0 ** -13) * val.abs(), "gelu")
    h = moe.gated(z, eye, torch.zeros_like(eye), b_up=torch.ones(8, device="cuda"), act="gelu")
    within(h, val, (U8 + (1 + U8) * 2.0 ** -13) * val.abs(), "gated gelu")
    cfg, dx = moe.dense_config(160, 8, 8, "gelu"), torch.empty_like(z)
    moe.moe_linear_backward(cfg, torch.ones_like(z), z, eye, z, dx, None, None, moe.linear_backward_workspace(cfg))
    within(dx, slope, (U8 + (1 + U8) * 2.0 ** -12) * slope.abs(), "slope")


# --------------------------------------------------------- largest sizes
def test_more_than_two_to_the_30_columns(gpu_lib):
    """One row, 2^30 + 264 outputs (or inputs) of eight: every column."""
    moe, g = gpu_lib, gen_of(23)
    W, step = 2 ** 30 + 264, 2 ** 26
    w = torch.empty((W, 8), dtype=BF, device="cuda").normal_(generator=g)
    x = rnd(g, 1, 8)
    y = moe.linear(x, w)
    for c in range(0, W, step):
        v = w[c:c + step].double()
        ref, size = v @ x[0].double(), v.abs() @ x[0].double().abs()
        within(y[0, c:c + step], ref, U8 * ref.abs() + (1 + U8) * acc_tol(8) * size, f"y from {c}")
    del y
    w = w.view(8, W)
    x, dy = rnd(g, 1, W), rnd(g, 1, 8)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    cfg = moe.dense_config(1, W, 8, grad_dtype="bf16")
    ws = moe.linear_backward_workspace(cfg)
    moe.moe_linear_backward(cfg, dy, x, w, None, dx, dw, None, ws)
    for c in range(0, W, step):
        v = w[:, c:c + step].double()
        ref, size = dy[0].double() @ v, dy[0].double().abs() @ v.abs()
        within(dx[0, c:c + step], ref, U8 * ref.abs() + (1 + U8) * acc_tol(8) * size, f"dx from {c}")
        assert torch.equal(dw[:, c:c + step], (dy.float().t() * x[:, c:c + step].float()).to(BF)), f"d_w from {c}"
    assert moe.moe_dense_get_device_status(ws) == 0


# ------------------------------------------------------------ neighbours
def test_neighbours_and_in_place(gpu_lib):
    """Tensors that touch, end to start, are not an overlap; the norm's dx in
    place of x, of dy and of d_residual."""
    moe, g = gpu_lib, gen_of(24)
    T, K, N = 24, 64, 40

    def packed(*shapes, dtype=BF):
        sizes = [math.prod(s) for s in shapes]
        return [t.view(s) for t, s in zip(torch.empty(sum(sizes), dtype=dtype, device="cuda").split(sizes), shapes)]

    x, w, wu, res, y, z, u, dx, dw, dwu = packed((T, K), (N, K), (N, K), (T, N), (T, N), (T, N), (T, N), (T, K), (N, K),
                                                 (N, K))
    b, db, dbu = packed((N,), (N,), (N,), dtype=F32)
    for t in (x, w, wu, res, b):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
    cfg = moe.dense_config(T, K, N, "silu", grad_dtype="bf16")
    ws = moe._new_ws(max(moe.moe_gated_backward_workspace_size(cfg), moe.moe_linear_workspace_size(cfg)), "cuda")
    moe.moe_linear_forward(cfg, x, w, b, res, y, z, ws)
    assert torch.equal(y, moe.linear(x.clone(), w.clone(), b.clone(), res.clone(), "silu"))
    moe.moe_gated_forward(cfg, x, w, wu, b, None, y, z, u, ws)
    assert torch.equal(y, moe.gated(x.clone(), w.clone(), wu.clone(), b.clone()))
    moe.moe_gated_backward(cfg, res, x, w, wu, z, u, dx, dw, dwu, db, dbu, ws)
    own = [torch.empty_like(t) for t in (dx, dw, dwu, db, dbu)]
    moe.moe_gated_backward(cfg, res.clone(), x.clone(), w.clone(), wu.clone(), z.clone(), u.clone(), *own,
                           moe.gated_backward_workspace(cfg))
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, dwu, db, dbu), own))
    # rows of every ring form: one warp and several, two rows and one kept
    for T, H, dt in ((700, 264, BF), (700, 4104, BF), (300, 8200, F32), (200, 16384, F32)):
        x, dy, dr = (rnd(g, T, H, dtype=dt) for _ in range(3))
        mean, rstd = (torch.empty(T, device="cuda") for _ in range(2))
        moe.norm(x, mean_out=mean, rstd_out=rstd)
        cfg = moe.norm_config(T, H, dtype="bf16" if dt == BF else "f32")
        ws = moe.norm_workspace(cfg)

        def grads(x, dy, dr, dx):
            dw, db = (torch.empty(H, device="cuda") for _ in range(2))
            moe.moe_norm_backward(cfg, dy, x, None, mean, rstd, dr, dx, dw, db, ws)
            return dx, dw, db

        want = grads(x, dy, dr, torch.empty_like(x))
        for i in range(3):
            a = [x.clone(), dy.clone(), dr.clone()]
            assert all(torch.equal(p, q) for p, q in zip(grads(*a, a[i]), want)), (H, i)


# ------------------------------------- the weight gradient beside the other
@pytest.mark.parametrize("T,K,N", [(1, 2048, 768), (65, 2048, 768), (1000, 264, 136), (1500, 2048, 768),
                                   (3000, 520, 264)])
def test_operands_written_just_before(gpu_lib, T, K, N):
    """A weight gradient that starts beside the input gradient reads what the
    kernels before both have written: x by a norm chained in front, dg and du by
    the call's own first kernel.  The bits are those of calls with a wait in
    between, and each call leaves the workspace's header clear."""
    moe, g = gpu_lib, gen_of(T + K)
    rounds = 8
    src = [rnd(g, T, K) for _ in range(rounds)]
    w, wu, dy, u = rnd(g, N, K, scale=K ** -0.5), rnd(g, N, K, scale=K ** -0.5), rnd(g, T, N), rnd(g, T, N)
    ncfg, cfg = moe.norm_config(T, K, "rms"), moe.dense_config(T, K, N, "none")
    gcfg = moe.dense_config(T, K, N, "silu")
    ws = moe._new_ws(max(moe.moe_linear_backward_workspace_size(cfg), moe.moe_gated_backward_workspace_size(gcfg)),
                     "cuda")
    x = torch.empty_like(src[0])

    def step(i, wait):
        out = [torch.empty_like(x), torch.empty((N, K), device="cuda")]
        out += [torch.empty_like(x), torch.empty((N, K), device="cuda"), torch.empty((N, K), device="cuda")]
        for call in (lambda: moe.moe_norm_forward(ncfg, src[i], None, None, x),
                     lambda: moe.moe_linear_backward(cfg, dy, x, w, None, *out[:2], None, ws),
                     lambda: moe.moe_gated_backward(gcfg, dy, x, w, wu, dy, u, *out[2:], ws=ws)):
            call()
            if wait:
                torch.cuda.synchronize()
                assert (ws[:moe.DENSE_WS_HEADER] == 0).all()
        return out

    want = [step(i, True) for i in range(rounds)]
    for _ in range(4):
        got = [step(i, False) for i in range(rounds)]
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [step(i, False) for i in range(rounds)]
    for _ in range(2):
        graph.replay()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert (ws[:moe.DENSE_WS_HEADER] == 0).all()


# -------------------------------------------- rings used again and again
# more rows per group of warps than its ring has slots, and then some: the slots
# are filled again and their barriers change phase, at every number of warps per row
@pytest.mark.parametrize("T,H,kind,dt", [(24000, 512, "layer", BF), (20000, 264, "rms", F32), (12000, 1024, "rms", BF),
                                         (8000, 2056, "layer", BF), (4000, 2880, "rms", BF), (2500, 4104, "layer", F32),
                                         (1300, 8200, "layer", BF), (1300, 16384, "rms", BF), (800, 16384, "layer", F32)])
def test_norm_of_many_rows(gpu_lib, T, H, kind, dt):
    check_norm_forward(gpu_lib, T, H, kind, dt, "wb")
    check_norm_backward(gpu_lib, T, H, kind, dt, False, False)
    check_norm_backward(gpu_lib, T, H, kind, dt, True, True)


# ------------------------------------------------- the form a product takes
def kernels(moe, call):
    """Names of the kernels that a call launches."""
    moe.moe_trace_begin(64)
    call()
    return [name for name, _ in moe.moe_trace_end()]


def form_of(moe, op, T, K, N):
    x, w = torch.zeros((T, K), dtype=BF, device="cuda"), torch.zeros((N, K), dtype=BF, device="cuda")
    return kernels(moe, (lambda: moe.linear(x, w)) if op == "linear" else (lambda: moe.gated(x, w, w)))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,K,N,split", [(2000, 1000, 1016, False), (4000, 520, 1288, False), (700, 2880, 5000, False),
                                         (1030, 3200, 4104, True)])
def test_linear_of_many_rows(gpu_lib, T, K, N, split, act):
    """Tiles of 128 and of 256 columns, ragged on both sides; tiles split along
    the reduction."""
    assert form_of(gpu_lib, "linear", T, K, N) == ["linear_fwd"]
    cfg = gpu_lib.dense_config(T, K, N)
    assert (gpu_lib.moe_linear_workspace_size(cfg) > gpu_lib.DENSE_WS_HEADER) == split
    check_linear_forward(gpu_lib, T, K, N, act)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,K,N,form,split", [
    (2000, 328, 1000, "gated_fwd", False), (2600, 136, 1032, "gated_fwd", False), (1500, 4104, 2056, "gated_fwd", True),
    (129, 264, 1032, "gated_fwd_skinny", False), (17, 2048, 520, "gated_fwd_skinny", False)])
def test_gated_forms(gpu_lib, T, K, N, form, split, act):
    """Every activation in both forms of the gate/up kernel."""
    assert form_of(gpu_lib, "gated", T, K, N) == [form]
    cfg = gpu_lib.dense_config(T, K, N, act)
    assert (gpu_lib.moe_gated_workspace_size(cfg) > gpu_lib.DENSE_WS_HEADER) == split
    check_gated_forward(gpu_lib, T, K, N, act)


@pytest.mark.parametrize("T,K,N,names", [
    (65, 2048, 768, ["gated_dgu", "gated_dgrad_skinny", "gated_wgrad"]),
    (1000, 264, 136, ["gated_dgu", "gated_dgrad_skinny", "gated_wgrad", "wgrad_sum"]),
    (2000, 2048, 768, ["gated_dgu", "gated_dgrad", "gated_wgrad"]),
    (2000, 520, 264, ["gated_dgu", "gated_dgrad", "gated_wgrad", "wgrad_sum"])])
def test_gated_backward_forms(gpu_lib, T, K, N, names):
    moe, g = gpu_lib, gen_of(25)
    cfg = moe.dense_config(T, K, N, "gelu")
    t, w = rnd(g, T, N), rnd(g, N, K)
    dw = [torch.empty((N, K), device="cuda") for _ in range(2)]
    ws = moe.gated_backward_workspace(cfg)
    x = rnd(g, T, K)
    assert kernels(moe, lambda: moe.moe_gated_backward(cfg, t, x, w, w, t, t, torch.empty_like(x), *dw, ws=ws)) == names
    check_gated_backward(moe, T, K, N, "gelu", "f32")


@pytest.mark.parametrize("T,K,N,names", [
    (1000, 264, 136, ["linear_dz", "linear_dgrad_skinny", "linear_wgrad", "wgrad_sum"]),
    (1500, 2048, 768, ["linear_dz", "linear_dgrad", "linear_wgrad"]),
    (3000, 520, 264, ["linear_dz", "linear_dgrad", "linear_wgrad", "wgrad_sum"])])
def test_linear_backward_forms(gpu_lib, T, K, N, names):
    moe, g = gpu_lib, gen_of(27)
    cfg = moe.dense_config(T, K, N, "silu")
    x, t, w, dw = rnd(g, T, K), rnd(g, T, N), rnd(g, N, K), torch.empty((N, K), device="cuda")
    ws = moe.linear_backward_workspace(cfg)
    assert kernels(moe, lambda: moe.moe_linear_backward(cfg, t, x, w, t, torch.empty_like(x), dw, None, ws)) == names
    check_linear_backward(moe, T, K, N, "silu", "f32")


def test_one_workspace_for_split_products(gpu_lib):
    """Calls whose tiles are split 2, 3 and 8 ways, on different numbers of
    tiles, one after another in one workspace: the counters of each are back at
    zero when it ends, and its bits are those of a workspace of its own."""
    moe, g = gpu_lib, gen_of(26)
    calls = []

    def operands(T, K, N):
        return (rnd(g, T, K), *(rnd(g, N, K, scale=K ** -0.5) for _ in range(2)), *(rnd(g, T, N) for _ in range(3)))

    for T, K, N in ((1500, 2880, 3304), (300, 18432, 4944), (1030, 3200, 4104)):
        x, w, _, _, _, res = operands(T, K, N)
        cfg = moe.dense_config(T, K, N)
        assert form_of(moe, "linear", T, K, N) == ["linear_fwd"]
        calls.append((moe.moe_linear_workspace_size(cfg),
                      lambda ws, x=x, w=w, res=res: [moe.linear(x, w, None, res, "silu", ws=ws)]))
    for T, K, N in ((1500, 4104, 2056), (1030, 3200, 2056)):
        x, w, wu, _, _, _ = operands(T, K, N)
        assert form_of(moe, "gated", T, K, N) == ["gated_fwd"]
        calls.append((moe.moe_gated_workspace_size(moe.dense_config(T, K, N, "silu")),
                      lambda ws, x=x, w=w, wu=wu: [moe.gated(x, w, wu, ws=ws)]))
    for T, K, N in ((1030, 4104, 2056), (2000, 2880, 2880)):
        x, w, wu, dh, gg, u = operands(T, K, N)
        cfg = moe.dense_config(T, K, N, "silu", grad_dtype="bf16")

        def backward(ws, cfg=cfg, x=x, w=w, wu=wu, dh=dh, gg=gg, u=u):
            out = [torch.empty_like(t) for t in (x, w, wu)]
            moe.moe_gated_backward(cfg, dh, x, w, wu, gg, u, *out, ws=ws)
            return out

        calls.append((moe.moe_gated_backward_workspace_size(cfg), backward))
        names = kernels(moe, lambda: backward(moe.gated_backward_workspace(cfg)))
        assert "gated_dgrad" in names and "gated_dgrad_skinny" not in names
    assert all(n > moe.DENSE_WS_HEADER for n, _ in calls)
    want = [call(moe._new_ws(n, "cuda")) for n, call in calls]
    ws = moe._new_ws(max(n for n, _ in calls), "cuda")
    for order in (range(len(calls)), reversed(range(len(calls)))):
        for i in order:
            got = calls[i][1](ws)
            assert (ws[:moe.DENSE_WS_HEADER] == 0).all(), i
            assert all(torch.equal(p, q) for p, q in zip(got, want[i])), i


# ---------------------------------------------------- long reductions, normwise
@pytest.mark.parametrize("T,K,N", [(300, 18432, 4944), (33, 16392, 264), (2100, 264, 16392), (40, 136, 16392),
                                   (20000, 264, 136), (16391, 72, 520)])
def test_long_reductions_normwise(gpu_lib, T, K, N):
    """The whole tensor's error over its norm, where one element's bound is wide.
    Step j of a reduction of n = K / 16 steps is off by at most 17 units of 2^-23 of
    the sum so far, of norm sqrt(j / n) of the result's for independent terms
    (on average 2/3), and of its own 16 terms' sizes (under 0.43 of it from 64 steps
    on): 17 * 2^-23 * n * 1.1 in all, and the rounding's 2^-8.  One 64-deep step left
    out of 18432 would be 0.059."""
    moe, g = gpu_lib, gen_of(T + K + N)
    x, w, dy = rnd(g, T, K), rnd(g, N, K, scale=K ** -0.5), rnd(g, T, N)

    def close(got, ref, depth, what):
        err = (got.double() - ref).norm() / ref.norm()
        assert err <= U8 + 17 * 2.0 ** -23 * max(depth / 16, 1) * 1.1, (what, float(err))

    u = torch.empty_like(dy)
    close(moe.linear(x, w), x.double() @ w.double().t(), K, "y")
    moe.gated(x, w, w, act="none", u_out=u)
    close(u, x.double() @ w.double().t(), K, "u")
    cfg, dx, dw = moe.dense_config(T, K, N), torch.empty_like(x), torch.empty((N, K), device="cuda")
    moe.moe_linear_backward(cfg, dy, x, w, None, dx, dw, None, moe.linear_backward_workspace(cfg))
    close(dx, dy.double() @ w.double(), N, "dx")
    close(dw, dy.double().t() @ x.double(), T, "d_w")
