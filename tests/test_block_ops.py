"""The operators around the routed layer on the GPU (moe_norm_*, moe_linear_*,
moe_gated_*), element by element against their formulas in float64 on the
exact input values.

Tolerances, per element, before any run:
  * one rounding to bf16: 2^-8 of the value (half a step, finfo.eps / 2), to
    float32 2^-24;
  * a tensor-core sum of K products: 17 * 2^-23 * (K / 16 + 8) * sum |a b|
    (16 exact products per step, each step's additions off by at most 17
    units of 2^-23 of what is added; 8 more steps for split sums);
  * an activation's argument error times 1.13 (the largest slope of any of
    them), plus 2^-19 (1 + |z|) for the function itself (the exponential's
    argument carries |z| 2^-24 relative error, its value a few 2^-22);
  * an operand rounded to bf16 before a product (dz, dg, du): 2^-8 of each
    term's size, summed;
  * a norm's statistics: sums of H float32 terms, at most 48 additions deep
    (32 per thread, the rest in trees), so 64 * 2^-24 of the sum of the terms'
    sizes leaves room for the elementwise steps.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U8, U24 = 2.0 ** -8, 2.0 ** -24
ACTS = ("none", "silu", "gelu", "gelu_tanh", "relu")


def acc_tol(K):
    return 17 * 2.0 ** -23 * (K / 16 + 8)


def act64(a, z):
    if a == "none":
        return z, torch.ones_like(z)
    if a == "relu":
        return z.clamp(min=0), (z > 0).double()
    if a == "silu":
        p = torch.sigmoid(z)
        return z * p, p * (1 + z * torch.sigmoid(-z))
    if a == "gelu":
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    q = math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)
    p = torch.sigmoid(q)
    return z * p, p + z * p * torch.sigmoid(-q) * math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * z * z)


def within(got, ref, tol, what):
    d = (got.double() - ref).abs()
    bad = ~(d <= tol)
    if bad.any():
        i = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first {i}: got {got[tuple(i)]} "
                             f"want {ref[tuple(i)]} tol {tol[tuple(i)]}")


def rnd(gen, *shape, scale=1.0, dtype=BF, shift=0.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale + shift).to(dtype)


def gen_of(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def guarded(T, N, dtype=BF, rows=3):
    """[T, N] view of a larger buffer whose rows behind the last are a canary."""
    big = torch.full((T + rows, N), 7.0, dtype=dtype, device="cuda")
    return big[:T], big


def canary_intact(big, T):
    return bool((big[T:].float() == 7.0).all())


# ----------------------------------------------------------------- norm
NORM = [(1, 8, "layer", F32), (3, 8, "rms", BF), (5, 264, "layer", BF), (9, 520, "rms", F32), (17, 1024, "layer", BF),
        (2, 1032, "layer", F32), (33, 2056, "rms", BF), (65, 2880, "layer", BF), (700, 512, "layer", BF),
        (613, 4104, "rms", F32), (7, 8200, "layer", BF), (3, 16384, "layer", F32), (2, 16384, "rms", BF)]


def norm64(x, w, b, kind, eps):
    x = x.double()
    mu = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    r = ((x - mu) ** 2).mean(1, keepdim=True).add(eps).rsqrt()
    xh = (x - mu) * r
    y = xh if w is None else xh * w.double()
    return y if b is None else y + b.double(), mu, r, xh


@pytest.mark.parametrize("affine", ["wb", "w", ""])
@pytest.mark.parametrize("T,H,kind,dt", NORM)
def test_norm_forward(gpu_lib, T, H, kind, dt, affine):
    moe, g = gpu_lib, gen_of(T * 31 + H)
    x = rnd(g, T, H, scale=1.5, dtype=dt, shift=0.3)
    x[-1] += 40.0  # a row far from zero: its variance must not be lost in its mean
    w = rnd(g, H, scale=0.1, dtype=F32, shift=1.0) if "w" in affine else None
    b = rnd(g, H, dtype=F32) if "b" in affine else None
    y, big = guarded(T, H, dt)
    mean, rstd = (torch.full((T,), 5.0, device="cuda") for _ in range(2))
    cfg = moe.norm_config(T, H, kind, 1e-5, "bf16" if dt == BF else "f32")
    moe.moe_norm_forward(cfg, x, w, b, y, mean, rstd)
    ref, mu, r, xh = norm64(x, w, b, kind, 1e-5)
    ws = 1.0 if w is None else w.double().abs()
    e_mu = 64 * U24 * x.double().abs().mean(1, keepdim=True) if kind == "layer" else 0 * r
    # relative error of r: half that of the mean square, whose terms err by 2 e_mu |x - mu|
    e_r = 64 * U24 + e_mu * r
    # xh's own terms err by the difference's rounding (2^-24 of |x| + |mu|) and by e_mu
    e_xh = (4 * U24 * (x.double().abs() + mu.abs()) + e_mu) * r + xh.abs() * e_r
    tol = (U8 if dt == BF else 2 * U24) * ref.abs() + ws * e_xh * (1 + U8) + 4 * U24 * (0 if b is None else b.abs())
    within(y, ref, tol, "y")
    within(rstd, r[:, 0], (e_r + U24)[:, 0] * r[:, 0], "rstd")
    if kind == "layer":
        within(mean, mu[:, 0], e_mu[:, 0], "mean")
    else:
        assert (mean == 5.0).all(), "the RMS form has no mean to write"
    assert canary_intact(big, T)


@pytest.mark.parametrize("dyf,res", [(False, False), (True, True)])
@pytest.mark.parametrize("T,H,kind,dt", NORM)
def test_norm_backward(gpu_lib, T, H, kind, dt, dyf, res):
    moe, g = gpu_lib, gen_of(T * 37 + H)
    gt = F32 if dyf or dt == F32 else BF
    x = rnd(g, T, H, scale=1.5, dtype=dt, shift=0.3)
    w = rnd(g, H, scale=0.1, dtype=F32, shift=1.0) if T != 9 else None
    dy = rnd(g, T, H, dtype=gt)
    d_res = rnd(g, T, H, dtype=dt) if res else None
    _, mu, r, _ = norm64(x, None, None, kind, 1e-5)
    mean, rstd = mu[:, 0].float(), r[:, 0].float()
    cfg = moe.norm_config(T, H, kind, 1e-5, "bf16" if dt == BF else "f32", "f32" if gt == F32 else "bf16")
    dx, big = guarded(T, H, dt)
    dw, db = (torch.full((H,), float("nan"), device="cuda") for _ in range(2))
    ws = moe.norm_workspace(cfg)
    moe.moe_norm_backward(cfg, dy, x, w, mean if kind == "layer" else None, rstd, d_res, dx, dw, db, ws)
    mu, r = (mean.double()[:, None] if kind == "layer" else 0 * r), rstd.double()[:, None]
    xa, d = x.double().abs() + mu.abs(), dy.double()
    xh = (x.double() - mu) * r
    a = d if w is None else d * w.double()
    m1 = a.mean(1, keepdim=True) if kind == "layer" else 0 * r
    m2 = (a * xh).mean(1, keepdim=True)
    ref = r * (a - m1 - xh * m2)
    if res:
        ref = ref + d_res.double()
    e_xh = 3 * U24 * xa * r
    am = a.abs().mean(1, keepdim=True)
    e_m2 = 64 * U24 * (a.abs() * xa * r).mean(1, keepdim=True)
    tol = (U8 if dt == BF else 2 * U24) * ref.abs() + (1 + U8) * r * (
        4 * U24 * (a.abs() + m1.abs() + (xh * m2).abs()) + 64 * U24 * am + xh.abs() * e_m2 + e_xh * m2.abs())
    if res:
        tol = tol + 2 * U24 * d_res.double().abs()
    within(dx, ref, tol, "dx")
    depth = T / 64 + 64  # rows of a CTA in turn, then at most 592 / 32 partials and a tree
    within(dw, (d * xh).sum(0), depth * U24 * (d.abs() * xa * r).sum(0), "d_weight")
    within(db, d.sum(0), depth * U24 * d.abs().sum(0) + 1e-30, "d_bias")
    assert canary_intact(big, T)
    # skipping the weight gradients changes nothing else
    dx2 = torch.empty_like(dx)
    moe.moe_norm_backward(cfg, dy, x, w, mean if kind == "layer" else None, rstd, d_res, dx2, None, None, ws)
    assert torch.equal(dx2, dx)


def test_norm_in_place_and_constant_rows(gpu_lib):
    """y = x in place, dx in place of d_residual; a constant row has xh = 0."""
    moe, g = gpu_lib, gen_of(3)
    x = rnd(g, 40, 256)
    x[7] = 3.0
    w, b = rnd(g, 256, dtype=F32), rnd(g, 256, dtype=F32)
    y = moe.norm(x, w, b)
    assert torch.equal(y[7], b.to(BF))
    x2 = x.clone()
    moe.moe_norm_forward(moe.norm_config(40, 256), x2, w, b, x2)
    assert torch.equal(x2, y)
    cfg = moe.norm_config(40, 256, "rms")
    _, _, r, _ = norm64(x, None, None, "rms", 1e-5)
    dy, dr, dx = rnd(g, 40, 256), rnd(g, 40, 256), torch.empty_like(x)
    rstd, dw, ws = r[:, 0].float(), torch.empty(256, device="cuda"), moe.norm_workspace(cfg)
    moe.moe_norm_backward(cfg, dy, x, w, None, rstd, dr, dx, dw, None, ws)
    dr2 = dr.clone()
    moe.moe_norm_backward(cfg, dy, x, w, None, rstd, dr2, dr2, dw, None, ws)
    assert torch.equal(dr2, dx)
    dy2 = dy.clone()
    moe.moe_norm_backward(cfg, dy2, x, w, None, rstd, dr, dy2, dw, None, ws)
    assert torch.equal(dy2, dx)


# ----------------------------------------------------------------- linear
# rows from one to several 256-row tiles, ragged K and N, more tiles than pairs
# (4000 x 1288), split and whole tiles, the few-row kernel's split and unsplit clusters
LIN = [(1, 64, 8), (1, 4096, 264), (5, 72, 136), (16, 520, 128), (17, 2048, 520), (129, 200, 1032), (256, 72, 264),
       (257, 1032, 264), (300, 8, 520), (513, 64, 72), (700, 328, 1000), (2200, 72, 2040), (4000, 648, 1288)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,K,N", LIN)
def test_linear_forward(gpu_lib, T, K, N, act):
    moe, g = gpu_lib, gen_of(T + K + N)
    x, w = rnd(g, T, K), rnd(g, N, K, scale=2 * K ** -0.5)
    b, res = rnd(g, N, dtype=F32), rnd(g, T, N)
    z64 = x.double() @ w.double().t()
    S = acc_tol(K) * (x.double().abs() @ w.double().abs().t())
    cfg = moe.dense_config(T, K, N, act)
    ws = moe.linear_workspace(cfg)
    for use_b, use_r, keep in ((False, False, False), (True, True, True), (True, False, True), (False, True, False)):
        y, big = guarded(T, N)
        zo, zbig = guarded(T, N)
        moe.moe_linear_forward(cfg, x, w, b if use_b else None, res if use_r else None, y, zo if keep else None, ws)
        z = z64 + b.double() if use_b else z64
        e = S + 4 * U24 * z.abs()
        a = act64(act, z)[0]
        ref = a + res.double() if use_r else a
        ea = 1.13 * e + (0 if act in ("none", "relu") else 2.0 ** -19 * (1 + z.abs()))
        within(y, ref, U8 * ref.abs() + (1 + U8) * (ea + 2 * U24 * a.abs()), f"y b={use_b} r={use_r}")
        if keep:
            within(zo, z, U8 * z.abs() + (1 + U8) * e, "z")
        else:
            assert (zbig == 7.0).all()
        assert canary_intact(big, T) and canary_intact(zbig, T)
    r2 = res.clone()  # in place of the residual
    moe.moe_linear_forward(cfg, x, w, None, r2, r2, None, ws)
    assert torch.equal(r2, y)
    assert moe.moe_dense_get_device_status(ws) == 0


# Fewer tiles than CTA pairs: narrow tiles, whole and ragged ones.
@pytest.mark.parametrize("T,K,N", [(2048, 1024, 1024), (1500, 1000, 1016), (600, 4096, 3304)])
def test_linear_forward_few_tiles(gpu_lib, T, K, N):
    test_linear_forward(gpu_lib, T, K, N, "gelu_tanh")


# The last wave's tiles split along the reduction, and added in the kernel.
@pytest.mark.parametrize("T,K,N", [(1500, 2880, 3304), (1030, 3200, 4104), (300, 18432, 4944)])
def test_linear_forward_split_tiles(gpu_lib, T, K, N):
    moe = gpu_lib
    assert moe.moe_linear_workspace_size(moe.dense_config(T, K, N)) > moe.DENSE_WS_HEADER
    test_linear_forward(moe, T, K, N, "silu")


LIN_BWD = [(1, 64, 8, "silu"), (1, 264, 4096, "none"), (7, 136, 72, "gelu"), (64, 520, 264, "relu"),
           (65, 72, 200, "gelu_tanh"), (257, 264, 136, "none"), (300, 2040, 72, "silu"), (72, 2040, 2200, "none"),
           (2100, 264, 328, "gelu"), (5000, 72, 136, "none"), (1031, 520, 8, "silu"), (2200, 2040, 72, "none"),
           (4000, 1288, 328, "silu")]


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,N,act", LIN_BWD)
def test_linear_backward(gpu_lib, T, K, N, act, grad):
    moe, g = gpu_lib, gen_of(T + 3 * K + N)
    x, w, dy = rnd(g, T, K), rnd(g, N, K, scale=K ** -0.5), rnd(g, T, N)
    z = rnd(g, T, N, scale=2.0) if act != "none" else None
    cfg = moe.dense_config(T, K, N, act, grad_dtype=grad)
    ws = moe.linear_backward_workspace(cfg)
    gt = F32 if grad == "f32" else BF
    dx, big = guarded(T, K)
    dw, wbig = guarded(N, K, gt)
    db = torch.full((N,), float("nan"), device="cuda")
    moe.moe_linear_backward(cfg, dy, x, w, z, dx, dw, db, ws)
    s = torch.ones_like(dy.double()) if z is None else act64(act, z.double())[1]
    dz = dy.double() * s
    # the slope's own error, then the rounding to bf16 of the operand
    e_f = 0 * dz if act in ("none", "relu") else dy.double().abs() * 2.0 ** -18
    e_z = e_f + (0 if act == "none" else U8) * dz.abs()
    ref = dz @ w.double()
    within(dx, ref, U8 * ref.abs() + (1 + U8) * ((e_z + acc_tol(N) * dz.abs()) @ w.double().abs()), "dx")
    ref = dz.t() @ x.double()
    t = (e_z + acc_tol(T) * dz.abs()).t() @ x.double().abs()
    dw_ref, dw_tol = ref, (U8 if gt == BF else U24) * ref.abs() + (1 + U8) * t
    within(dw, dw_ref, dw_tol, "d_w")
    within(db, dz.sum(0), e_f.sum(0) + (T / 8 + 64) * U24 * dz.abs().sum(0), "d_bias")
    assert canary_intact(big, T) and canary_intact(wbig, N)
    # each output alone: the bias gradient has the same bits; the forms of the
    # two products may follow from whether they run side by side
    dx2, dw2, db2 = torch.empty_like(dx), torch.empty_like(dw), torch.empty_like(db)
    moe.moe_linear_backward(cfg, dy, None, w, z, dx2, None, None, ws)
    moe.moe_linear_backward(cfg, dy, x, None, z, None, dw2, None, ws)
    moe.moe_linear_backward(cfg, dy, None, None, z, None, None, db2, ws)
    assert torch.equal(db2, db)
    within(dw2, dw_ref, dw_tol, "d_w alone")
    ref = dz @ w.double()
    within(dx2, ref, U8 * ref.abs() + (1 + U8) * ((e_z + acc_tol(N) * dz.abs()) @ w.double().abs()), "dx alone")
    assert moe.moe_dense_get_device_status(ws) == 0


# ----------------------------------------------------------------- gated
def test_linear_backward_split_tiles(gpu_lib):
    test_linear_backward(gpu_lib, 1500, 4104, 4096, "none", "bf16")


GATED = [(1, 64, 8), (1, 1024, 264), (6, 72, 136), (17, 520, 128), (128, 200, 328), (129, 264, 1032), (256, 72, 72),
         (257, 1032, 136), (300, 8, 520), (700, 328, 1000)]


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "none"])
@pytest.mark.parametrize("T,K,N", GATED)
def test_gated_forward(gpu_lib, T, K, N, act):
    moe, gen = gpu_lib, gen_of(T + K + 5 * N)
    x = rnd(gen, T, K)
    wg, wu = (rnd(gen, N, K, scale=2 * K ** -0.5) for _ in range(2))
    bg, bu = (rnd(gen, N, dtype=F32) for _ in range(2))
    cfg = moe.dense_config(T, K, N, act)
    ws = moe.gated_workspace(cfg)
    first = None
    for use_b, kg, ku in ((False, False, False), (True, True, True), (False, True, False), (True, False, True)):
        h, hbig = guarded(T, N)
        go, gbig = guarded(T, N)
        uo, ubig = guarded(T, N)
        moe.moe_gated_forward(cfg, x, wg, wu, bg if use_b else None, bu if use_b else None, h, go if kg else None,
                              uo if ku else None, ws)
        g, u = (x.double() @ v.double().t() + (b.double() if use_b else 0) for v, b in ((wg, bg), (wu, bu)))
        eg, eu = (acc_tol(K) * (x.double().abs() @ v.double().abs().t()) + 4 * U24 * p.abs()
                  for v, p in ((wg, g), (wu, u)))
        a = act64(act, g)[0]
        ea = 1.13 * eg + (0 if act == "none" else 2.0 ** -19 * (1 + g.abs()))
        ref = a * u
        within(h, ref, U8 * ref.abs() + (1 + U8) * (ea * (u.abs() + eu) + a.abs() * eu + 2 * U24 * ref.abs()), "h")
        for keep, o, big, p, e, what in ((kg, go, gbig, g, eg, "g"), (ku, uo, ubig, u, eu, "u")):
            if keep:
                within(o, p, U8 * p.abs() + (1 + U8) * e, what)
                assert canary_intact(big, T)
            else:
                assert (big == 7.0).all()
        assert canary_intact(hbig, T)
        if first is None:
            first = h
        elif not use_b:
            assert torch.equal(first, h), "keeping g changes h"
    assert moe.moe_dense_get_device_status(ws) == 0


def test_gated_forward_split_tiles(gpu_lib):
    moe = gpu_lib
    T, K, N = 1030, 3200, 2056
    assert moe.moe_gated_workspace_size(moe.dense_config(T, K, N)) > moe.DENSE_WS_HEADER
    test_gated_forward(moe, T, K, N, "silu")


GATED_BWD = [(1, 64, 8, "silu"), (3, 4096, 264, "silu"), (65, 264, 72, "gelu"), (256, 136, 520, "relu"),
             (257, 264, 136, "silu"), (300, 72, 1000, "silu"), (300, 2040, 72, "gelu_tanh"), (72, 1032, 2200, "none"), (2100, 200, 328, "silu"),
             (4200, 72, 136, "silu")]


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,N,act", GATED_BWD)
def test_gated_backward(gpu_lib, T, K, N, act, grad):
    moe, gen = gpu_lib, gen_of(T + 7 * K + N)
    x = rnd(gen, T, K)
    wg, wu = (rnd(gen, N, K, scale=K ** -0.5) for _ in range(2))
    dh, g, u = rnd(gen, T, N), rnd(gen, T, N, scale=2.0), rnd(gen, T, N)
    cfg = moe.dense_config(T, K, N, act, grad_dtype=grad)
    ws = moe.gated_backward_workspace(cfg)
    gt = F32 if grad == "f32" else BF
    dx, big = guarded(T, K)
    (dwg, gbig), (dwu, ubig) = guarded(N, K, gt), guarded(N, K, gt)
    dbg, dbu = (torch.full((N,), float("nan"), device="cuda") for _ in range(2))
    moe.moe_gated_backward(cfg, dh, x, wg, wu, g, u, dx, dwg, dwu, dbg, dbu, ws)
    a, s = act64(act, g.double())
    d, du64 = dh.double() * s * u.double(), dh.double() * a
    fn = 0 if act in ("none", "relu") else 2.0 ** -18
    fg = fn * (dh.double() * u.double()).abs() + 4 * U24 * d.abs()
    fu = fn * dh.double().abs() * (1 + g.double().abs()) + 4 * U24 * du64.abs()
    eg, eu = fg + U8 * d.abs(), fu + U8 * du64.abs()
    ref = d @ wg.double() + du64 @ wu.double()
    t = (eg + acc_tol(2 * N) * d.abs()) @ wg.double().abs() + (eu + acc_tol(2 * N) * du64.abs()) @ wu.double().abs()
    dx_ref, dx_tol = ref, U8 * ref.abs() + (1 + U8) * t
    within(dx, dx_ref, dx_tol, "dx")
    for got, p, e, what in ((dwg, d, eg, "d_w_gate"), (dwu, du64, eu, "d_w_up")):
        ref = p.t() @ x.double()
        t = (e + acc_tol(T) * p.abs()).t() @ x.double().abs()
        within(got, ref, (U8 if gt == BF else U24) * ref.abs() + (1 + U8) * t, what)
    for got, p, e, what in ((dbg, d, fg, "d_b_gate"), (dbu, du64, fu, "d_b_up")):
        within(got, p.sum(0), e.sum(0) + (T / 8 + 64) * U24 * p.abs().sum(0), what)
    assert canary_intact(big, T) and canary_intact(gbig, N) and canary_intact(ubig, N)
    dbu2, dx2 = torch.empty_like(dbu), torch.empty_like(dx)
    moe.moe_gated_backward(cfg, dh, None, None, None, g, u, None, None, None, None, dbu2, ws)
    moe.moe_gated_backward(cfg, dh, None, wg, wu, g, u, dx2, None, None, ws=ws)
    assert torch.equal(dbu2, dbu)
    within(dx2, dx_ref, dx_tol, "dx alone")
    assert moe.moe_dense_get_device_status(ws) == 0


def test_gated_backward_split_tiles(gpu_lib):
    test_gated_backward(gpu_lib, 1030, 4104, 2056, "silu", "f32")


# ----------------------------------------------------- activations far out
@pytest.mark.parametrize("act", ACTS)
def test_activations_at_large_arguments(gpu_lib, act):
    """Values and slopes far from zero are those of the limits, with no NaN
    from an overflowing intermediate; a NaN stays one."""
    moe = gpu_lib
    z = torch.tensor([[-1e30, -300.0, -88.0, -20.0, 0.0, 20.0, 300.0, 1e30]], device="cuda").to(BF)
    eye = torch.eye(8, device="cuda").to(BF)
    y = moe.linear(z, eye, act=act)
    want, slope = act64(act, z.double().clamp(-1e9, 1e9))
    within(y, torch.where(z.double() > 1e9, z.double(), torch.where((z.double() < -1e9) & (act != "none"), 0.0,
                                                                    z.double() if act == "none" else want)),
           U8 * z.double().abs() * (z > 0) + 1e-6 + (U8 * z.double().abs() if act == "none" else 0), "value")
    cfg = moe.dense_config(1, 8, 8, act)
    dx = torch.empty_like(z)
    moe.moe_linear_backward(cfg, torch.ones_like(z), z, eye, z if act != "none" else None, dx, None, None,
                            moe.linear_backward_workspace(cfg))
    lim = torch.where(z > 100, 1.0, torch.where((z < -100) & (act != "none"), 0.0, slope if act != "none" else 1.0))
    within(dx, lim.double(), U8 * lim.double().abs() + 1e-6, "slope")
    nan = z.clone()
    nan[0, 2] = float("nan")
    assert moe.linear(nan, eye, act=act).isnan().all()  # every output sums 0 * NaN


# ------------------------------------------------------------ zero rows
def test_zero_rows(gpu_lib):
    """T = 0: nothing to write but weight gradients of exactly zero."""
    moe = gpu_lib
    e = lambda n: torch.empty((0, n), dtype=BF, device="cuda")
    nan = lambda *s: torch.full(s, float("nan"), device="cuda")
    w = torch.ones((16, 8), dtype=BF, device="cuda")
    assert moe.linear(e(8), w).shape == (0, 16) and moe.gated(e(8), w, w).shape == (0, 16)
    assert moe.norm(e(8)).shape == (0, 8)
    cfg = moe.dense_config(0, 8, 16, "silu")
    outs = [nan(16, 8), nan(16, 8), nan(16), nan(16)]
    moe.moe_gated_backward(cfg, e(16), e(8), w, w, e(16), e(16), e(8), *outs, moe.gated_backward_workspace(cfg))
    dw, db = nan(16, 8), nan(16)
    moe.moe_linear_backward(cfg, e(16), e(8), w, e(16), e(8), dw, db, moe.linear_backward_workspace(cfg))
    ncfg = moe.norm_config(0, 8)
    nw, nb, st = nan(8), nan(8), torch.empty(0, device="cuda")
    moe.moe_norm_backward(ncfg, e(8), e(8), None, st, st, None, e(8), nw, nb, moe.norm_workspace(ncfg))
    for t in outs + [dw, db, nw, nb]:
        assert (t == 0).all()


# ------------------------------------------- streams, graphs, devices, runs
def test_repeatable_and_other_stream(gpu_lib):
    """The same bits again, and on a stream other than the current one."""
    moe, g = gpu_lib, gen_of(11)
    x, w, wu = rnd(g, 300, 520), rnd(g, 264, 520, scale=0.05), rnd(g, 264, 520, scale=0.05)
    few = x[:9].clone()
    a = moe.gated(x, w, wu)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    b = moe.gated(x, w, wu, stream=st)
    y = moe.linear(few, w, stream=st)
    st.synchronize()
    assert torch.equal(a, b) and torch.equal(a, moe.gated(x, w, wu))
    assert torch.equal(y, moe.linear(few, w))


def test_captured_and_replayed(gpu_lib):
    """Forward and backward in a CUDA graph, replayed on new input values."""
    moe, g = gpu_lib, gen_of(12)
    T, K, N = 300, 264, 136
    x, w, dy = rnd(g, T, K), rnd(g, N, K, scale=0.06), rnd(g, T, N)
    cfg = moe.dense_config(T, K, N, "gelu")
    wf, wb = moe.linear_workspace(cfg), moe.linear_backward_workspace(cfg)
    y, z, dx = torch.empty_like(dy), torch.empty_like(dy), torch.empty_like(x)
    dw, db = torch.empty((N, K), device="cuda"), torch.empty(N, device="cuda")

    def step():
        moe.moe_linear_forward(cfg, x, w, db, None, y, z, wf)
        moe.moe_linear_backward(cfg, dy, x, w, z, dx, dw, db, wb)

    db.zero_()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        x.copy_(rnd(gen_of(seed), T, K))
        db.zero_()
        graph.replay()
        got = [t.clone() for t in (y, z, dx, dw, db)]
        db.zero_()
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (y, z, dx, dw, db)))
    assert moe.moe_dense_get_device_status(wf) == 0 and moe.moe_dense_get_device_status(wb) == 0


def test_two_streams_at_once(gpu_lib):
    """The same products on two streams at the same time, each with its own
    workspace: split tiles (wgrad of 5000 rows), clusters and rings side by side."""
    moe, g = gpu_lib, gen_of(13)
    T, K, N = 5000, 72, 136
    x, w, dy = rnd(g, T, K), rnd(g, N, K, scale=0.1), rnd(g, T, N)
    cfg = moe.dense_config(T, K, N)
    run = []
    for _ in range(2):
        run.append((torch.cuda.Stream(), moe.linear_backward_workspace(cfg), torch.empty_like(x),
                    torch.empty((N, K), device="cuda"), torch.empty(N, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(20):
        for st, ws, dx, dw, db in run:
            moe.moe_linear_backward(cfg, dy, x, w, None, dx, dw, db, ws, stream=st)
    torch.cuda.synchronize()
    (_, ws0, *a), (_, ws1, *b) = run
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    one = [torch.empty_like(t) for t in a]
    moe.moe_linear_backward(cfg, dy, x, w, None, *one, ws0)
    assert all(torch.equal(p, q) for p, q in zip(a, one))
    assert moe.moe_dense_get_device_status(ws0) == 0 and moe.moe_dense_get_device_status(ws1) == 0


def test_one_workspace_for_several_sizes(gpu_lib):
    """A workspace of the largest size serves smaller calls between its own:
    the counters are back at zero after each."""
    moe, g = gpu_lib, gen_of(14)
    sizes = [(5000, 72, 136), (300, 2040, 72), (2100, 264, 328), (1, 264, 136)]
    cfgs = [moe.dense_config(*s) for s in sizes]
    ws = moe._new_ws(max(moe.moe_linear_backward_workspace_size(c) for c in cfgs), "cuda")
    want = {}
    for rep in range(2):
        for (T, K, N), cfg in zip(sizes, cfgs):
            gg = gen_of(T)
            x, w, dy = rnd(gg, T, K), rnd(gg, N, K, scale=0.1), rnd(gg, T, N)
            out = [torch.empty_like(x), torch.empty((N, K), device="cuda"), torch.empty(N, device="cuda")]
            moe.moe_linear_backward(cfg, dy, x, w, None, *out, ws)
            if rep == 0:
                own = [torch.empty_like(t) for t in out]
                moe.moe_linear_backward(cfg, dy, x, w, None, *own, moe.linear_backward_workspace(cfg))
                want[T] = own
            assert all(torch.equal(a, b) for a, b in zip(out, want[T])), (rep, T)
    assert (ws[:moe.DENSE_WS_HEADER] == 0).all()


def test_one_workspace_for_the_block(gpu_lib):
    """The norm's backward pass leaves the header of a workspace that the dense
    calls use too, whose forward here splits its tiles (counters)."""
    moe, g = gpu_lib, gen_of(16)
    T, K, N = 1500, 2880, 3304
    x, w = rnd(g, T, K), rnd(g, N, K, scale=K ** -0.5)
    cfg, ncfg = moe.dense_config(T, K, N), moe.norm_config(T, K)
    ws = moe._new_ws(max(moe.moe_linear_workspace_size(cfg), moe.moe_norm_workspace_size(ncfg)), "cuda")
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    moe.norm(x, mean_out=mean, rstd_out=rstd)
    want = moe.linear(x, w)
    for _ in range(2):
        dx, dw, db = torch.empty_like(x), torch.empty(K, device="cuda"), torch.empty(K, device="cuda")
        moe.moe_norm_backward(ncfg, x, x, None, mean, rstd, None, dx, dw, db, ws)
        assert (ws[:moe.DENSE_WS_HEADER] == 0).all()
        assert torch.equal(moe.linear(x, w, ws=ws), want)
    assert moe.moe_dense_get_device_status(ws) == 0


def test_offsets_past_32_bits(gpu_lib):
    """Tensors of more than 2^31 elements: the last rows are as right as the first."""
    moe, g = gpu_lib, gen_of(15)
    T, H = 140000, 16384
    x = torch.zeros((T, H), dtype=BF, device="cuda")
    x[-2:] = rnd(g, 2, H)
    y = moe.norm(x)
    assert torch.equal(y[-2:], moe.norm(x[-2:].clone())) and (y[0] == 0).all()
    del x, y
    T, K, N = 300000, 64, 8192
    x = torch.zeros((T, K), dtype=BF, device="cuda")
    x[-3:] = rnd(g, 3, K)
    w = rnd(g, N, K, scale=K ** -0.5)
    y = moe.linear(x, w, act="relu")
    ref = (x[-3:].double() @ w.double().t()).clamp(min=0)
    within(y[-3:], ref, U8 * ref.abs() + 1e-4, "last rows")
    assert (y[0] == 0).all() and (y[T // 2] == 0).all()


# ---------------------------------------------------- a block, and the layer
def block64(x, nw, nb, wg, wu, wd, kind, act):
    n, _, _, _ = norm64(x, nw, nb, kind, 1e-5)
    return x + (act64(act, n @ wg.t())[0] * (n @ wu.t())) @ wd.t()


@pytest.mark.parametrize("kind,act", [("rms", "silu"), ("layer", "gelu_tanh")])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_ffn_block(gpu_lib, T, kind, act):
    """norm -> gated -> linear with the residual, and all of its gradients,
    against float64 autograd of the formula; the bf16 tensors between the
    steps make this the layer's 2e-2 bar, normwise per tensor.  The gradient of
    one scalar is also compared with a central difference."""
    moe, g = gpu_lib, gen_of(T)
    H, I = 264, 520
    x, dy = rnd(g, T, H), rnd(g, T, H)
    nw = rnd(g, H, scale=0.1, dtype=F32, shift=1.0)
    nb = rnd(g, H, scale=0.1, dtype=F32) if kind == "layer" else None
    wg, wu, wd = rnd(g, I, H, scale=H ** -0.5), rnd(g, I, H, scale=H ** -0.5), rnd(g, H, I, scale=I ** -0.5)
    y, kept = moe.ffn_block(x, nw, wg, wu, wd, nb, kind, act=act, keep=True)
    assert torch.equal(y, moe.ffn_block(x, nw, wg, wu, wd, nb, kind, act=act))
    grads = moe.ffn_block_backward(dy, kept)
    leaf = [None if t is None else t.double().requires_grad_() for t in (x, nw, nb, wg, wu, wd)]
    ref = block64(*leaf, kind, act)
    ref.backward(dy.double())

    def close(got, want, what):
        err = (got.double() - want).abs().max() / want.abs().max()
        assert err <= 2e-2, (what, float(err))

    close(y, ref.detach(), "y")
    names = ("dx", "d_norm_w", "d_norm_b", "d_w_gate", "d_w_up", "d_w_down")
    for name, t in zip(names, leaf):
        if t is None:
            assert grads[name] is None
        else:
            close(grads[name], t.grad, name)
    # the directional derivative along a random direction of every leaf
    dirs = [None if t is None else torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64) * 0.1
            for t in leaf]
    vals = []
    with torch.no_grad():
        for h in (1e-4, -1e-4):
            p = [None if t is None else t + h * v for t, v in zip(leaf, dirs)]
            vals.append((block64(*p, kind, act) * dy.double()).sum())
    diff = (vals[0] - vals[1]) / 2e-4
    dot = sum((grads[n].double() * v).sum() for n, v in zip(names, dirs) if v is not None)
    size = sum((grads[n].double() * v).square().sum() for n, v in zip(names, dirs) if v is not None).sqrt()
    assert abs(diff - dot) <= 2e-2 * size, (float(diff), float(dot), float(size))


def test_forward_behind_its_norm(gpu_lib):
    """forward(norm_kind=...) is the routed layer on the normed rows."""
    moe, g = gpu_lib, gen_of(9)
    T, H, I, E, k = 70, 256, 128, 8, 2
    x, rw = rnd(g, T, H, scale=3.0), rnd(g, E, H, scale=H ** -0.5)
    wg, wu, wd = rnd(g, E, I, H, scale=H ** -0.5), rnd(g, E, I, H, scale=H ** -0.5), rnd(g, E, H, I, scale=I ** -0.5)
    nw = rnd(g, H, scale=0.1, dtype=F32, shift=1.0)
    y = moe.forward(x, rw, wg, wu, wd, k, norm_w=nw, norm_kind="rms")
    n = moe.norm(x, nw, kind="rms")
    assert torch.equal(y, moe.forward(n, rw, wg, wu, wd, k))
