"""Measured cases of the block operators around the routed FFN layer.

Three operators, each forward and backward: the norm in front of an FFN
(``norm``), the gate/up projections with their activation and product
(``gated``) and the matrix product with bias, activation and residual
(``linear``).  ``run`` computes a case either in its plain form (elementary
torch operations in 32 bits, rounded once at the end) or, with ``own`` set,
through the package's entry points.

Layouts: x [T, K], weights [N, K] (nn.Linear), biases and norm weights
float32, activations and weights bfloat16 unless a case says ``f32``.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
ACTS = ("none", "silu", "gelu", "gelu_tanh", "relu")
_DT = {BF16: torch.bfloat16, F32: torch.float32}
_ES = {BF16: 2, F32: 4}
_MAX_FLOPS = 8.0 * 4096 * 4096 * 14336  # the largest listed case
_MAX_NORM = 16384 * 7168


def _norm(name, d, T, H, kind="layer", dtype=BF16, dy=BF16, bias=True, res=False, stats=False):
    return {"name": name, "op": "norm", "dir": d, "T": T, "H": H, "kind": kind, "dtype": dtype, "dy": dy,
            "bias": bias, "res": res, "stats": stats, "eps": 1e-5}


def _dense(name, op, d, T, K, N, act, bias=False, res=False, save=False, grad=BF16):
    return {"name": name, "op": op, "dir": d, "T": T, "K": K, "N": N, "act": act, "bias": bias, "res": res,
            "save": save, "grad": grad}


def listed():
    return [
        # the pre-norm of one generated token per sequence, eight sequences (gpt-oss-20b width): latency
        _norm("norm_fwd_decode", "fwd", 8, 2880, kind="rms", bias=False),
        # the pre-norm of a training batch of the 32768-token layer, statistics kept for the backward pass
        _norm("norm_fwd_batch", "fwd", 32768, 2048, stats=True),
        # its backward pass on the widest layer: the upstream gradient is the routed layer's float32 dx,
        # and the residual stream's own gradient is added
        _norm("norm_bwd_batch", "bwd", 16384, 7168, kind="rms", dy=F32, bias=False, res=True),
        # a float32 layer's backward pass, an odd batch
        _norm("norm_bwd_f32", "bwd", 513, 4096, dtype=F32, dy=F32),
        # down projection of one generated token, the residual stream added (Mixtral-8x7B sizes)
        _dense("linear_fwd_decode", "linear", "fwd", 1, 14336, 4096, "none", res=True),
        # a biased, activated projection of a ragged serving batch
        _dense("linear_fwd_ragged", "linear", "fwd", 333, 2880, 2880, "gelu", bias=True, save=True),
        # down projection of a training batch with the residual
        _dense("linear_fwd_batch", "linear", "fwd", 8192, 2048, 7168, "none", res=True),
        # backward pass of a biased, activated projection
        _dense("linear_bwd_batch", "linear", "bwd", 8191, 2880, 2880, "gelu_tanh", bias=True),
        # gate/up of eight generated tokens (Mixtral-8x7B sizes): the weights' stream
        _dense("gated_fwd_decode", "gated", "fwd", 8, 4096, 14336, "silu"),
        # gate/up of a training batch, the two projections kept for the backward pass
        _dense("gated_fwd_batch", "gated", "fwd", 4096, 4096, 14336, "silu", save=True),
        # backward pass of a small odd batch on small experts (Qwen3-30B-A3B sizes)
        _dense("gated_bwd_small", "gated", "bwd", 65, 2048, 768, "silu"),
        # backward pass of a training batch: the largest case
        _dense("gated_bwd_batch", "gated", "bwd", 4096, 4096, 14336, "silu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "linear", "linear", "gated", "gated"))
    d = rng.choice(("fwd", "bwd"))
    while True:
        T = _log(rng, 1, 32768)
        if op == "norm":
            H = 8 * _log(rng, 8, 1024)
            dtype = rng.choice((BF16, BF16, F32))
            c = _norm("", d, T, H, kind=rng.choice(("layer", "rms")), dtype=dtype,
                      dy=F32 if dtype == F32 else rng.choice((BF16, F32)), bias=rng.random() < 0.5,
                      res=d == "bwd" and rng.random() < 0.5, stats=rng.random() < 0.5)
            if T * H > _MAX_NORM:
                continue
        else:
            K, N = 8 * _log(rng, 8, 2048), 8 * _log(rng, 8, 2048)
            act = rng.choice(ACTS if op == "linear" else ACTS[1:])
            c = _dense("", op, d, T, K, N, act, bias=rng.random() < 0.5,
                       res=op == "linear" and d == "fwd" and rng.random() < 0.5,
                       save=d == "fwd" and rng.random() < 0.5,
                       # float32 weight gradients where dz is dy itself (nothing is rounded before the product)
                       grad=F32 if op == "linear" and act == "none" and rng.random() < 0.5 else BF16)
            if work(c)["flops"] > _MAX_FLOPS:
                continue
        del c["name"]
        return c


def work(case):
    T = case["T"]
    if case["op"] == "norm":
        n, e, H = T * case["H"], _ES[case["dtype"]], case["H"]
        vec = 4 * H * (1 + case["bias"])
        if case["dir"] == "fwd":
            stat = 4 * T * (1 + (case["kind"] == "layer")) if case["stats"] else 0
            return {"bytes": 2 * n * e + vec + stat, "flops": 8 * n}
        by = n * (_ES[case["dy"]] + 2 * e + (e if case["res"] else 0))
        stat = 4 * T * (1 + (case["kind"] == "layer"))
        return {"bytes": by + 4 * H + vec + stat, "flops": 14 * n}
    K, N = case["K"], case["N"]
    p = 2 if case["op"] == "gated" else 1
    if case["dir"] == "fwd":
        by = 2 * (T * K + p * N * K + T * N)
        by += 4 * p * N if case["bias"] else 0
        by += 2 * T * N if case["res"] else 0
        by += 2 * p * T * N if case["save"] else 0
        return {"bytes": by, "flops": 2 * p * T * K * N}
    by = 2 * (T * N + T * K + p * N * K + T * K) + p * N * K * _ES[case["grad"]]
    by += 2 * p * T * N if p == 2 or case["act"] != "none" else 0
    by += 4 * p * N if case["bias"] else 0
    return {"bytes": by, "flops": 4 * p * T * K * N}


# ------------------------------------------------------------------ inputs
def _inputs(case, seed):
    """The case's tensors, from the seed alone: activations and gradients of
    unit size, weights of 1/sqrt(fan-in), norm weights around one."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape, scale=1.0, dtype=BF16, shift=0.0):
        t = torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)
        return t.mul_(scale).add_(shift).to(_DT[dtype])

    T = case["T"]
    s = {}
    if case["op"] == "norm":
        H, dt = case["H"], case["dtype"]
        s["x"] = rnd(T, H, scale=1.5, dtype=dt, shift=0.2)
        s["w"] = rnd(H, scale=0.1, dtype=F32, shift=1.0)
        s["b"] = rnd(H, scale=0.1, dtype=F32) if case["bias"] else None
        if case["dir"] == "bwd":
            s["dy"] = rnd(T, H, dtype=case["dy"])
            s["res"] = rnd(T, H, dtype=dt) if case["res"] else None
            x = s["x"].double()
            mu = x.mean(1) if case["kind"] == "layer" else torch.zeros_like(x[:, 0])
            s["mean"] = mu.float() if case["kind"] == "layer" else None
            s["rstd"] = ((x - mu[:, None]).square().mean(1) + case["eps"]).rsqrt().float()
        return s
    K, N = case["K"], case["N"]
    names = ("w",) if case["op"] == "linear" else ("w_gate", "w_up")
    s["x"] = rnd(T, K)
    for n in names:
        s[n] = rnd(N, K, scale=K ** -0.5)
        s[n.replace("w", "b", 1)] = rnd(N, scale=0.1, dtype=F32) if case["bias"] else None
    if case["dir"] == "fwd":
        s["res"] = rnd(T, N) if case["res"] else None
    else:
        s["dy"] = rnd(T, N)
        # the projections as the forward pass keeps them
        for n, z in zip(names, ("z",) if case["op"] == "linear" else ("g", "u")):
            b = s[n.replace("w", "b", 1)]
            v = (s["x"] @ s[n].t()).float()
            s[z] = (v if b is None else v + b).to(torch.bfloat16)
        if case["op"] == "linear" and case["act"] == "none":
            s["z"] = None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if not own:
        return s
    import sparse_mixture_experts_19_b200 as moe

    dev = "cuda"
    T = case["T"]
    if case["op"] == "norm":
        H, dt = case["H"], _DT[case["dtype"]]
        s["cfg"] = cfg = moe.norm_config(T, H, kind=case["kind"], eps=case["eps"], dtype=case["dtype"],
                                         dy_dtype=case["dy"])
        layer = case["kind"] == "layer"
        if case["dir"] == "fwd":
            s["y"] = torch.empty(T, H, dtype=dt, device=dev)
            s["mean"] = torch.empty(T, device=dev) if case["stats"] and layer else None
            s["rstd"] = torch.empty(T, device=dev) if case["stats"] else None
        else:
            s["dx"] = torch.empty(T, H, dtype=dt, device=dev)
            s["dw"] = torch.empty(H, device=dev)
            s["db"] = torch.empty(H, device=dev) if case["bias"] else None
            s["ws"] = moe.norm_workspace(cfg)
        return s
    K, N = case["K"], case["N"]
    s["cfg"] = cfg = moe.dense_config(T, K, N, act=case["act"], grad_dtype=case["grad"])
    gated = case["op"] == "gated"

    def buf(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device=dev)

    if case["dir"] == "fwd":
        s["ws"] = moe.gated_workspace(cfg) if gated else moe.linear_workspace(cfg)
        s["y"] = buf(T, N)
        for z in ("g", "u") if gated else ("z",):
            s[z] = buf(T, N) if case["save"] else None
    else:
        s["ws"] = moe.gated_backward_workspace(cfg) if gated else moe.linear_backward_workspace(cfg)
        s["dx"] = buf(T, K)
        for n in ("_gate", "_up") if gated else ("",):
            s["dw" + n] = buf(N, K, dtype=_DT[case["grad"]])
            s["db" + n] = buf(N, dtype=torch.float32) if case["bias"] else None
    return s


# ------------------------------------------------------------------ passes
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _outs(*ts):
    return [t for t in ts if t is not None]


def _run_own(s):
    import sparse_mixture_experts_19_b200 as moe

    c, cfg = s["case"], s["cfg"]
    if c["op"] == "norm":
        if c["dir"] == "fwd":
            moe.moe_norm_forward(cfg, s["x"], s["w"], s["b"], s["y"], s["mean"], s["rstd"])
            return _outs(s["y"], s["mean"], s["rstd"])
        moe.moe_norm_backward(cfg, s["dy"], s["x"], s["w"], s["mean"], s["rstd"], s["res"], s["dx"], s["dw"],
                              s["db"], s["ws"])
        return _outs(s["dx"], s["dw"], s["db"])
    if c["op"] == "linear":
        if c["dir"] == "fwd":
            moe.moe_linear_forward(cfg, s["x"], s["w"], s["b"], s["res"], s["y"], s["z"], s["ws"])
            return _outs(s["y"], s["z"])
        moe.moe_linear_backward(cfg, s["dy"], s["x"], s["w"], s["z"], s["dx"], s["dw"], s["db"], s["ws"])
        return _outs(s["dx"], s["dw"], s["db"])
    if c["dir"] == "fwd":
        moe.moe_gated_forward(cfg, s["x"], s["w_gate"], s["w_up"], s["b_gate"], s["b_up"], s["y"], s["g"], s["u"],
                              s["ws"])
        return _outs(s["y"], s["g"], s["u"])
    moe.moe_gated_backward(cfg, s["dy"], s["x"], s["w_gate"], s["w_up"], s["g"], s["u"], s["dx"], s["dw_gate"],
                           s["dw_up"], s["db_gate"], s["db_up"], s["ws"])
    return _outs(s["dx"], s["dw_gate"], s["dw_up"], s["db_gate"], s["db_up"])


def _act(a, z):
    """(act(z), act'(z)) elementwise, in z's type."""
    if a == "none":
        return z, torch.ones_like(z)
    if a == "relu":
        return z.clamp(min=0), (z > 0).to(z.dtype)
    if a == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return z * sg, sg * (1 + z * (1 - sg))
    if a == "gelu":
        cdf = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)


def _run_plain(s):
    c = s["case"]
    f = torch.Tensor.float
    x = f(s["x"])
    bf = torch.bfloat16
    if c["op"] == "norm":
        layer, dt = c["kind"] == "layer", _DT[c["dtype"]]
        if c["dir"] == "fwd":
            mu = x.mean(1, keepdim=True) if layer else None
            xc = x - mu if layer else x
            r = (xc.square().mean(1, keepdim=True) + c["eps"]).rsqrt()
            y = xc * r * s["w"]
            y = y if s["b"] is None else y + s["b"]
            return _outs(y.to(dt), mu[:, 0] if layer and c["stats"] else None, r[:, 0] if c["stats"] else None)
        dy, r = f(s["dy"]), s["rstd"][:, None]
        xh = (x - s["mean"][:, None] if layer else x) * r
        a = dy * s["w"]
        dx = a - xh * (a * xh).mean(1, keepdim=True)
        dx = r * (dx - a.mean(1, keepdim=True) if layer else dx)
        dx = dx if s["res"] is None else dx + f(s["res"])
        return _outs(dx.to(dt), (dy * xh).sum(0), dy.sum(0) if c["bias"] else None)

    def proj(w, b):
        z = x @ f(w).t()
        return z if b is None else z + b

    gd = _DT[c["grad"]]
    if c["op"] == "linear":
        if c["dir"] == "fwd":
            z = proj(s["w"], s["b"])
            y = _act(c["act"], z)[0]
            y = y if s["res"] is None else y + f(s["res"])
            return _outs(y.to(bf), z.to(bf) if c["save"] else None)
        dz = f(s["dy"])
        dz = dz if s["z"] is None else dz * _act(c["act"], f(s["z"]))[1]
        return _outs((dz @ f(s["w"])).to(bf), (dz.t() @ x).to(gd), dz.sum(0) if c["bias"] else None)
    if c["dir"] == "fwd":
        g, u = proj(s["w_gate"], s["b_gate"]), proj(s["w_up"], s["b_up"])
        keep = c["save"]
        return _outs((_act(c["act"], g)[0] * u).to(bf), g.to(bf) if keep else None, u.to(bf) if keep else None)
    dh = f(s["dy"])
    a, da = _act(c["act"], f(s["g"]))
    dg, du = dh * f(s["u"]) * da, dh * a
    dx = dg @ f(s["w_gate"]) + du @ f(s["w_up"])
    return _outs(dx.to(bf), (dg.t() @ x).to(gd), (du.t() @ x).to(gd), dg.sum(0) if c["bias"] else None,
                 du.sum(0) if c["bias"] else None)


# ------------------------------------------------------------------- exact
def _phi(a, z):
    """The activation's value and slope from its definition, float64."""
    if a == "none":
        return z, torch.full_like(z, 1.0)
    if a == "relu":
        return torch.where(z > 0, z, 0.0), torch.where(z > 0, 1.0, 0.0).to(z)
    if a == "silu":
        p = torch.sigmoid(z)
        return p * z, p + z * p * torch.sigmoid(-z)
    if a == "gelu":
        p = torch.special.ndtr(z)
        return p * z, p + z * (z.square() / -2).exp() / (2 * math.pi) ** 0.5
    # gelu_tanh: z * sigmoid(2 q), q = sqrt(2 / pi) (z + 0.044715 z^3)
    q2 = (8 / math.pi) ** 0.5 * (z + 0.044715 * z.pow(3))
    p = torch.sigmoid(q2)
    return z * p, p + z * p * torch.sigmoid(-q2) * (8 / math.pi) ** 0.5 * (1 + 0.134145 * z.square())


def exact(case, seed):
    s = {k: v.double() if torch.is_tensor(v) else v for k, v in _inputs(case, seed).items()}
    fwd = case["dir"] == "fwd"
    if case["op"] == "norm":
        x, layer = s["x"], case["kind"] == "layer"
        if fwd:
            var, mu = torch.var_mean(x, dim=1, correction=0)
            ms = var if layer else torch.einsum("th,th->t", x, x) / x.shape[1]
            mu = mu if layer else torch.zeros_like(mu)
            sd = torch.sqrt(ms + case["eps"])
            y = (x - mu.unsqueeze(1)) / sd.unsqueeze(1) * s["w"]
            if case["bias"]:
                y += s["b"]
            out = [y]
            if case["stats"]:
                out += [mu, 1 / sd] if layer else [1 / sd]
            return out
        xh = torch.einsum("th,t->th", x - s["mean"].unsqueeze(1) if layer else x, s["rstd"])
        a = s["dy"] * s["w"]
        c2 = torch.einsum("th,th->t", a, xh) / x.shape[1]
        g = a - torch.einsum("t,th->th", c2, xh)
        if layer:
            g -= a.mean(dim=1, keepdim=True)
        g = torch.einsum("th,t->th", g, s["rstd"])
        if case["res"]:
            g += s["res"]
        out = [g, torch.einsum("th,th->h", s["dy"], xh)]
        return out + [s["dy"].sum(dim=0)] if case["bias"] else out

    def project(w, b):
        z = torch.einsum("tk,nk->tn", s["x"], s[w])
        return z + s[b] if case["bias"] else z

    if case["op"] == "linear":
        if fwd:
            z = project("w", "b")
            y = _phi(case["act"], z)[0]
            y = y + s["res"] if case["res"] else y
            return [y, z] if case["save"] else [y]
        dz = s["dy"] if s["z"] is None else s["dy"] * _phi(case["act"], s["z"])[1]
        out = [torch.einsum("tn,nk->tk", dz, s["w"]), torch.einsum("tn,tk->nk", dz, s["x"])]
        return out + [dz.sum(dim=0)] if case["bias"] else out
    if fwd:
        g, u = project("w_gate", "b_gate"), project("w_up", "b_up")
        h = _phi(case["act"], g)[0] * u
        return [h, g, u] if case["save"] else [h]
    a, slope = _phi(case["act"], s["g"])
    du = s["dy"] * a
    dg = s["dy"] * slope * s["u"]
    out = [torch.einsum("tn,nk->tk", dg, s["w_gate"]) + torch.einsum("tn,nk->tk", du, s["w_up"]),
           torch.einsum("tn,tk->nk", dg, s["x"]), torch.einsum("tn,tk->nk", du, s["x"])]
    return out + [dg.sum(dim=0), du.sum(dim=0)] if case["bias"] else out
