// C ABI of the operators around the routed layer (norm, linear, gated):
// argument checks, workspace carving and launch sequencing.  Like moe_abi.cu:
// nothing here allocates device memory or synchronises, except
// moe_dense_get_device_status (documented to wait).
#include <math.h>

#include <algorithm>
#include <initializer_list>

#include "abi_util.cuh"
#include "dense.cuh"

namespace moe {
namespace {

moe_status_t check_norm(const moe_norm_config_t* c) {
    if (!c) return fail(MOE_ERR_INVALID_ARG, "cfg is NULL");
    if (c->T < 0) return fail(MOE_ERR_INVALID_ARG, "T = %d < 0", c->T);
    if (c->H < 8 || c->H % 8) return fail(MOE_ERR_INVALID_ARG, "H = %d must be a positive multiple of 8", c->H);
    if (c->kind != MOE_NORM_LAYER && c->kind != MOE_NORM_RMS)
        return fail(MOE_ERR_INVALID_ARG, "kind = %d unknown", c->kind);
    if (!isfinite(c->eps) || c->eps < 0.f) return fail(MOE_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (c->dtype != MOE_F32 && c->dtype != MOE_BF16) return fail(MOE_ERR_INVALID_ARG, "dtype = %d unknown", c->dtype);
    if (c->dy_dtype != MOE_F32 && c->dy_dtype != MOE_BF16)
        return fail(MOE_ERR_INVALID_ARG, "dy_dtype = %d unknown", c->dy_dtype);
    if (c->dtype == MOE_F32 && c->dy_dtype != MOE_F32)
        return fail(MOE_ERR_UNSUPPORTED, "float32 rows take a float32 dy");
    if (c->H > kMaxNormWidth) return fail(MOE_ERR_UNSUPPORTED, "H = %d above %d", c->H, kMaxNormWidth);
    return MOE_OK;
}

size_t norm_ws_bytes(const moe_norm_config_t* c) {
    return MOE_DENSE_WS_HEADER + align_up(sizeof(float) * 2 * c->H * (c->T > 0 ? norm_bwd_blocks(c->T) : 1));
}

moe_status_t check_dense(const moe_dense_config_t* c) {
    if (!c) return fail(MOE_ERR_INVALID_ARG, "cfg is NULL");
    if (c->T < 0) return fail(MOE_ERR_INVALID_ARG, "T = %d < 0", c->T);
    if (c->K < 8 || c->K % 8) return fail(MOE_ERR_INVALID_ARG, "K = %d must be a positive multiple of 8", c->K);
    if (c->N < 8 || c->N % 8) return fail(MOE_ERR_INVALID_ARG, "N = %d must be a positive multiple of 8", c->N);
    if (c->act < MOE_ACT_NONE || c->act > MOE_ACT_RELU) return fail(MOE_ERR_INVALID_ARG, "act = %d unknown", c->act);
    if (c->dtype != MOE_F32 && c->dtype != MOE_BF16) return fail(MOE_ERR_INVALID_ARG, "dtype = %d unknown", c->dtype);
    if (c->grad_dtype != MOE_F32 && c->grad_dtype != MOE_BF16)
        return fail(MOE_ERR_INVALID_ARG, "grad_dtype = %d unknown", c->grad_dtype);
    if (c->dtype != MOE_BF16) return fail(MOE_ERR_UNSUPPORTED, "the dense products take bf16 tensors");
    return MOE_OK;
}

// Pieces of a dense workspace.
struct DensePlan {
    // flags and counters first: the header that moe_dense_get_device_status clears
    DenseWs ws;   // the forward product, or the input gradient
    DenseWs wws;  // the weight gradient (no counters: a second kernel adds its splits)
    bf16* dz0;   // [T, N], unless the linear layer has no activation
    bf16* dz1;   // gated
    float* sums; // partial bias gradients
    size_t bytes;
};

void make_dense_plan(const moe_dense_config_t* c, bool gated, bool backward, void* ws, DensePlan* p) {
    size_t off = 0;
    char* base = (char*)ws;
    auto take = [&](size_t bytes) -> void* {
        void* r = base ? base + off : nullptr;
        off += align_up(bytes);
        return r;
    };
    *p = DensePlan{};
    p->ws.flags = (int32_t*)take(64);
    p->ws.counters = (uint32_t*)take(kDenseCounterBytes);
    if (base) p->ws.gate = p->ws.counters + kDenseGateOffset / sizeof(uint32_t);
    p->wws.flags = p->ws.flags;
    p->wws.gate = p->ws.gate;
    const int two = gated ? 2 : 1;
    if (backward && c->T > 0) {
        const size_t tn = (size_t)c->T * c->N;
        if (gated || c->act != MOE_ACT_NONE) p->dz0 = (bf16*)take(tn * 2);
        if (gated) p->dz1 = (bf16*)take(tn * 2);
        p->sums = (float*)take(sizeof(float) * two * c->N * dense_dz_row_blocks(c->T, c->N, gated));
        p->ws.part = (float*)take(sizeof(float) * dense_dgrad_part_floats(c->T, c->K, c->N, two));
        p->wws.part = (float*)take(sizeof(float) * dense_wgrad_part_floats(c->T, c->K, c->N, two));
    } else if (c->T > 0) {
        p->ws.part = (float*)take(sizeof(float) * dense_fwd_part_floats(c->T, c->K, c->N, gated));
    }
    p->bytes = off;
}

moe_status_t dense_plan_for(const moe_dense_config_t* c, bool gated, bool backward, void* ws, size_t ws_bytes,
                            DensePlan* p) {
    moe_status_t s = check_dense(c);
    if (s != MOE_OK) return s;
    make_dense_plan(c, gated, backward, ws, p);
    if (!ws) return fail(MOE_ERR_WORKSPACE, "workspace is NULL");
    if ((uintptr_t)ws % kWsAlign) return fail(MOE_ERR_WORKSPACE, "workspace not %d-byte aligned", kWsAlign);
    if (ws_bytes < p->bytes)
        return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, p->bytes);
    return MOE_OK;
}

size_t dense_ws_size(const moe_dense_config_t* c, bool gated, bool backward) {
    if (check_dense(c) != MOE_OK) return 0;
    DensePlan p;
    make_dense_plan(c, gated, backward, nullptr, &p);
    return p.bytes;
}

size_t grad_bytes(const moe_dense_config_t* c) {
    return (size_t)c->N * c->K * (c->grad_dtype == MOE_F32 ? 4 : 2);
}

// A tensor of a call: n bytes at p (null: not given).  in_place: an input that
// the first output may replace.
struct Span {
    const char* name;
    const void* p;
    size_t n;
    bool in_place = false;
    bool meets(const Span& o) const {
        const uintptr_t a = (uintptr_t)p, b = (uintptr_t)o.p;
        return p && o.p && n && o.n && a < b + o.n && b < a + n;
    }
};

moe_status_t shared(const Span& a, const Span& b) {
    return a.p == b.p ? fail(MOE_ERR_INVALID_ARG, "%s and %s are the same tensor", a.name, b.name)
                      : fail(MOE_ERR_INVALID_ARG, "%s overlaps %s", a.name, b.name);
}

// Refuses an output that shares bytes with another tensor of the call, and a
// workspace that shares bytes with any.
moe_status_t check_apart(std::initializer_list<Span> out, std::initializer_list<Span> in, const Span& ws = {}) {
    for (const Span* o = out.begin(); o != out.end(); ++o) {
        for (const Span& i : in)
            if (o->meets(i) && !(i.in_place && o == out.begin() && o->p == i.p && o->n == i.n)) return shared(*o, i);
        for (const Span* q = o + 1; q != out.end(); ++q)
            if (o->meets(*q)) return shared(*q, *o);
    }
    for (auto list : {out, in})
        for (const Span& t : list)
            if (t.meets(ws)) return shared(t, ws);
    return MOE_OK;
}

size_t f32s(int64_t n) { return (size_t)n * sizeof(float); }

// Bytes of a dense call's tensors: bf16 [T, K], [T, N], [N, K]; float32 [N]; a
// weight gradient.
struct DenseBytes {
    size_t tk, tn, nk, n, dw;
    explicit DenseBytes(const moe_dense_config_t* c)
        : tk((size_t)c->T * c->K * 2),
          tn((size_t)c->T * c->N * 2),
          nk((size_t)c->N * c->K * 2),
          n(f32s(c->N)),
          dw(grad_bytes(c)) {}
};

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_norm_workspace_size(const moe_norm_config_t* cfg) {
    return check_norm(cfg) == MOE_OK ? norm_ws_bytes(cfg) : 0;
}

moe_status_t moe_norm_forward(const moe_norm_config_t* cfg, const void* x, const float* weight, const float* bias,
                              void* y, float* mean_out, float* rstd_out, moe_stream_t stream) {
    moe_status_t s = check_norm(cfg);
    if (s != MOE_OK) return s;
    OPTIONAL_PTR(weight);
    OPTIONAL_PTR(bias);
    OPTIONAL_PTR(mean_out);
    OPTIONAL_PTR(rstd_out);
    const size_t es = cfg->dtype == MOE_F32 ? 4 : 2, rows = (size_t)cfg->T * cfg->H * es;
    s = check_apart({{"y", y, rows}, {"mean_out", mean_out, f32s(cfg->T)}, {"rstd_out", rstd_out, f32s(cfg->T)}},
                    {{"x", x, rows, true}, {"weight", weight, f32s(cfg->H)}, {"bias", bias, f32s(cfg->H)}});
    if (s != MOE_OK) return s;
    if (cfg->T == 0) return MOE_OK;
    REQUIRE_PTR(x);
    REQUIRE_PTR(y);
    NormArgs a{};
    a.T = cfg->T;
    a.H = cfg->H;
    a.layer = cfg->kind == MOE_NORM_LAYER;
    a.eps = cfg->eps;
    a.x = x;
    a.w = weight;
    a.b = bias;
    a.y = y;
    a.mean_out = mean_out;
    a.rstd_out = rstd_out;
    CUDA_TRY(launch_norm_fwd(a, cfg->dtype == MOE_F32, (cudaStream_t)stream), "norm_fwd");
    return MOE_OK;
}

moe_status_t moe_norm_backward(const moe_norm_config_t* cfg, const void* dy, const void* x, const float* weight,
                               const float* mean, const float* rstd, const void* d_residual, void* dx,
                               float* d_weight, float* d_bias, void* ws, size_t ws_bytes, moe_stream_t stream) {
    moe_status_t s = check_norm(cfg);
    if (s != MOE_OK) return s;
    if (!ws) return fail(MOE_ERR_WORKSPACE, "workspace is NULL");
    if ((uintptr_t)ws % kWsAlign) return fail(MOE_ERR_WORKSPACE, "workspace not %d-byte aligned", kWsAlign);
    if (ws_bytes < norm_ws_bytes(cfg))
        return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, norm_ws_bytes(cfg));
    OPTIONAL_PTR(weight);
    OPTIONAL_PTR(d_residual);
    OPTIONAL_PTR(d_weight);
    OPTIONAL_PTR(d_bias);
    const size_t n = (size_t)cfg->T * cfg->H, rows = n * (cfg->dtype == MOE_F32 ? 4 : 2);
    s = check_apart({{"dx", dx, rows}, {"d_weight", d_weight, f32s(cfg->H)}, {"d_bias", d_bias, f32s(cfg->H)}},
                    {{"dy", dy, n * (cfg->dy_dtype == MOE_F32 ? 4 : 2), true},
                     {"x", x, rows, true},
                     {"d_residual", d_residual, rows, true},
                     {"weight", weight, f32s(cfg->H)},
                     {"mean", mean, f32s(cfg->T)},
                     {"rstd", rstd, f32s(cfg->T)}},
                    {"ws", ws, norm_ws_bytes(cfg)});
    if (s != MOE_OK) return s;
    cudaStream_t st = (cudaStream_t)stream;
    if (cfg->T == 0) {
        if (d_weight) CUDA_TRY(cudaMemsetAsync(d_weight, 0, sizeof(float) * cfg->H, st), "memset");
        if (d_bias) CUDA_TRY(cudaMemsetAsync(d_bias, 0, sizeof(float) * cfg->H, st), "memset");
        return MOE_OK;
    }
    REQUIRE_PTR(dy);
    REQUIRE_PTR(x);
    if (cfg->kind == MOE_NORM_LAYER) REQUIRE_PTR(mean);
    REQUIRE_PTR(rstd);
    REQUIRE_PTR(dx);
    NormArgs a{};
    a.T = cfg->T;
    a.H = cfg->H;
    a.layer = cfg->kind == MOE_NORM_LAYER;
    a.x = x;
    a.w = weight;
    a.dy = dy;
    a.mean = mean;
    a.rstd = rstd;
    a.d_res = d_residual;
    a.dx = dx;
    // behind the header of the dense calls, which may share the workspace
    a.part = d_weight || d_bias ? (float*)((char*)ws + MOE_DENSE_WS_HEADER) : nullptr;
    a.dw_out = d_weight;
    a.db_out = d_bias;
    CUDA_TRY(launch_norm_bwd(a, cfg->dtype == MOE_F32, cfg->dy_dtype == MOE_F32, st), "norm_bwd");
    return MOE_OK;
}

size_t moe_linear_workspace_size(const moe_dense_config_t* cfg) { return dense_ws_size(cfg, false, false); }
size_t moe_linear_backward_workspace_size(const moe_dense_config_t* cfg) { return dense_ws_size(cfg, false, true); }
size_t moe_gated_workspace_size(const moe_dense_config_t* cfg) { return dense_ws_size(cfg, true, false); }
size_t moe_gated_backward_workspace_size(const moe_dense_config_t* cfg) { return dense_ws_size(cfg, true, true); }

moe_status_t moe_linear_forward(const moe_dense_config_t* cfg, const void* x, const void* w, const float* bias,
                                const void* residual, void* y, void* z_out, void* ws, size_t ws_bytes,
                                moe_stream_t stream) {
    DensePlan p;
    moe_status_t s = dense_plan_for(cfg, false, false, ws, ws_bytes, &p);
    if (s != MOE_OK) return s;
    if (cfg->T == 0) return MOE_OK;
    REQUIRE_PTR(x);
    REQUIRE_PTR(w);
    OPTIONAL_PTR(bias);
    OPTIONAL_PTR(residual);
    REQUIRE_PTR(y);
    OPTIONAL_PTR(z_out);
    const DenseBytes b(cfg);
    s = check_apart({{"y", y, b.tn}, {"z_out", z_out, b.tn}},
                    {{"x", x, b.tk}, {"w", w, b.nk}, {"bias", bias, b.n}, {"residual", residual, b.tn, true}},
                    {"ws", ws, p.bytes});
    if (s != MOE_OK) return s;
    DenseOut o{};
    o.act = cfg->act;
    o.bias0 = bias;
    o.res = (const bf16*)residual;
    o.y = (bf16*)y;
    o.z0 = (bf16*)z_out;
    CUDA_TRY(launch_dense_fwd(x, w, nullptr, cfg->T, cfg->K, cfg->N, o, p.ws, (cudaStream_t)stream), "linear_fwd");
    return MOE_OK;
}

moe_status_t moe_linear_backward(const moe_dense_config_t* cfg, const void* dy, const void* x, const void* w,
                                 const void* z, void* dx, void* d_w, float* d_bias, void* ws, size_t ws_bytes,
                                 moe_stream_t stream) {
    DensePlan p;
    moe_status_t s = dense_plan_for(cfg, false, true, ws, ws_bytes, &p);
    if (s != MOE_OK) return s;
    OPTIONAL_PTR(dx);
    OPTIONAL_PTR(d_w);
    OPTIONAL_PTR(d_bias);
    const DenseBytes b(cfg);
    s = check_apart({{"dx", dx, b.tk}, {"d_w", d_w, b.dw}, {"d_bias", d_bias, b.n}},
                    {{"dy", dy, b.tn}, {"x", x, b.tk}, {"w", w, b.nk}, {"z", z, b.tn}}, {"ws", ws, p.bytes});
    if (s != MOE_OK) return s;
    cudaStream_t st = (cudaStream_t)stream;
    if (cfg->T == 0) {
        if (d_w) CUDA_TRY(cudaMemsetAsync(d_w, 0, grad_bytes(cfg), st), "memset");
        if (d_bias) CUDA_TRY(cudaMemsetAsync(d_bias, 0, sizeof(float) * cfg->N, st), "memset");
        return MOE_OK;
    }
    const bool act = cfg->act != MOE_ACT_NONE;
    REQUIRE_PTR(dy);
    if (d_w) REQUIRE_PTR(x);
    if (dx) REQUIRE_PTR(w);
    if (act) REQUIRE_PTR(z);
    const bf16* dz = act ? p.dz0 : (const bf16*)dy;
    if (d_bias || (act && (dx || d_w))) {
        DenseDzArgs a{};
        a.T = cfg->T;
        a.N = cfg->N;
        a.dy = (const bf16*)dy;
        a.z = (const bf16*)z;
        a.dz = act ? p.dz0 : nullptr;
        a.part = p.sums;
        CUDA_TRY(launch_dense_dz(a, false, cfg->act, d_bias, nullptr, st), "linear_dz");
    }
    WgradPlan plan{true, false};
    if (dx)
        CUDA_TRY(launch_dense_dgrad(dz, nullptr, w, nullptr, cfg->T, cfg->K, cfg->N, dx, d_w != nullptr, &plan, p.ws,
                                    st),
                 "linear_dgrad");
    if (d_w)
        CUDA_TRY(launch_dense_wgrad(dz, nullptr, x, cfg->T, cfg->K, cfg->N, d_w, nullptr, cfg->grad_dtype == MOE_F32,
                                    plan, p.wws, st),
                 "linear_wgrad");
    return MOE_OK;
}

moe_status_t moe_gated_forward(const moe_dense_config_t* cfg, const void* x, const void* w_gate, const void* w_up,
                               const float* b_gate, const float* b_up, void* h, void* g_out, void* u_out, void* ws,
                               size_t ws_bytes, moe_stream_t stream) {
    DensePlan p;
    moe_status_t s = dense_plan_for(cfg, true, false, ws, ws_bytes, &p);
    if (s != MOE_OK) return s;
    if (cfg->T == 0) return MOE_OK;
    REQUIRE_PTR(x);
    REQUIRE_PTR(w_gate);
    REQUIRE_PTR(w_up);
    OPTIONAL_PTR(b_gate);
    OPTIONAL_PTR(b_up);
    REQUIRE_PTR(h);
    OPTIONAL_PTR(g_out);
    OPTIONAL_PTR(u_out);
    const DenseBytes b(cfg);
    s = check_apart({{"h", h, b.tn}, {"g_out", g_out, b.tn}, {"u_out", u_out, b.tn}},
                    {{"x", x, b.tk}, {"w_gate", w_gate, b.nk}, {"w_up", w_up, b.nk}, {"b_gate", b_gate, b.n},
                     {"b_up", b_up, b.n}},
                    {"ws", ws, p.bytes});
    if (s != MOE_OK) return s;
    DenseOut o{};
    o.act = cfg->act;
    o.bias0 = b_gate;
    o.bias1 = b_up;
    o.y = (bf16*)h;
    o.z0 = (bf16*)g_out;
    o.z1 = (bf16*)u_out;
    CUDA_TRY(launch_dense_fwd(x, w_gate, w_up, cfg->T, cfg->K, cfg->N, o, p.ws, (cudaStream_t)stream), "gated_fwd");
    return MOE_OK;
}

moe_status_t moe_gated_backward(const moe_dense_config_t* cfg, const void* dh, const void* x, const void* w_gate,
                                const void* w_up, const void* g, const void* u, void* dx, void* d_w_gate,
                                void* d_w_up, float* d_b_gate, float* d_b_up, void* ws, size_t ws_bytes,
                                moe_stream_t stream) {
    DensePlan p;
    moe_status_t s = dense_plan_for(cfg, true, true, ws, ws_bytes, &p);
    if (s != MOE_OK) return s;
    OPTIONAL_PTR(dx);
    OPTIONAL_PTR(d_w_gate);
    OPTIONAL_PTR(d_w_up);
    OPTIONAL_PTR(d_b_gate);
    OPTIONAL_PTR(d_b_up);
    if (!d_w_gate != !d_w_up) return fail(MOE_ERR_INVALID_ARG, "d_w_gate and d_w_up go together");
    const DenseBytes b(cfg);
    s = check_apart({{"dx", dx, b.tk}, {"d_w_gate", d_w_gate, b.dw}, {"d_w_up", d_w_up, b.dw}, {"d_b_gate", d_b_gate, b.n},
                     {"d_b_up", d_b_up, b.n}},
                    {{"dh", dh, b.tn}, {"x", x, b.tk}, {"w_gate", w_gate, b.nk}, {"w_up", w_up, b.nk}, {"g", g, b.tn},
                     {"u", u, b.tn}},
                    {"ws", ws, p.bytes});
    if (s != MOE_OK) return s;
    cudaStream_t st = (cudaStream_t)stream;
    if (cfg->T == 0) {
        if (d_w_gate) CUDA_TRY(cudaMemsetAsync(d_w_gate, 0, grad_bytes(cfg), st), "memset");
        if (d_w_up) CUDA_TRY(cudaMemsetAsync(d_w_up, 0, grad_bytes(cfg), st), "memset");
        if (d_b_gate) CUDA_TRY(cudaMemsetAsync(d_b_gate, 0, sizeof(float) * cfg->N, st), "memset");
        if (d_b_up) CUDA_TRY(cudaMemsetAsync(d_b_up, 0, sizeof(float) * cfg->N, st), "memset");
        return MOE_OK;
    }
    REQUIRE_PTR(dh);
    REQUIRE_PTR(g);
    REQUIRE_PTR(u);
    if (d_w_gate) REQUIRE_PTR(x);
    if (dx) {
        REQUIRE_PTR(w_gate);
        REQUIRE_PTR(w_up);
    }
    DenseDzArgs a{};
    a.T = cfg->T;
    a.N = cfg->N;
    a.dy = (const bf16*)dh;
    a.z = (const bf16*)g;
    a.u = (const bf16*)u;
    a.dz = p.dz0;
    a.dz1 = p.dz1;
    a.part = p.sums;
    CUDA_TRY(launch_dense_dz(a, true, cfg->act, d_b_gate, d_b_up, st), "gated_dgu");
    WgradPlan plan{true, false};
    if (dx)
        CUDA_TRY(launch_dense_dgrad(p.dz0, p.dz1, w_gate, w_up, cfg->T, cfg->K, cfg->N, dx, d_w_gate != nullptr,
                                    &plan, p.ws, st),
                 "gated_dgrad");
    if (d_w_gate)
        CUDA_TRY(launch_dense_wgrad(p.dz0, p.dz1, x, cfg->T, cfg->K, cfg->N, d_w_gate, d_w_up,
                                    cfg->grad_dtype == MOE_F32, plan, p.wws, st),
                 "gated_wgrad");
    return MOE_OK;
}

moe_status_t moe_dense_get_device_status(void* ws, size_t ws_bytes, moe_stream_t stream, int32_t* flags_out) {
    if (!ws) return fail(MOE_ERR_WORKSPACE, "workspace is NULL");
    if ((uintptr_t)ws % kWsAlign) return fail(MOE_ERR_WORKSPACE, "workspace not %d-byte aligned", kWsAlign);
    static_assert(MOE_DENSE_WS_HEADER == kWsAlign + kDenseCounterBytes, "workspace header");
    if (ws_bytes < MOE_DENSE_WS_HEADER)
        return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %d", ws_bytes, MOE_DENSE_WS_HEADER);
    const moe_status_t s = read_device_flags((int32_t*)ws, (cudaStream_t)stream, flags_out);
    // a call that gave up may have left its counters counting
    if (s == MOE_ERR_DEVICE_CHECK)
        CUDA_TRY(cudaMemsetAsync((char*)ws + kWsAlign, 0, kDenseCounterBytes, (cudaStream_t)stream), "counters clear");
    return s;
}

}  // extern "C"
