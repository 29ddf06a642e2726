// api_block.cu -- the extern "C" boundary of what stands around the layer: norm,
// 8-bit data and experts, balance loss over sequences (declared in moe.h).
// Arguments are checked before anything is enqueued.
#include <math.h>

#include "internal.h"

namespace moe {

static bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
static bool al32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }
static bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

static moe_status check_scratch(const void* ws, size_t bytes, size_t need)
{
    if (ws == nullptr || bytes < need) return MOE_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)) != 0) return MOE_ERR_ALIGN;
    return MOE_OK;
}

static moe_status check_rows(int64_t T, int64_t D, int32_t dtype)
{
    if (T < 1 || D < 1 || T > (int64_t)INT32_MAX) return MOE_ERR_SHAPE;
    if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_ARG;
    return MOE_OK;
}

// cfg of the 8-bit experts
static moe_status check_mx8_config(const moe_config* cfg)
{
    moe_status st = moe_check_config(cfg);
    if (st != MOE_OK) return st;
    if (cfg->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
    if (cfg->D % 32 != 0 || cfg->F % 32 != 0) return MOE_ERR_ALIGN;
    return MOE_OK;
}

static moe_status check_mx8_weights(const moe_mx8_weights* w)
{
    if (w == nullptr) return MOE_ERR_ARG;
    const void* p[6] = {w->gate, w->gate_scales, w->up, w->up_scales, w->down, w->down_scales};
    for (const void* q : p) {
        if (q == nullptr) return MOE_ERR_ARG;
        if (!al16(q)) return MOE_ERR_ALIGN;
    }
    return MOE_OK;
}

// the status region, the experts' A maps, the parts of a cut down product
static size_t mx8_maps_at() { return align_up(64 * sizeof(int)); }
static size_t mx8_part_at(const moe_config& c) { return mx8_maps_at() + align_up(2 * (size_t)c.E * kTensorMapBytes); }
static size_t mx8_ws_bytes(const moe_config& c)
{
    return mx8_part_at(c) + align_up(mx8_part_bytes(c, max_rows_of(c)));
}

struct FwdMx8Layout {
    WsLayout ws;
    size_t amaps, part, ids, w, counts, kept, offsets, perm, row_of;
    size_t xq, xs, xq_perm, xs_perm, hq, hs, y_perm, total;
};
static FwdMx8Layout fwd_mx8_layout(const moe_config& c)
{
    FwdMx8Layout F;
    F.ws = ws_layout(c);
    const size_t tk = (size_t)c.T * c.K, R = (size_t)max_rows_of(c);
    size_t o = F.ws.total;
    F.amaps = o;   o += align_up(2 * (size_t)c.E * kTensorMapBytes);
    F.part = o;    o += align_up(mx8_part_bytes(c, max_rows_of(c)));
    F.ids = o;     o += align_up(tk * sizeof(int32_t));
    F.w = o;       o += align_up(tk * sizeof(float));
    F.counts = o;  o += align_up((size_t)c.E * sizeof(int32_t));
    F.kept = o;    o += align_up((size_t)c.E * sizeof(int32_t));
    F.offsets = o; o += align_up((size_t)(c.E + 1) * sizeof(int32_t));
    F.perm = o;    o += align_up(R * sizeof(int32_t));
    F.row_of = o;  o += align_up(tk * sizeof(int32_t));
    F.xq = o;      o += align_up((size_t)c.T * c.D);
    F.xs = o;      o += align_up((size_t)c.T * c.D / 32);
    F.xq_perm = o; o += align_up(R * c.D);
    F.xs_perm = o; o += align_up(R * c.D / 32);
    F.hq = o;      o += align_up(R * c.F);
    F.hs = o;      o += align_up(R * c.F / 32);
    F.y_perm = o;  o += align_up(R * c.D * 2);
    F.total = o;
    return F;
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_rmsnorm(int64_t T, int32_t D, int32_t dtype, const void* x, const void* residual, const float* gamma,
                       float eps, void* s, void* n, float* rstd, void* q, void* q_scales, void* stream)
{
    moe_status st = check_rows(T, D, dtype);
    if (st != MOE_OK) return st;
    if (D > 65536) return MOE_ERR_UNSUPPORTED;
    if (x == nullptr || gamma == nullptr || (n == nullptr && q == nullptr)) return MOE_ERR_ARG;
    if ((q == nullptr) != (q_scales == nullptr) || (s != nullptr && residual == nullptr)) return MOE_ERR_ARG;
    if (s != nullptr && s == n) return MOE_ERR_ARG;
    if (!(eps >= 0.0f) || !isfinite(eps)) return MOE_ERR_ARG;
    if (D % 8 != 0 || (q != nullptr && D % 32 != 0)) return MOE_ERR_ALIGN;
    if (!al16(x) || !al16(residual) || !al16(gamma) || !al16(s) || !al16(n) || !al4(rstd) || !al16(q))
        return MOE_ERR_ALIGN;
    return cuda_status(launch_rmsnorm(T, D, dtype, x, residual, gamma, eps, s, n, rstd, q, q_scales,
                                      static_cast<cudaStream_t>(stream)));
}

moe_status moe_rmsnorm_backward_workspace_size(int64_t T, int32_t D, size_t* bytes)
{
    moe_status st = check_rows(T, D, MOE_BF16);
    if (st != MOE_OK) return st;
    if (D > 65536) return MOE_ERR_UNSUPPORTED;
    if (D % 8 != 0) return MOE_ERR_ALIGN;
    if (bytes == nullptr) return MOE_ERR_ARG;
    *bytes = rmsnorm_backward_bytes(T, D);
    return MOE_OK;
}

moe_status moe_rmsnorm_backward(int64_t T, int32_t D, int32_t dtype, const void* dn, const void* ds, const void* s,
                                const float* gamma, const float* rstd, void* dx, float* dgamma, void* workspace,
                                size_t workspace_bytes, void* stream)
{
    moe_status st = check_rows(T, D, dtype);
    if (st != MOE_OK) return st;
    if (D > 65536) return MOE_ERR_UNSUPPORTED;
    if (!dn || !s || !gamma || !rstd || !dx || !dgamma) return MOE_ERR_ARG;
    if (D % 8 != 0) return MOE_ERR_ALIGN;
    if (!al16(dn) || !al16(ds) || !al16(s) || !al16(gamma) || !al4(rstd) || !al16(dx) || !al16(dgamma))
        return MOE_ERR_ALIGN;
    st = check_scratch(workspace, workspace_bytes, rmsnorm_backward_bytes(T, D));
    if (st != MOE_OK) return st;
    return cuda_status(launch_rmsnorm_backward(T, D, dtype, dn, ds, s, gamma, rstd, dx, dgamma, workspace,
                                               static_cast<cudaStream_t>(stream)));
}

static moe_status check_mx8_rows(int64_t rows, int32_t cols, int32_t dtype, const void* a, const void* q,
                                 const void* scales)
{
    moe_status st = check_rows(rows, cols, dtype);
    if (st != MOE_OK) return st;
    if (!a || !q || !scales) return MOE_ERR_ARG;
    if (cols % 32 != 0 || !al16(a) || !al16(q)) return MOE_ERR_ALIGN;
    // one block of 256 threads per 2048 elements
    if (rows > ((int64_t)INT32_MAX * 2048) / cols) return MOE_ERR_SHAPE;
    return MOE_OK;
}

moe_status moe_mx8_quantize(int64_t rows, int32_t cols, int32_t dtype, const void* x, void* q, void* scales,
                            void* stream)
{
    moe_status st = check_mx8_rows(rows, cols, dtype, x, q, scales);
    if (st != MOE_OK) return st;
    return cuda_status(launch_mx8_quantize(rows * cols, dtype, x, q, scales, static_cast<cudaStream_t>(stream)));
}

moe_status moe_mx8_dequantize(int64_t rows, int32_t cols, int32_t dtype, const void* q, const void* scales,
                              void* out, void* stream)
{
    moe_status st = check_mx8_rows(rows, cols, dtype, out, q, scales);
    if (st != MOE_OK) return st;
    return cuda_status(launch_mx8_dequantize(rows * cols, dtype, q, scales, out, static_cast<cudaStream_t>(stream)));
}

moe_status moe_mx8_prepare_weight(int32_t E, int32_t K, int32_t N, int32_t dtype, const void* w, void* q,
                                  void* scales, void* stream)
{
    if (E < 1 || K < 1 || N < 1) return MOE_ERR_SHAPE;
    if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_ARG;
    if (!w || !q || !scales) return MOE_ERR_ARG;
    if (K % 32 != 0 || N % 8 != 0 || !al16(w) || !al16(q)) return MOE_ERR_ALIGN;
    if (E > 65535 || K / 32 > 65535) return MOE_ERR_UNSUPPORTED;
    return cuda_status(launch_mx8_weight(E, K, N, dtype, w, q, scales, static_cast<cudaStream_t>(stream)));
}

moe_status moe_mx8_workspace_size(const moe_config* cfg, size_t* bytes)
{
    moe_status st = check_mx8_config(cfg);
    if (st != MOE_OK) return st;
    if (bytes == nullptr) return MOE_ERR_ARG;
    *bytes = mx8_ws_bytes(*cfg);
    return MOE_OK;
}

moe_status moe_expert_ffn_mx8(const moe_config* cfg, const void* xq, const void* xs, const int32_t* offsets,
                              const int32_t* perm, const float* topk_w, const moe_mx8_weights* weights, void* hq,
                              void* hs, void* y_perm, void* workspace, size_t workspace_bytes, void* stream)
{
    moe_status st = check_mx8_config(cfg);
    if (st != MOE_OK) return st;
    st = check_mx8_weights(weights);
    if (st != MOE_OK) return st;
    if (!xq || !xs || !offsets || !hq || !hs || !y_perm) return MOE_ERR_ARG;
    if ((perm == nullptr) != (topk_w == nullptr)) return MOE_ERR_ARG;
    if (!al16(xq) || !al16(xs) || !al16(hs)) return MOE_ERR_ALIGN;
    if (!al32(hq) || !al32(y_perm)) return MOE_ERR_ALIGN;  // stored 32 bytes at a time
    st = check_scratch(workspace, workspace_bytes, mx8_ws_bytes(*cfg));
    if (st != MOE_OK) return st;
    return cuda_status(launch_ffn_mx8(*cfg, max_rows_of(*cfg), xq, xs, offsets, perm, topk_w, *weights, hq, hs,
                                      y_perm, static_cast<char*>(workspace) + mx8_maps_at(),
                                      static_cast<char*>(workspace) + mx8_part_at(*cfg), static_cast<int*>(workspace),
                                      static_cast<cudaStream_t>(stream)));
}

moe_status moe_forward_mx8_workspace_size(const moe_config* cfg, size_t* bytes)
{
    moe_status st = check_mx8_config(cfg);
    if (st != MOE_OK) return st;
    if (bytes == nullptr) return MOE_ERR_ARG;
    *bytes = fwd_mx8_layout(*cfg).total;
    return MOE_OK;
}

moe_status moe_forward_mx8(const moe_config* cfg, const void* x, const void* xq, const void* xs,
                           const float* w_router, const void* w_router_terms, const float* router_bias,
                           const float* selection_bias, const float* logit_noise, const moe_mx8_weights* weights,
                           const void* y_add, void* y, float* losses, float* mean_prob, int32_t* counts,
                           int32_t* topk_ids, float* topk_w, void* workspace, size_t workspace_bytes, void* stream)
{
    moe_status st = check_mx8_config(cfg);
    if (st != MOE_OK) return st;
    if (cfg->F_shared != 0) return MOE_ERR_UNSUPPORTED;
    st = check_mx8_weights(weights);
    if (st != MOE_OK) return st;
    if (!x || !w_router || !y || (xq == nullptr) != (xs == nullptr)) return MOE_ERR_ARG;
    if (!al16(x) || !al16(xq) || !al16(xs) || !al16(y_add) || !al16(y) || !al16(w_router_terms)) return MOE_ERR_ALIGN;
    const moe_config& c = *cfg;
    const FwdMx8Layout F = fwd_mx8_layout(c);
    st = check_scratch(workspace, workspace_bytes, F.total);
    if (st != MOE_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    const int64_t max_rows = max_rows_of(c);
    int* status = reinterpret_cast<int*>(ws + F.ws.status);
    int32_t* ids = topk_ids ? topk_ids : reinterpret_cast<int32_t*>(ws + F.ids);
    float* w = topk_w ? topk_w : reinterpret_cast<float*>(ws + F.w);
    int32_t* cnt = counts ? counts : reinterpret_cast<int32_t*>(ws + F.counts);
    int32_t* kept = reinterpret_cast<int32_t*>(ws + F.kept);
    int32_t* offsets = reinterpret_cast<int32_t*>(ws + F.offsets);
    int32_t* perm = reinterpret_cast<int32_t*>(ws + F.perm);
    int32_t* row_of = reinterpret_cast<int32_t*>(ws + F.row_of);
    cudaError_t e = cudaSuccess;
    if (xq == nullptr) {
        e = launch_mx8_quantize(c.T * c.D, c.dtype, x, ws + F.xq, ws + F.xs, s);
        xq = ws + F.xq;
        xs = ws + F.xs;
    }
    const RouterPlan rp = router_plan(c);
    if (e == cudaSuccess)
        e = launch_router(c, rp, x, w_router, w_router_terms, router_bias, selection_bias, logit_noise, nullptr,
                          nullptr, nullptr, ids, w, mean_prob, losses, ws, F.ws, s);
    if (e == cudaSuccess)
        e = launch_dispatch_index(c, capacity_of(c), ids, cnt, kept, offsets, perm, row_of, ws, F.ws, s);
    if (e == cudaSuccess)
        e = launch_mx8_gather(c, xq, xs, offsets, perm, ws + F.xq_perm, ws + F.xs_perm, max_rows, status, s);
    if (e == cudaSuccess)
        e = launch_ffn_mx8(c, max_rows, ws + F.xq_perm, ws + F.xs_perm, offsets, perm, w, *weights, ws + F.hq,
                           ws + F.hs, ws + F.y_perm, ws + F.amaps, ws + F.part, status, s);
    if (e == cudaSuccess) e = launch_combine(c, ws + F.y_perm, row_of, nullptr, y_add, y, max_rows, s);
    return cuda_status(e);
}

static moe_status check_balance(const moe_config* cfg, int64_t S)
{
    moe_status st = moe_check_config(cfg);
    if (st != MOE_OK) return st;
    if (S < 1 || S > ((int64_t)INT32_MAX - 1) / cfg->E || cfg->T > (int64_t)INT32_MAX) return MOE_ERR_SHAPE;
    return MOE_OK;
}

moe_status moe_balance_workspace_size(const moe_config* cfg, int64_t S, size_t* bytes)
{
    moe_status st = check_balance(cfg, S);
    if (st != MOE_OK) return st;
    if (bytes == nullptr) return MOE_ERR_ARG;
    *bytes = balance_bytes(*cfg, S);
    return MOE_OK;
}

moe_status moe_balance_loss(const moe_config* cfg, int64_t S, const float* logits, const int32_t* topk_ids,
                            const int32_t* seq_starts, const uint8_t* token_mask, float c_balance, float c_z,
                            int32_t* counts, float* losses, float* seq_loss, float* dlogits, void* workspace,
                            size_t workspace_bytes, void* stream)
{
    moe_status st = check_balance(cfg, S);
    if (st != MOE_OK) return st;
    if (!logits || !topk_ids || !seq_starts || !counts || !losses || !seq_loss) return MOE_ERR_ARG;
    if (!isfinite(c_balance) || !isfinite(c_z)) return MOE_ERR_ARG;
    if (!al16(logits) || !al16(topk_ids) || !al4(seq_starts) || !al16(counts) || !al4(losses) || !al4(seq_loss) ||
        !al16(dlogits))
        return MOE_ERR_ALIGN;
    st = check_scratch(workspace, workspace_bytes, balance_bytes(*cfg, S));
    if (st != MOE_OK) return st;
    return cuda_status(launch_balance(*cfg, S, logits, topk_ids, seq_starts, token_mask, c_balance, c_z, counts,
                                      losses, seq_loss, dlogits, workspace, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
