// ops_api.cu -- extern "C" entry points of the block-scaled e4m3 operators
// and of the balance loss (declared in include/moe.h): argument validation,
// workspace carving, launches.  No allocation, no host synchronisation.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/moe.h"
#include "api_internal.h"
#include "common.cuh"
#include "fp8.cuh"
#include "kernels.h"

namespace {

using namespace moe;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool given(const void *p) { return p != nullptr && aligned16(p); }
bool given4(const void *p) { return p != nullptr && aligned4(p); }
// Rows of E values are read four at a time if E is a multiple of four.
bool given_rows(const void *p, int32_t dtype, int32_t E)
{
    const uintptr_t es = dtype == MOE_F32 ? 4 : 2;
    return p != nullptr && reinterpret_cast<uintptr_t>(p) % (E % 4 == 0 ? 4 * es : es) == 0;
}
constexpr int64_t kMaxRows = static_cast<int64_t>(1) << 31;
constexpr int32_t kMaxWidth = 1 << 30;  // 32-bit column arithmetic keeps room for a tile

// Runs an entry point's body; nothing thrown inside crosses the C boundary.
template <typename F> moe_status guarded(F &&f)
{
    try {
        return f();
    } catch (...) {
        return MOE_ERR_CUDA;
    }
}

moe_status done(cudaError_t err) { return err == cudaSuccess ? MOE_OK : record_cuda_error(err); }

// Scales that are powers of two are applied by the tensor core, others on
// the CUDA cores.
cudaError_t product(int32_t any_scales, const Fp8GemmArgs &g, cudaStream_t s)
{
    return any_scales ? launch_gemm_fp8(g, device_sms(), s) : launch_gemm_mxfp8(g, device_sms(), s);
}

size_t align256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

struct FfnLayout {
    size_t xq, xs, hq, hs, total;
};

FfnLayout ffn_layout(const moe_config *c)
{
    const size_t A = static_cast<size_t>(c->N) * static_cast<size_t>(c->k);
    FfnLayout L{};
    L.xq = 0;
    L.xs = L.xq + align256(A * c->d_model);
    L.hq = L.xs + align256(A * fp8_blocks(c->d_model) * 4);
    L.hs = L.hq + align256(A * c->d_ff);
    L.total = L.hs + align256(A * fp8_blocks(c->d_ff) * 4) + 256;
    return L;
}

moe_status check_fp8_config(const moe_config *c)
{
    const moe_status st = validate_config(c);
    if (st != MOE_OK) return st;
    if (c->dtype != MOE_BF16 || c->d_model % 16 != 0 || c->d_ff % 16 != 0) return MOE_ERR_UNSUPPORTED;
    if (c->d_model > kMaxWidth || c->d_ff > kMaxWidth) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

moe_status check_balance(int32_t dtype, int32_t scores, int64_t N, int32_t E, int32_t S)
{
    if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (scores != MOE_SCORES_SOFTMAX && scores != MOE_SCORES_SIGMOID) return MOE_ERR_INVALID_ARG;
    if (N < 0 || E <= 0 || S <= 0) return MOE_ERR_INVALID_ARG;
    if (E > kMaxE || N >= kMaxRows || static_cast<int64_t>(S) * ((E + 31) / 32) >= kMaxRows) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_quantize_rows(int32_t dtype, const void *x, int64_t rows, int32_t cols, void *q, float *scales,
                             moe_stream_t stream)
{
    return guarded([&] {
        if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
        if (rows < 0 || cols <= 0) return MOE_ERR_INVALID_ARG;
        if (cols % 16 != 0 || cols > kMaxWidth || rows >= kMaxRows) return MOE_ERR_UNSUPPORTED;
        if (rows == 0) return MOE_OK;
        if (!given(x) || !given(q) || !given4(scales)) return MOE_ERR_INVALID_ARG;
        return done(launch_quantize_rows(dtype, x, rows, cols, q, scales, reinterpret_cast<cudaStream_t>(stream)));
    });
}

moe_status moe_quantize_weights(int32_t dtype, const void *W, int32_t E, int32_t rows, int32_t cols,
                                int32_t transpose, void *q, float *scales, moe_stream_t stream)
{
    return guarded([&] {
        if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
        if (E <= 0 || rows <= 0 || cols <= 0 || (transpose != 0 && transpose != 1)) return MOE_ERR_INVALID_ARG;
        if (rows % 16 != 0 || cols % 16 != 0 || rows > kMaxWidth || cols > kMaxWidth) return MOE_ERR_UNSUPPORTED;
        if (static_cast<int64_t>(E) * fp8_blocks(rows) * fp8_blocks(cols) >= kMaxRows) return MOE_ERR_UNSUPPORTED;
        if (!given(W) || !given(q) || !given4(scales)) return MOE_ERR_INVALID_ARG;
        return done(launch_quantize_weights(dtype, W, E, rows, cols, transpose, q, scales,
                                            reinterpret_cast<cudaStream_t>(stream)));
    });
}

moe_status moe_expert_matmul_fp8(int64_t rows, int32_t n, int32_t k, int32_t E, const void *a_q,
                                 const float *a_scales, const int32_t *offsets, const void *w_q,
                                 const float *w_scales, int32_t any_scales, int32_t out_dtype, void *out,
                                 int32_t *dev_status, moe_stream_t stream)
{
    return guarded([&] {
        if (out_dtype != MOE_F32 && out_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
        if (rows < 0 || n <= 0 || k <= 0 || E <= 0 || (any_scales != 0 && any_scales != 1)) return MOE_ERR_INVALID_ARG;
        if (E > kMaxE || n % 16 != 0 || k % 16 != 0 || n > kMaxWidth || k > kMaxWidth || rows >= kMaxRows)
            return MOE_ERR_UNSUPPORTED;
        if (!given4(offsets) || !aligned4(dev_status) || !given(w_q) || !given4(w_scales)) return MOE_ERR_INVALID_ARG;
        if (rows == 0) return MOE_OK;
        if (!given(a_q) || !given4(a_scales) || !given(out)) return MOE_ERR_INVALID_ARG;
        Fp8GemmArgs g{};
        g.epi = out_dtype == MOE_F32 ? kFp8F32 : kFp8Bf16;
        g.a = a_q;
        g.a_scales = a_scales;
        g.offsets = offsets;
        g.w = w_q;
        g.w_scales = w_scales;
        g.out = out;
        g.status = dev_status;
        g.rows = rows;
        g.E = E;
        g.n = n;
        g.k = k;
        return done(product(any_scales, g, reinterpret_cast<cudaStream_t>(stream)));
    });
}

size_t moe_expert_ffn_fp8_workspace_size(const moe_config *cfg)
{
    return check_fp8_config(cfg) == MOE_OK ? ffn_layout(cfg).total : 0;
}

moe_status moe_expert_ffn_fp8(const moe_config *cfg, const void *x_sorted, const int32_t *offsets,
                              const moe_fp8_experts *w, void *y_sorted, int32_t *dev_status, void *ws,
                              size_t ws_bytes, moe_stream_t stream)
{
    return guarded([&] {
        const moe_status st = check_fp8_config(cfg);
        if (st != MOE_OK) return st;
        const bool swiglu = cfg->act == MOE_ACT_SWIGLU;
        if (!given4(offsets) || !aligned4(dev_status) || !w) return MOE_ERR_INVALID_ARG;
        if (cfg->N > 0 && (!given(x_sorted) || !given(y_sorted))) return MOE_ERR_INVALID_ARG;
        if (!given(w->W1) || !given4(w->W1_scales) || !given(w->W2) || !given4(w->W2_scales)) return MOE_ERR_INVALID_ARG;
        if (swiglu ? (!given(w->W3) || !given4(w->W3_scales) || w->b1) : (w->W3 || w->W3_scales)) return MOE_ERR_INVALID_ARG;
        if (!aligned16(w->b1) || !aligned16(w->b2)) return MOE_ERR_INVALID_ARG;
        if (w->any_scales != 0 && w->any_scales != 1) return MOE_ERR_INVALID_ARG;
        const FfnLayout L = ffn_layout(cfg);
        if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || ws_bytes < L.total) return MOE_ERR_WORKSPACE;
        if (cfg->N == 0) return MOE_OK;
        cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
        uint8_t *base = static_cast<uint8_t *>(ws);
        float *xs = reinterpret_cast<float *>(base + L.xs), *hs = reinterpret_cast<float *>(base + L.hs);
        const int64_t rows = cfg->N * cfg->k;
        cudaError_t err = launch_quantize_rows(kBF16, x_sorted, rows, cfg->d_model, base + L.xq, xs, s);
        if (err != cudaSuccess) return record_cuda_error(err);
        Fp8GemmArgs g{};
        g.epi = swiglu ? kFp8Swiglu : kFp8Gelu;
        g.a = base + L.xq;
        g.a_scales = xs;
        g.offsets = offsets;
        g.w = w->W1;
        g.w_scales = w->W1_scales;
        g.w3 = w->W3;
        g.w3_scales = w->W3_scales;
        g.bias = w->b1;
        g.out = base + L.hq;
        g.h_scales = hs;
        g.status = dev_status;
        g.rows = rows;
        g.E = cfg->E;
        g.n = cfg->d_ff;
        g.k = cfg->d_model;
        g.early = 1;  // each product follows a kernel of this call, which writes only its rows
        if ((err = product(w->any_scales, g, s)) != cudaSuccess) return record_cuda_error(err);
        g.epi = kFp8Bf16;
        g.a = base + L.hq;
        g.a_scales = hs;
        g.w = w->W2;
        g.w_scales = w->W2_scales;
        g.w3 = nullptr;
        g.w3_scales = nullptr;
        g.bias = w->b2;
        g.out = y_sorted;
        g.h_scales = nullptr;
        g.n = cfg->d_model;
        g.k = cfg->d_ff;
        return done(product(w->any_scales, g, s));
    });
}

size_t moe_balance_loss_workspace_size(int64_t N, int32_t E, int32_t S)
{
    return check_balance(MOE_F32, MOE_SCORES_SOFTMAX, N, E, S) == MOE_OK ? balance_workspace(N, E, S) : 0;
}

moe_status moe_balance_loss(int32_t dtype, int32_t scores, const void *logits, const int32_t *topk_ids,
                            const int32_t *seq_offsets, const uint8_t *token_mask, int64_t N, int32_t E, int32_t k,
                            int32_t S, float *loss_out, int32_t *counts_out, float *seq_weight_out,
                            int32_t *dev_status, void *ws, size_t ws_bytes, moe_stream_t stream)
{
    return guarded([&] {
        const moe_status st = check_balance(dtype, scores, N, E, S);
        if (st != MOE_OK) return st;
        if (k <= 0 || k > E) return MOE_ERR_INVALID_ARG;
        if (k > kMaxK || N * k >= kMaxRows) return MOE_ERR_UNSUPPORTED;
        if (!seq_offsets && S != 1) return MOE_ERR_INVALID_ARG;
        if (N > 0 && (!given_rows(logits, dtype, E) || !given4(topk_ids))) return MOE_ERR_INVALID_ARG;
        if (!given4(loss_out) || !given4(counts_out) || !given4(seq_weight_out)) return MOE_ERR_INVALID_ARG;
        if (!aligned4(seq_offsets) || !aligned4(dev_status)) return MOE_ERR_INVALID_ARG;
        if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || ws_bytes < balance_workspace(N, E, S))
            return MOE_ERR_WORKSPACE;
        BalanceArgs a{};
        a.dtype = dtype;
        a.sigmoid = scores == MOE_SCORES_SIGMOID;
        a.logits = logits;
        a.ids = topk_ids;
        a.seq_offsets = seq_offsets;
        a.mask = token_mask;
        a.N = N;
        a.E = E;
        a.k = k;
        a.S = S;
        a.counts = counts_out;
        a.seq_weight = seq_weight_out;
        a.loss = loss_out;
        a.status = dev_status;
        a.ws = ws;
        return done(launch_balance_loss(a, reinterpret_cast<cudaStream_t>(stream)));
    });
}

moe_status moe_balance_loss_backward(int32_t dtype, int32_t scores, const void *logits, const int32_t *seq_offsets,
                                     const uint8_t *token_mask, int64_t N, int32_t E, int32_t S,
                                     const int32_t *counts, const float *seq_weight, float coef, const float *dloss,
                                     float *dlogits, moe_stream_t stream)
{
    return guarded([&] {
        const moe_status st = check_balance(dtype, scores, N, E, S);
        if (st != MOE_OK) return st;
        if (!seq_offsets && S != 1) return MOE_ERR_INVALID_ARG;
        if (!std::isfinite(coef)) return MOE_ERR_INVALID_ARG;
        if (N == 0) return MOE_OK;
        if (!given_rows(logits, dtype, E) || !given4(counts) || !given4(seq_weight) || !given_rows(dlogits, MOE_F32, E))
            return MOE_ERR_INVALID_ARG;
        if (!aligned4(seq_offsets) || !aligned4(dloss)) return MOE_ERR_INVALID_ARG;
        BalanceArgs a{};
        a.dtype = dtype;
        a.sigmoid = scores == MOE_SCORES_SIGMOID;
        a.logits = logits;
        a.seq_offsets = seq_offsets;
        a.mask = token_mask;
        a.N = N;
        a.E = E;
        a.S = S;
        a.counts = const_cast<int32_t *>(counts);
        a.seq_weight = const_cast<float *>(seq_weight);
        a.dloss = dloss;
        a.coef = coef;
        a.dlogits = dlogits;
        return done(launch_balance_backward(a, device_sms(), reinterpret_cast<cudaStream_t>(stream)));
    });
}

}  // extern "C"
