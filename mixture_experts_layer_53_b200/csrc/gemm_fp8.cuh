// gemm_fp8.cuh -- pieces shared by the two grouped GEMMs on block-scaled e4m3
// operands: arguments, the tile list over ragged slices, the wait for TMEM
// loads.
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "fp8.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace moe {
namespace fp8 {

using namespace sm100;

enum { EPI_SWIGLU = 0, EPI_GELU = 1, EPI_BF16 = 2, EPI_F32 = 3 };

constexpr int BK = kFp8Block;    // a k-block: one scale block, one 128-byte swizzled row
constexpr int SUM_WARPS = 8;     // epilogue warps: lane quarter x column half
constexpr int FIRST_SUM_WARP = 4;
constexpr int THREADS = 32 * (FIRST_SUM_WARP + SUM_WARPS);
constexpr int LAUNCH_REGS = 168;  // a thread of 384 launches with

struct GemmArgs {
    const int32_t *offsets;
    const uint8_t *a, *w, *w3;  // [rows, K], [E, n_out, K], [E, n_out, K] (SwiGLU)
    const float *a_scales;   // [kblocks, rows]
    const float *w_scales;   // [E, nblocks, kblocks]
    const float *w3_scales;  // SwiGLU
    const __nv_bfloat16 *bias;  // [E, n_out] or null
    void *out;               // bf16 / f32 rows, or e4m3 h
    float *h_scales;         // [nblocks, rows] (SwiGLU, GELU)
    int32_t *status;
    int64_t rows;
    int E, K, n_out, n_tiles;
    int early;               // offsets and weights are older than the stream's previous kernel
};

inline GemmArgs gemm_args(const Fp8GemmArgs &a, int tile_n)
{
    GemmArgs g{};
    g.offsets = a.offsets;
    g.a = static_cast<const uint8_t *>(a.a);
    g.w = static_cast<const uint8_t *>(a.w);
    g.w3 = static_cast<const uint8_t *>(a.w3);
    g.a_scales = a.a_scales;
    g.w_scales = a.w_scales;
    g.w3_scales = a.w3_scales;
    g.bias = static_cast<const __nv_bfloat16 *>(a.bias);
    g.out = a.out;
    g.h_scales = a.h_scales;
    g.status = a.status;
    g.rows = a.rows;
    g.E = a.E;
    g.K = a.k;
    g.n_out = a.n;
    g.n_tiles = (a.n + tile_n - 1) / tile_n;
    g.early = a.early;
    return g;
}

// Slices of the rows and the prefix of their m-tile counts.  Whatever
// `offsets` says, the slices lie inside 0 .. rows and none begins before the
// end of an earlier one, so that there are never more tiles than the launch
// allows for (a cluster that shares a tile takes one, and waits for its CTAs).
struct Slices {
    int warp_sum[kMaxE / 32];
    int off[kMaxE];
    int end[kMaxE];
    int mt[kMaxE + 1];
};

// All threads of the CTA; ends with the CTA synchronised.
template <int TILE_M> __device__ __forceinline__ void load_slices(Slices *c, const GemmArgs &g)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int tiles = 0;
    bool falls = false;
    if (threadIdx.x < kMaxE) {
        const int e = threadIdx.x;
        if (e < g.E) {
            const int64_t lo = min64(max64(g.offsets[e], 0), g.rows), hi = min64(max64(g.offsets[e + 1], lo), g.rows);
            c->off[e] = static_cast<int>(lo);
            c->end[e] = static_cast<int>(hi);
            tiles = static_cast<int>((hi - lo + TILE_M - 1) / TILE_M);
            falls = g.offsets[e + 1] < g.offsets[e];
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, tiles, o);
            if (lane >= o) tiles += v;
        }
        if (lane == 31) c->warp_sum[warp] = tiles;
        if (e == 0) c->mt[0] = 0;
    }
    if (__syncthreads_or(falls)) {  // offsets that decrease somewhere
        if (threadIdx.x == 0) {
            int end = 0, sum = 0;
            for (int e = 0; e < g.E; ++e) {
                c->off[e] = end = max(end, c->off[e]);
                c->end[e] = end = max(end, c->end[e]);
                sum += static_cast<int>((static_cast<unsigned>(end - c->off[e]) + TILE_M - 1) / TILE_M);
                c->mt[e + 1] = sum;
            }
        }
        __syncthreads();
        return;
    }
    if (threadIdx.x < kMaxE) {
        for (int w = 0; w < warp; ++w) tiles += c->warp_sum[w];
        c->mt[threadIdx.x + 1] = tiles;
    }
    __syncthreads();
}

struct Tile {
    int e, m_tile, n_tile;
};

__device__ __forceinline__ Tile decode_tile(int t, const Slices *c, int E, int n_tiles)
{
    const int q = t / n_tiles;
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (c->mt[mid] <= q) lo = mid;
        else hi = mid - 1;
    }
    const int mt_e = c->mt[lo + 1] - c->mt[lo];
    const int local = t - c->mt[lo] * n_tiles;
    return Tile{lo, local % mt_e, local / mt_e};
}

// Until this thread's TMEM loads have landed; r ties the uses of the loaded
// values to this point.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}

}  // namespace fp8
}  // namespace moe
