// gemm_fp8.cuh -- pieces shared by the grouped GEMMs on block-scaled e4m3
// operands: arguments, the tile list over ragged slices, TMEM loads and the
// epilogues' stores.
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

constexpr int BM = 128;          // rows of a CTA's tile
constexpr int BN = 256;          // accumulator columns of a tile
constexpr int BK = kFp8Block;    // a k-block: one scale block, one 128-byte swizzled row
constexpr int SUM_WARPS = 8;     // epilogue warps: lane quarter x column half
constexpr int FIRST_SUM_WARP = 4;
constexpr int THREADS = 32 * (FIRST_SUM_WARP + SUM_WARPS);
constexpr int LAUNCH_REGS = 168;  // a thread of 384 launches with
constexpr int CHUNK_BYTES = 32 * 64;  // a warp's staging: 32 rows of 64 bytes

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

template <int EPI> __host__ __device__ constexpr int out_cols() { return EPI == EPI_SWIGLU ? 128 : 256; }

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

// 32 values of a thread's row from column c on, as e4m3.
__device__ __forceinline__ void store_h32(const float *h, float inv, uint8_t *row, int c, int n_out)
{
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        if (c + 16 * p < n_out) {
            const float *v = h + 16 * p;
            st16(row + c + 16 * p,
                 make_uint4(cvt_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                            cvt_e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv),
                            cvt_e4m3x4(v[8] * inv, v[9] * inv, v[10] * inv, v[11] * inv),
                            cvt_e4m3x4(v[12] * inv, v[13] * inv, v[14] * inv, v[15] * inv)));
        }
    }
}

// The two halves of a row's 128 hidden units (SwiGLU: two warps) exchange
// their largest |h|.  Two sets of values by phase: a warp that is a tile
// ahead writes the other set, and it cannot be two ahead.
struct Exchange {
    uint32_t amax[2][2][BM];  // [phase][half][row]
    uint64_t there[4];        // per lane quarter: both halves' values are there (count 2)
};
__device__ __forceinline__ bool exchange_amax(Exchange *x, uint32_t &m, uint32_t phase, int quarter, int half, int lane,
                                              volatile int *abort_flag, int32_t *status)
{
    x->amax[phase][half][quarter * 32 + lane] = m;
    __syncwarp();
    if (lane == 0) mbar_arrive(&x->there[quarter]);
    if (!__all_sync(0xffffffffu, mbar_wait(&x->there[quarter], phase, abort_flag, status))) return false;
    m = max(m, x->amax[phase][half ^ 1][quarter * 32 + lane]);
    return true;
}

// Eight bias values of columns c .. c+7 (zero past n_out or without bias).
__device__ __forceinline__ void bias8(const __nv_bfloat16 *bias, int c, int n_out, float (&b)[8])
{
    const uint4 v = (bias && c < n_out) ? __ldg(reinterpret_cast<const uint4 *>(bias + c)) : make_uint4(0u, 0u, 0u, 0u);
    unpack16(v, b, static_cast<const __nv_bfloat16 *>(nullptr));
}

// Writes the four 16-byte pieces that each lane holds of its own row as
// 64-byte row segments: through the warp's staging buffer, piece j of row r
// at j ^ ((r >> 1) & 3) (free of bank conflicts both ways).
__device__ __forceinline__ void store_chunk(const uint4 (&p)[4], uint8_t *stage, uint8_t *out, int64_t row_bytes,
                                            int64_t row_first, int64_t row_end, int64_t byte0, int64_t byte_end, int lane)
{
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j) st16(stage + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4), p[j]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2), j = lane & 3;
        const uint4 v = *reinterpret_cast<const uint4 *>(stage + r * 64 + ((j ^ ((r >> 1) & 3)) << 4));
        if (row_first + r < row_end && byte0 + j * 16 < byte_end)
            st16(out + (row_first + r) * row_bytes + byte0 + j * 16, v);
    }
}

// A chunk of 32 result columns from column col on (v: a thread's row, bias
// not yet added), as bf16 or fp32 rows.
template <int EPI>
__device__ __forceinline__ void store_columns(float (&v)[32], const __nv_bfloat16 *bias, const GemmArgs &g, int col,
                                              int64_t row_first, int64_t row_end, uint8_t *stage, int lane)
{
    constexpr int ES = EPI == EPI_BF16 ? 2 : 4;
    const int64_t row_bytes = static_cast<int64_t>(g.n_out) * ES;
    if (bias) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float b[8];
            bias8(bias, col + 8 * j, g.n_out, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[8 * j + i] += b[i];
        }
    }
#pragma unroll
    for (int q = 0; q < ES / 2; ++q) {
        uint4 p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (EPI == EPI_BF16) p[j] = pack16(v + 8 * j, static_cast<const __nv_bfloat16 *>(nullptr));
            else p[j] = pack16(v + 16 * q + 4 * j, static_cast<const float *>(nullptr));
        }
        store_chunk(p, stage, static_cast<uint8_t *>(g.out), row_bytes, row_first, row_end,
                    static_cast<int64_t>(col) * ES + 64 * q, row_bytes, lane);
    }
}

}  // namespace fp8
}  // namespace moe
