// quantize.cu -- block-scaled e4m3 quantisation of activations (1 x 128
// blocks) and of expert weights (128 x 128 blocks, optionally transposed).
//
// Both kernels read every value once, keep it in registers while the block's
// max |x| is formed, and write one byte per value: they are bound by HBM
// (3 bytes per bf16 value, 5 per fp32 value, plus the scales).  Measured:
// 32768 x 7168 bf16 rows in 115 us (6.2 TB/s), 8 x 14336 x 4096 bf16 weights,
// transposed, in 231 us (6.1 TB/s), calls with changing inputs; a copy reaches
// 6.55.
#include <cuda_runtime.h>

#include "common.cuh"
#include "fp8.cuh"
#include "host_util.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kRowsPerCta = 8;  // one 32-byte sector of block-major scales
constexpr int kThreads = 256;

// The values of one 16-byte load, scaled and converted.
__device__ __forceinline__ uint2 quant16(const uint4 &v, float inv, const __nv_bfloat16 *)
{
    float f[8];
    unpack16(v, f, static_cast<const __nv_bfloat16 *>(nullptr));
    return make_uint2(cvt_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                      cvt_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
}
__device__ __forceinline__ uint32_t quant16(const uint4 &v, float inv, const float *)
{
    return cvt_e4m3x4(__uint_as_float(v.x) * inv, __uint_as_float(v.y) * inv, __uint_as_float(v.z) * inv,
                      __uint_as_float(v.w) * inv);
}

__device__ __forceinline__ uint32_t amax16(const uint4 &v, const float *)
{
    return max(max(v.x & 0x7FFFFFFFu, v.y & 0x7FFFFFFFu), max(v.z & 0x7FFFFFFFu, v.w & 0x7FFFFFFFu));
}
// bf16 bits order like the values too: the larger of each packed pair.
__device__ __forceinline__ uint32_t amax16(const uint4 &v, const __nv_bfloat16 *)
{
    const uint32_t w = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
    return max(w << 16, w & 0xFFFF0000u);
}

// Rows.  A warp holds kRowsPerCta rows of one 128-column block (all loads in
// flight at once), a CTA eight consecutive blocks of the same rows, so each
// row is read in 2 KB (bf16) or 4 KB (fp32) pieces and each scale store fills
// a 32-byte sector of the block-major scales.
template <typename T>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const T *x, uint8_t *q, float *scales, int64_t rows,
                                                                 int cols, int col_groups)
{
    pdl_enter();
    constexpr int V = Vec16<T>::n;                // values per load
    constexpr int L = kFp8Block / V;              // lanes per block of a row: 16 or 32
    constexpr int R = 32 / L;                     // rows per load of the warp
    constexpr int U = kRowsPerCta / R;            // loads in flight
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / col_groups) * kRowsPerCta;
    const int b = static_cast<int>(blockIdx.x % col_groups) * (kThreads / 32) + warp;
    const int c = b * kFp8Block + (lane % L) * V;
    if (b * kFp8Block >= cols) return;
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t r = row0 + u * R + lane / L;
        v[u] = (r < rows && c < cols) ? ld_stream16(x + r * cols + c) : make_uint4(0u, 0u, 0u, 0u);
    }
    float mine = 0.0f;  // lane j < 8: the scale of row j
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t r = row0 + u * R + lane / L;
        uint32_t m = amax16(v[u], static_cast<const T *>(nullptr));
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float2 s = fp8_scale(m);
        const float theirs = __shfl_sync(0xffffffffu, s.x, (lane % R) * L);
        if (lane / R == u) mine = theirs;
        if (r < rows && c < cols) {
            const auto p = quant16(v[u], s.y, static_cast<const T *>(nullptr));
            *reinterpret_cast<decltype(quant16(v[u], s.y, static_cast<const T *>(nullptr))) *>(q + r * cols + c) = p;
        }
    }
    if (lane < kRowsPerCta && row0 + lane < rows) scales[static_cast<int64_t>(b) * rows + row0 + lane] = mine;
}

// Weights.  One CTA per 128 x 128 block.  A thread holds groups of four
// consecutive rows of its V columns, so that the transposed form can pack a
// column's four rows into one word; the transposed tile goes through shared
// memory as [column][row] words, word w of column c at w ^ (c >> 2): free of
// bank conflicts for the word writes and the 16-byte reads.
template <typename T, bool TRANSPOSE>
__global__ void __launch_bounds__(kThreads) quantize_weights_kernel(const T *W, uint8_t *q, float *scales, int rows,
                                                                    int cols, int rb, int cb)
{
    pdl_enter();
    constexpr int V = Vec16<T>::n;
    constexpr int L = kFp8Block / V;           // threads across the columns
    constexpr int G = kThreads / L;            // four-row groups held at once
    constexpr int H = kFp8Block / (4 * G);     // row groups per thread
    __shared__ uint32_t part[kThreads / 32];
    __shared__ __align__(16) uint32_t tile[TRANSPOSE ? kFp8Block * 32 : 4];
    const int bc = static_cast<int>(blockIdx.x % cb);
    const int br = static_cast<int>((blockIdx.x / cb) % rb);
    const int e = static_cast<int>(blockIdx.x / (static_cast<unsigned>(cb) * rb));
    const int lc = (threadIdx.x % L) * V, g = threadIdx.x / L;
    const int c = bc * kFp8Block + lc;
    const int64_t base = static_cast<int64_t>(e) * rows * cols;
    uint4 v[H * 4];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < H * 4; ++i) {
        const int r = br * kFp8Block + (i / 4) * 4 * G + 4 * g + i % 4;
        v[i] = (r < rows && c < cols) ? ld_stream16(W + base + static_cast<int64_t>(r) * cols + c)
                                      : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < H * 4; ++i) m = max(m, amax16(v[i], static_cast<const T *>(nullptr)));
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) m = max(m, part[i]);
    const float2 s = fp8_scale(m);
    if (threadIdx.x == 0)
        scales[TRANSPOSE ? (static_cast<int64_t>(e) * cb + bc) * rb + br : (static_cast<int64_t>(e) * rb + br) * cb + bc] =
            s.x;
    if constexpr (!TRANSPOSE) {
#pragma unroll
        for (int i = 0; i < H * 4; ++i) {
            const int r = br * kFp8Block + (i / 4) * 4 * G + 4 * g + i % 4;
            if (r < rows && c < cols) {
                const auto p = quant16(v[i], s.y, static_cast<const T *>(nullptr));
                *reinterpret_cast<decltype(quant16(v[i], s.y, static_cast<const T *>(nullptr))) *>(
                    q + base + static_cast<int64_t>(r) * cols + c) = p;
            }
        }
    } else {
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int w = h * G + g;  // word (four rows) of the tile
            uint32_t p[4][V / 4];     // four rows of V columns, a byte each
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const auto k = quant16(v[h * 4 + i], s.y, static_cast<const T *>(nullptr));
                if constexpr (V == 8) {
                    p[i][0] = k.x;
                    p[i][V / 4 - 1] = k.y;
                } else {
                    p[i][0] = k;
                }
            }
#pragma unroll
            for (int j = 0; j < V / 4; ++j) {
                // 4 x 4 byte transpose
                const uint32_t a = __byte_perm(p[0][j], p[1][j], 0x5140), b = __byte_perm(p[2][j], p[3][j], 0x5140);
                const uint32_t a2 = __byte_perm(p[0][j], p[1][j], 0x7362), b2 = __byte_perm(p[2][j], p[3][j], 0x7362);
                const uint32_t o[4] = {__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632),
                                       __byte_perm(a2, b2, 0x5410), __byte_perm(a2, b2, 0x7632)};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int col = lc + 4 * j + u;
                    tile[col * 32 + (w ^ (col >> 2))] = o[u];
                }
            }
        }
        __syncthreads();
        const int64_t obase = static_cast<int64_t>(e) * rows * cols;
#pragma unroll
        for (int i = 0; i < kFp8Block * 8 / kThreads; ++i) {
            const int idx = i * kThreads + threadIdx.x;
            const int col = idx >> 3, piece = idx & 7;       // 16 rows of one column
            const int x = col >> 2;
            const uint4 t = *reinterpret_cast<const uint4 *>(&tile[col * 32 + ((piece ^ (x >> 2)) << 2)]);
            // words of the piece sit at (word ^ (x & 3))
            const bool s1 = x & 1, s2 = x & 2;
            uint4 a = s1 ? make_uint4(t.y, t.x, t.w, t.z) : t;
            a = s2 ? make_uint4(a.z, a.w, a.x, a.y) : a;
            const int oc = bc * kFp8Block + col, r = br * kFp8Block + piece * 16;
            if (oc < cols && r < rows) st16(q + obase + static_cast<int64_t>(oc) * rows + r, a);
        }
    }
}

}  // namespace

cudaError_t launch_quantize_rows(int dtype, const void *x, int64_t rows, int cols, void *q, float *scales,
                                 cudaStream_t s)
{
    const int groups = (fp8_blocks(cols) + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t ctas = (rows + kRowsPerCta - 1) / kRowsPerCta * groups;
    if (ctas == 0) return cudaSuccess;
    if (ctas >= (static_cast<int64_t>(1) << 31)) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(ctas));
    if (dtype == kF32)
        return launch_k(quantize_rows_kernel<float>, grid, dim3(kThreads), 0, s, static_cast<const float *>(x),
                        static_cast<uint8_t *>(q), scales, rows, cols, groups);
    return launch_k(quantize_rows_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, s,
                    static_cast<const __nv_bfloat16 *>(x), static_cast<uint8_t *>(q), scales, rows, cols, groups);
}

cudaError_t launch_quantize_weights(int dtype, const void *W, int E, int rows, int cols, int transpose, void *q,
                                    float *scales, cudaStream_t s)
{
    const int rb = fp8_blocks(rows), cb = fp8_blocks(cols);
    const int64_t ctas = static_cast<int64_t>(E) * rb * cb;
    if (ctas >= (static_cast<int64_t>(1) << 31)) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(ctas));
    auto go = [&](auto *kernel, auto *w) {
        return launch_k(kernel, grid, dim3(kThreads), 0, s, w, static_cast<uint8_t *>(q), scales, rows, cols, rb, cb);
    };
    if (dtype == kF32) {
        const float *w = static_cast<const float *>(W);
        return transpose ? go(quantize_weights_kernel<float, true>, w) : go(quantize_weights_kernel<float, false>, w);
    }
    const __nv_bfloat16 *w = static_cast<const __nv_bfloat16 *>(W);
    return transpose ? go(quantize_weights_kernel<__nv_bfloat16, true>, w)
                     : go(quantize_weights_kernel<__nv_bfloat16, false>, w);
}

}  // namespace moe
