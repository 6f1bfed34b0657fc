// gemm_fp8_sm100.cu -- ragged grouped GEMM on block-scaled e4m3 operands
// (tcgen05 kind::f8f6f4, 128 x 256 tiles, one CTA per tile).
//
// For row r of expert e (rows offsets[e] .. offsets[e+1]-1):
//   y[r, c] = sum_kb sA[kb, r] sW[e, c / 128, kb] sum_{k in kb} a[r, k] w[e, c, k]
// with kb the 128-column blocks of the reduction.  A k-block of 128 e4m3
// values is one 128-byte swizzled row, so a pipeline stage is exactly one
// scale block: the MMA of each k-block starts a fresh TMEM accumulator, and
// the epilogue warps read it back and add it, scaled, to fp32 sums that stay
// in their registers for the whole tile.  Sums inside a block are the tensor
// core's fp32 accumulation over 128 products, all others fp32 multiply-adds.
//
// Warp roles (384 threads, one CTA per SM, persistent over the tile list
// (expert, n-tile, m-tile), m-tiles innermost so that CTAs that run at the
// same time share an expert's weight tile through L2):
//   warp 0      TMA producer: A (16 KB) and W (32 KB) tiles, four stages
//   warp 1      allocates 512 TMEM columns (two accumulators); one lane
//               issues the MMAs (M = 128, N = 256, K = 32)
//   warps 2, 3  idle (a register split is made by whole warpgroups)
//   warps 4-11  sums and epilogue: a warp owns 32 rows (its TMEM lane
//               quarter) and half of the columns, 128 fp32 sums a thread
// The sums and two 32-column chunks on their way from TMEM need more than
// the 168 registers that 384 threads launch with: the first warpgroup hands
// registers over (128 x 56 + 256 x 224 = 384 x 168).
//
// SwiGLU: the W tile holds 128 rows of W1 and the same 128 rows of W3; a
// thread holds the gate and the up columns of 64 hidden units.  The 128
// hidden units of the tile are one scale block of h, so the epilogue
// quantises them on the spot (the two halves of a row exchange their max
// |h| through shared memory).  GELU: two scale blocks per tile, one per half.
#include <cuda.h>

#include "common.cuh"
#include "fp8.cuh"
#include "host_util.h"
#include "kernels.h"
#include "sm100.cuh"

namespace moe {
namespace {

using namespace sm100;

constexpr int BM = 128;
constexpr int BN = 256;
constexpr int BK = kFp8Block;
constexpr int STAGES = 4;
constexpr int A_BYTES = BM * BK;
constexpr int W_BYTES = BN * BK;
constexpr int STAGE_BYTES = A_BYTES + W_BYTES;
constexpr int SUM_WARPS = 8;
constexpr int FIRST_SUM_WARP = 4;
constexpr int THREADS = 32 * (FIRST_SUM_WARP + SUM_WARPS);
constexpr int LAUNCH_REGS = 168, ROLE_REGS = 56, SUM_REGS = 224;
static_assert(32 * FIRST_SUM_WARP * ROLE_REGS + 32 * SUM_WARPS * SUM_REGS <= THREADS * LAUNCH_REGS, "register split");
constexpr uint32_t TMEM_COLS = 512;
constexpr int CHUNK_BYTES = 32 * 64;  // a warp's staging: 32 rows of 64 bytes

enum { EPI_SWIGLU = 0, EPI_GELU = 1, EPI_BF16 = 2, EPI_F32 = 3 };

struct Args {
    const int32_t *offsets;
    const float *a_scales;   // [kblocks, rows]
    const float *w_scales;   // [E, nblocks, kblocks]
    const float *w3_scales;  // SwiGLU
    const __nv_bfloat16 *bias;  // [E, n_out] or null
    void *out;               // bf16 / f32 rows, or e4m3 h
    float *h_scales;         // [nblocks, rows] (SwiGLU, GELU)
    int32_t *status;
    int64_t rows;
    int E, K, n_out, n_tiles;
};

struct Ctl {
    alignas(1024) uint8_t stage[SUM_WARPS][CHUNK_BYTES];
    uint32_t amax[2][2][BM];  // [phase][half][row]
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t exchanged[4];  // per lane quarter: both halves' amax are there
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    int warp_sum[8];
    int off[kMaxE + 1];
    int end[kMaxE];
    int mt[kMaxE + 1];
};

constexpr size_t kSmemBytes = 1024 + STAGES * STAGE_BYTES + sizeof(Ctl);
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

struct Tile {
    int e, m_tile, n_tile;
};

__device__ __forceinline__ Tile decode_tile(int t, const Ctl *c, int E, int n_tiles)
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

// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 inputs, fp32 accumulate.
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor of kind::f8f6f4: fp32 accumulator [4,6) = 1, A and B
// e4m3 (0), both K-major, N >> 3 at [17,23), M >> 4 at [24,29).
constexpr uint32_t idesc_f8(int M, int N)
{
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Two fp32 sums in one register pair.
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &lo, float &hi)
{
    uint32_t a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
    lo = __uint_as_float(a);
    hi = __uint_as_float(b);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
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

// 64 values of a thread's row from column c on, as e4m3.
__device__ __forceinline__ void store_h64(const float (&h)[64], float inv, uint8_t *row, int c, int n_out)
{
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        if (c + 16 * p < n_out) {
            uint4 v;
            v.x = cvt_e4m3x4(h[16 * p] * inv, h[16 * p + 1] * inv, h[16 * p + 2] * inv, h[16 * p + 3] * inv);
            v.y = cvt_e4m3x4(h[16 * p + 4] * inv, h[16 * p + 5] * inv, h[16 * p + 6] * inv, h[16 * p + 7] * inv);
            v.z = cvt_e4m3x4(h[16 * p + 8] * inv, h[16 * p + 9] * inv, h[16 * p + 10] * inv, h[16 * p + 11] * inv);
            v.w = cvt_e4m3x4(h[16 * p + 12] * inv, h[16 * p + 13] * inv, h[16 * p + 14] * inv, h[16 * p + 15] * inv);
            st16(row + c + 16 * p, v);
        }
    }
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
                                            int64_t row_first, int64_t row_end, int byte0, int64_t byte_end, int lane)
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

// First accumulator column of a thread's chunk c of 32: SwiGLU, 64 gate and
// then 64 up columns; else 128 consecutive ones.
template <int EPI> __device__ __forceinline__ uint32_t chunk_col(int c, int half)
{
    return EPI == EPI_SWIGLU ? (c >> 1) * 128 + half * 64 + (c & 1) * 32 : half * 128 + c * 32;
}

template <int EPI>
__global__ void __launch_bounds__(THREADS, 1)
    ffn_gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
                        const __grid_constant__ CUtensorMap tmW3, const Args g)
{
    pdl_enter();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *tiles = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                 ~static_cast<uintptr_t>(1023));
    Ctl *ctl = reinterpret_cast<Ctl *>(tiles + STAGES * STAGE_BYTES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *abort_flag = &ctl->abort;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ctl->tfull[b], 1);
            mbar_init(&ctl->tempty[b], SUM_WARPS);
        }
        for (int q = 0; q < 4; ++q) mbar_init(&ctl->exchanged[q], 2);
        mbar_init(&ctl->drain, 1);
        ctl->abort = 0;
        ctl->mt[0] = 0;
        fence_mbar_init();
    }
    if (threadIdx.x == 32) {
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmW);
        if (EPI == EPI_SWIGLU) prefetch_tmap(&tmW3);
    }
    if (warp == 1) {
        tmem_alloc(&ctl->tmem_base, TMEM_COLS);
        tmem_relinquish();
    }
    // slices (held inside 0 .. rows whatever offsets says) and the prefix of
    // their m-tile counts
    int tiles_e = 0;
    if (threadIdx.x < kMaxE) {
        const int e = threadIdx.x;
        if (e < g.E) {
            const int64_t lo = min64(max64(g.offsets[e], 0), g.rows), hi = min64(max64(g.offsets[e + 1], lo), g.rows);
            ctl->off[e] = static_cast<int>(lo);
            ctl->end[e] = static_cast<int>(hi);
            tiles_e = static_cast<int>((hi - lo + BM - 1) / BM);
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, tiles_e, o);
            if (lane >= o) tiles_e += v;
        }
        if (lane == 31) ctl->warp_sum[warp] = tiles_e;
    }
    __syncthreads();
    if (threadIdx.x < kMaxE) {
        for (int w = 0; w < warp; ++w) tiles_e += ctl->warp_sum[w];
        ctl->mt[threadIdx.x + 1] = tiles_e;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    const uint32_t tmem_base = ctl->tmem_base;
    const int total = ctl->mt[g.E] * g.n_tiles;
    const int num_kb = (g.K + BK - 1) / BK;

    if (warp < FIRST_SUM_WARP) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(ROLE_REGS));
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------ TMA producer
            int stage = 0;
            uint32_t phase = 0, armed = 0, armed_parity = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                const Tile ti = decode_tile(t, ctl, g.E, g.n_tiles);
                const int row0 = ctl->off[ti.e] + ti.m_tile * BM;
                const int n0 = ti.n_tile * out_cols<EPI>();
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!mbar_wait(&ctl->empty[stage], phase ^ 1u, abort_flag, g.status)) {
                        ok = false;
                        break;
                    }
                    uint8_t *sA = tiles + stage * STAGE_BYTES;
                    uint8_t *sW = sA + A_BYTES;
                    mbar_arrive_expect_tx(&ctl->full[stage], STAGE_BYTES);
                    armed |= 1u << stage;
                    armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
                    tma_load_3d(sA, &tmA, &ctl->full[stage], kb * BK, row0, 0);
                    tma_load_3d(sW, &tmW, &ctl->full[stage], kb * BK, n0, ti.e);
                    if (EPI == EPI_SWIGLU)
                        tma_load_3d(sW + W_BYTES / 2, &tmW3, &ctl->full[stage], kb * BK, n0, ti.e);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (*abort_flag) {
                // let every copy this thread started land before the CTA exits
                for (int s = 0; s < STAGES; ++s)
                    if ((armed >> s) & 1u)
                        mbar_wait(&ctl->full[s], (armed_parity >> s) & 1u, abort_flag, g.status, false);
            }
        } else if (warp == 1 && lane == 0) {
            // -------------------------------------------------- MMA issuer
            constexpr uint32_t idesc = idesc_f8(BM, BN);
            int stage = 0, buf = 0;
            uint32_t phase = 0, tphase = 0;
            bool ok = true, issued = false;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!mbar_wait(&ctl->tempty[buf], tphase ^ 1u, abort_flag, g.status) ||
                        !mbar_wait(&ctl->full[stage], phase, abort_flag, g.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_addr = smem_u32(tiles + stage * STAGE_BYTES), w_addr = a_addr + A_BYTES;
                    const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * BN);
#pragma unroll
                    for (int kk = 0; kk < BK / 32; ++kk)
                        umma_f8(d_tmem, desc_sw128(a_addr + kk * 32), desc_sw128(w_addr + kk * 32), idesc,
                                kk != 0 ? 1u : 0u);
                    issued = true;
                    umma_commit(&ctl->empty[stage]);
                    umma_commit(&ctl->tfull[buf]);
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (++buf == 2) {
                        buf = 0;
                        tphase ^= 1u;
                    }
                }
            }
            if (*abort_flag && issued) {
                // wait for every MMA issued so far before TMEM is freed
                umma_commit(&ctl->drain);
                mbar_wait(&ctl->drain, 0, abort_flag, g.status, false);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SUM_REGS));
        // ---------------------------------------------- sums and epilogue
        const int quarter = warp & 3, half = (warp - FIRST_SUM_WARP) >> 2;
        uint8_t *stage = ctl->stage[warp - FIRST_SUM_WARP];
        const int nblocks = (g.n_out + kFp8Block - 1) / kFp8Block;
        int buf = 0;
        uint32_t tphase = 0, xphase = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
            const Tile ti = decode_tile(t, ctl, g.E, g.n_tiles);
            const int64_t row_first = ctl->off[ti.e] + ti.m_tile * BM + quarter * 32;
            const int64_t row_end = ctl->end[ti.e];
            const int64_t row = row_first + lane;
            const bool active = row_first < row_end;  // of the whole warp
            const int n0 = ti.n_tile * out_cols<EPI>();
            // this thread's columns: SwiGLU half*64 of the gate and of the
            // up projection, else half*128 (one scale block)
            const int nb = min(n0 / kFp8Block + (EPI == EPI_SWIGLU ? 0 : half), nblocks - 1);
            const float *as = g.a_scales + min64(row, g.rows - 1);
            const float *ws = g.w_scales + (static_cast<int64_t>(ti.e) * nblocks + nb) * num_kb;
            const float *ws3 = EPI == EPI_SWIGLU ? g.w3_scales + (static_cast<int64_t>(ti.e) * nblocks + nb) * num_kb : ws;
            uint64_t acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0;
            float sa = __ldg(as), sw = __ldg(ws), sw3 = __ldg(ws3);
            for (int kb = 0; kb < num_kb; ++kb) {
                const float s1 = sa * sw, s3 = sa * sw3;
                const uint64_t p1 = pack2(__float_as_uint(s1), __float_as_uint(s1));
                const uint64_t p3 = pack2(__float_as_uint(s3), __float_as_uint(s3));
                if (kb + 1 < num_kb) {
                    sa = __ldg(as + static_cast<int64_t>(kb + 1) * g.rows);
                    sw = __ldg(ws + kb + 1);
                    if (EPI == EPI_SWIGLU) sw3 = __ldg(ws3 + kb + 1);
                }
                if (!__all_sync(0xffffffffu, mbar_wait(&ctl->tfull[buf], tphase, abort_flag, g.status))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (active) {
                    const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                           static_cast<uint32_t>(buf * BN);
                    // 32 columns at a time, the next ones on their way
                    // while these are added
                    uint32_t r[2][32];
                    tmem_ld32(tbase + chunk_col<EPI>(0, half), r[0]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        tmem_ld_wait(r[c & 1]);
                        if (c < 3) tmem_ld32(tbase + chunk_col<EPI>(c + 1, half), r[(c + 1) & 1]);
                        const uint64_t p = (EPI == EPI_SWIGLU && c >= 2) ? p3 : p1;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            acc[c * 16 + i] = fma2(pack2(r[c & 1][2 * i], r[c & 1][2 * i + 1]), p, acc[c * 16 + i]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->tempty[buf]);
                if (++buf == 2) {
                    buf = 0;
                    tphase ^= 1u;
                }
            }
            if (!ok) break;
            if (!active) continue;

            if constexpr (EPI == EPI_SWIGLU) {
                float h[64];
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float g0, g1, u0, u1;
                    unpack2(acc[i], g0, g1);
                    unpack2(acc[32 + i], u0, u1);
                    h[2 * i] = silu_approx(g0) * u0;
                    h[2 * i + 1] = silu_approx(g1) * u1;
                    m = max(m, max(abs_bits(h[2 * i]), abs_bits(h[2 * i + 1])));
                }
                // The other half of the row's block.  Two sets of values by
                // phase: a warp that is a tile ahead writes the other set,
                // and it cannot be two ahead.
                ctl->amax[xphase][half][quarter * 32 + lane] = m;
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->exchanged[quarter]);
                if (!__all_sync(0xffffffffu, mbar_wait(&ctl->exchanged[quarter], xphase, abort_flag, g.status))) break;
                m = max(m, ctl->amax[xphase][half ^ 1][quarter * 32 + lane]);
                xphase ^= 1u;
                const float2 s = fp8_scale(m);
                if (row < row_end) {
                    store_h64(h, s.y, static_cast<uint8_t *>(g.out) + row * g.n_out, n0 + half * 64, g.n_out);
                    if (half == 0) g.h_scales[static_cast<int64_t>(nb) * g.rows + row] = s.x;
                }
            } else if constexpr (EPI == EPI_GELU) {
                const int c0 = n0 + half * 128;
                if (c0 >= g.n_out) continue;
                const __nv_bfloat16 *bias = g.bias ? g.bias + static_cast<int64_t>(ti.e) * g.n_out : nullptr;
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float b[8];
                    bias8(bias, c0 + 8 * j, g.n_out, b);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float v0, v1;
                        unpack2(acc[j * 4 + i], v0, v1);
                        v0 = gelu_erf(v0 + b[2 * i]);
                        v1 = gelu_erf(v1 + b[2 * i + 1]);
                        m = max(m, max(abs_bits(v0), abs_bits(v1)));
                        acc[j * 4 + i] = pack2(__float_as_uint(v0), __float_as_uint(v1));
                    }
                }
                const float2 s = fp8_scale(m);
                if (row < row_end) {
                    uint8_t *out = static_cast<uint8_t *>(g.out) + row * g.n_out;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float h[64];
#pragma unroll
                        for (int i = 0; i < 32; ++i) unpack2(acc[q * 32 + i], h[2 * i], h[2 * i + 1]);
                        store_h64(h, s.y, out, c0 + q * 64, g.n_out);
                    }
                    g.h_scales[static_cast<int64_t>(nb) * g.rows + row] = s.x;
                }
            } else {
                const __nv_bfloat16 *bias = g.bias ? g.bias + static_cast<int64_t>(ti.e) * g.n_out : nullptr;
                constexpr int ES = EPI == EPI_BF16 ? 2 : 4;
                constexpr int CC = 64 / ES;  // columns of a staged chunk
                uint8_t *out = static_cast<uint8_t *>(g.out);
                const int64_t row_bytes = static_cast<int64_t>(g.n_out) * ES;
#pragma unroll
                for (int c = 0; c < 128 / CC; ++c) {
                    const int col = n0 + half * 128 + c * CC;
                    if (col >= g.n_out) break;
                    float v[CC];
#pragma unroll
                    for (int i = 0; i < CC / 2; ++i) unpack2(acc[c * CC / 2 + i], v[2 * i], v[2 * i + 1]);
                    if (bias) {
#pragma unroll
                        for (int j = 0; j < CC / 8; ++j) {
                            float b[8];
                            bias8(bias, col + 8 * j, g.n_out, b);
#pragma unroll
                            for (int i = 0; i < 8; ++i) v[8 * j + i] += b[i];
                        }
                    }
                    uint4 p[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (EPI == EPI_BF16)
                            p[j] = pack16(v + 8 * j, static_cast<const __nv_bfloat16 *>(nullptr));
                        else
                            p[j] = pack16(v + 4 * j, static_cast<const float *>(nullptr));
                    }
                    store_chunk(p, stage, out, row_bytes, row_first, row_end, col * ES, row_bytes, lane);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

template <int EPI>
cudaError_t launch(const Fp8GemmArgs &a, int num_sms, cudaStream_t s)
{
    CUtensorMap tmA, tmW, tmW3;
    constexpr bool kTwo = EPI == EPI_SWIGLU;
    if (!make_tmap_u8(&tmA, a.a, a.k, a.rows, 1, BM) || !make_tmap_u8(&tmW, a.w, a.k, a.n, a.E, kTwo ? BN / 2 : BN) ||
        !make_tmap_u8(&tmW3, kTwo ? a.w3 : a.w, a.k, a.n, a.E, kTwo ? BN / 2 : BN))
        return cudaErrorInvalidValue;
    auto *kernel = ffn_gemm_fp8_kernel<EPI>;
    cudaError_t err = ensure_smem_attr(reinterpret_cast<const void *>(kernel), static_cast<int>(kSmemBytes));
    if (err != cudaSuccess) return err;
    Args g{};
    g.offsets = a.offsets;
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
    g.n_tiles = (a.n + out_cols<EPI>() - 1) / out_cols<EPI>();
    // every slice may end inside a tile
    const int64_t most = (a.rows / BM + min64(a.E, a.rows)) * g.n_tiles;
    if (most >= (static_cast<int64_t>(1) << 31)) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(min64(most, num_sms)));
    return launch_k(kernel, grid, dim3(THREADS), kSmemBytes, s, tmA, tmW, tmW3, g);
}

}  // namespace

cudaError_t launch_gemm_fp8(const Fp8GemmArgs &a, int num_sms, cudaStream_t s)
{
    if (a.rows == 0) return cudaSuccess;
    switch (a.epi) {
        case kFp8Swiglu: return launch<EPI_SWIGLU>(a, num_sms, s);
        case kFp8Gelu: return launch<EPI_GELU>(a, num_sms, s);
        case kFp8Bf16: return launch<EPI_BF16>(a, num_sms, s);
        default: return launch<EPI_F32>(a, num_sms, s);
    }
}

}  // namespace moe
