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
// It takes any scales; powers of two are faster left to the tensor core
// (gemm_mxfp8_sm100.cu).  What bounds it is the epilogue warps: reading and
// adding a k-block's accumulator takes them longer than the MMA's 512 cycles
// (short runs: Mixtral's FFN, 4096 tokens: 2.2-2.4 ms, and 1.25-1.45 ms with
// powers of two; DeepSeek-V3's 3.7-4.1 and 2.1-2.2 ms).  Few rows: 32 rows of 8
// experts, n = 4096, k = 14336: 91 us and 80; one token of DeepSeek-V3: 93 and 73.
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
#include <cuda_fp16.h>

#include "gemm_fp8.cuh"
#include "host_util.h"

namespace moe {
namespace {

using namespace fp8;

constexpr int BM = 128;          // rows of a CTA's tile
constexpr int BN = 256;          // accumulator columns of a tile
constexpr int STAGES = 4;
constexpr int CHUNK_BYTES = 32 * 64;  // a warp's staging: 32 rows of 64 bytes
constexpr int ROLE_REGS = 56, SUM_REGS = 224;
static_assert(32 * FIRST_SUM_WARP * ROLE_REGS + 32 * SUM_WARPS * SUM_REGS <= THREADS * LAUNCH_REGS, "register split");
constexpr int A_BYTES = BM * BK;
constexpr int W_BYTES = BN * BK;
constexpr int STAGE_BYTES = A_BYTES + W_BYTES;
constexpr uint32_t TMEM_COLS = 512;

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

struct Ctl {
    alignas(1024) uint8_t stage[SUM_WARPS][CHUNK_BYTES];
    Exchange exchange;
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    Slices slices;
};

constexpr size_t kSmemBytes = 1024 + STAGES * STAGE_BYTES + sizeof(Ctl);
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

template <int EPI> __host__ __device__ constexpr int out_cols() { return EPI == EPI_SWIGLU ? 128 : 256; }

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

// First accumulator column of a thread's chunk c of 32: SwiGLU, 64 gate and
// then 64 up columns; else 128 consecutive ones.
template <int EPI> __device__ __forceinline__ uint32_t chunk_col(int c, int half)
{
    return EPI == EPI_SWIGLU ? (c >> 1) * 128 + half * 64 + (c & 1) * 32 : half * 128 + c * 32;
}

__device__ __forceinline__ bool not_normal(float p) { return (__float_as_uint(p) & 0x7FFFFFFFu) - 0x00800000u >= 0x7F000000u; }

// Whether p, the fp32 product of the scales a and b, is too small or too large
// for a block's sums (zero, or 2^-18 to 2^25 in size): subnormal or zero, so
// that bits are lost, or infinite of finite scales, which times zero is no
// number.
__device__ __forceinline__ bool beyond_f32(float p, float a, float b)
{
    const uint32_t m = __float_as_uint(p) & 0x7FFFFFFFu;
    return m < 0x00800000u || (m == 0x7F800000u && fmaxf(fabsf(a), fabsf(b)) < INFINITY);
}

// Nonzero if one of 16 e4m3 values is.
__device__ __forceinline__ uint32_t nonzero16(const uint8_t *p)
{
    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
    return (v.x | v.y | v.z | v.w) & 0x7F7F7F7Fu;
}

// Two e4m3 values, exactly.
__device__ __forceinline__ float2 from_e4m3x2(uint32_t v)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// sum of a[i] w[i] over n (a multiple of 16) e4m3 values.
__device__ __forceinline__ float dot_e4m3(const uint8_t *a, const uint8_t *w, int n)
{
    float sum = 0.0f;
    for (int i = 0; i < n; i += 16) {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(a + i)), y = __ldg(reinterpret_cast<const uint4 *>(w + i));
        const uint32_t p[4] = {x.x, x.y, x.z, x.w}, q[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 u = from_e4m3x2(p[j / 2] >> (16 * (j & 1))), v = from_e4m3x2(q[j / 2] >> (16 * (j & 1)));
            sum = fmaf(u.x, v.x, fmaf(u.y, v.y, sum));
        }
    }
    return sum;
}

template <int EPI>
__global__ void __launch_bounds__(THREADS, 1)
    ffn_gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
                        const __grid_constant__ CUtensorMap tmW3, const GemmArgs g)
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
        for (int q = 0; q < 4; ++q) mbar_init(&ctl->exchange.there[q], 2);
        mbar_init(&ctl->drain, 1);
        ctl->abort = 0;
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
    tc_fence_before();
    load_slices<BM>(&ctl->slices, g);
    tc_fence_after();

    const uint32_t tmem_base = ctl->tmem_base;
    const int total = ctl->slices.mt[g.E] * g.n_tiles;
    const int num_kb = (g.K + BK - 1) / BK;

    if (warp < FIRST_SUM_WARP) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(ROLE_REGS));
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------ TMA producer
            int stage = 0;
            uint32_t phase = 0, armed = 0, armed_parity = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
                const Tile ti = decode_tile(t, &ctl->slices, g.E, g.n_tiles);
                const int row0 = ctl->slices.off[ti.e] + ti.m_tile * BM;
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
            const Tile ti = decode_tile(t, &ctl->slices, g.E, g.n_tiles);
            const int64_t row_first = static_cast<int64_t>(ctl->slices.off[ti.e]) + ti.m_tile * BM + quarter * 32;
            const int64_t row_end = ctl->slices.end[ti.e];
            const int64_t row = row_first + lane;
            const bool active = row_first < row_end;  // of the whole warp
            const int n0 = ti.n_tile * out_cols<EPI>();
            // this thread's columns: SwiGLU half*64 of the gate and of the
            // up projection, else half*128 (one scale block)
            const int nb = min(n0 / kFp8Block + (EPI == EPI_SWIGLU ? 0 : half), nblocks - 1);
            const float *as = g.a_scales + min64(row, g.rows - 1);
            const float *ws = g.w_scales + (static_cast<int64_t>(ti.e) * nblocks + nb) * num_kb;
            const float *ws3 = EPI == EPI_SWIGLU ? g.w3_scales + (static_cast<int64_t>(ti.e) * nblocks + nb) * num_kb : ws;
            float acc[128];
#pragma unroll
            for (int i = 0; i < 128; ++i) acc[i] = 0.0f;
            float sa = __ldg(as), sw = __ldg(ws), sw3 = __ldg(ws3);
            bool left = false;
            for (int kb = 0; kb < num_kb; ++kb) {
                const float a0 = sa, w0 = sw, w30 = sw3;
                if (kb + 1 < num_kb) {
                    sa = __ldg(as + static_cast<int64_t>(kb + 1) * g.rows);
                    sw = __ldg(ws + kb + 1);
                    if (EPI == EPI_SWIGLU) sw3 = __ldg(ws3 + kb + 1);
                }
                if (!__all_sync(0xffffffffu, mbar_wait(&ctl->tfull[buf], tphase, abort_flag, g.status))) {
                    ok = false;
                    break;
                }
                float s1 = a0 * w0, s3 = a0 * w30;
                if (__any_sync(0xffffffffu, not_normal(s1) || (EPI == EPI_SWIGLU && not_normal(s3)))) {
                    // such blocks are added below, after the others
                    const bool b1 = beyond_f32(s1, a0, w0), b3 = EPI == EPI_SWIGLU && beyond_f32(s3, a0, w30);
                    s1 = b1 ? 0.0f : s1;
                    s3 = b3 ? 0.0f : s3;
                    left |= b1 || b3;
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
                        const float p = (EPI == EPI_SWIGLU && c >= 2) ? s3 : s1;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            acc[c * 32 + i] = fmaf(__uint_as_float(r[c & 1][i]), p, acc[c * 32 + i]);
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
            // The blocks whose scales' product fp32 does not hold.  Most often
            // they are zeros under the quantiser's smallest scale, a whole
            // row of them: the warp looks at each such row (one row of eight
            // zero: 10% of a call of 4096 rows, n = 2048, k = 7168).
            bool again = false;
            for (uint32_t rows = __ballot_sync(0xffffffffu, left && row < row_end); rows != 0; rows &= rows - 1) {
                const int r = __ffs(rows) - 1;
                const uint8_t *a = g.a + (row_first + r) * g.K;
                uint32_t any = 0;
#pragma unroll 8
                for (int i = lane * 16; i < g.K; i += 32 * 16) any |= nonzero16(a + i);
                if (__any_sync(0xffffffffu, any != 0) && lane == r) again = true;
            }
            if (again) {  // summed once more, and scaled in 64 bits: right, but slow
                const uint8_t *a = g.a + row * g.K;
                for (int kb = 0; kb < num_kb; ++kb) {
                    const int n = min(BK, g.K - kb * BK);
                    const float sa = __ldg(as + kb * g.rows);
                    const auto beyond = [&](float sw) { return sa != 0.0f && sw != 0.0f && beyond_f32(sa * sw, sa, sw); };
                    if (!beyond(__ldg(ws + kb)) && !(EPI == EPI_SWIGLU && beyond(__ldg(ws3 + kb)))) continue;
                    uint32_t any = 0;
                    for (int i = 0; i < n; i += 16) any |= nonzero16(a + kb * BK + i);
                    for (int j = 0; j < 128 && any != 0; ++j) {
                        const bool up = EPI == EPI_SWIGLU && j >= 64;
                        const float sw = __ldg((up ? ws3 : ws) + kb);
                        const int col = n0 + (EPI == EPI_SWIGLU ? half * 64 + (j & 63) : half * 128 + j);
                        if (!beyond(sw) || col >= g.n_out) continue;
                        const uint8_t *w = (up ? g.w3 : g.w) + (static_cast<int64_t>(ti.e) * g.n_out + col) * g.K;
                        const float v = static_cast<float>(dot_e4m3(a + kb * BK, w + kb * BK, n) * (static_cast<double>(sa) * sw));
#pragma unroll
                        for (int i = 0; i < 128; ++i)
                            if (i == j) acc[i] += v;
                    }
                }
            }

            const __nv_bfloat16 *bias = g.bias ? g.bias + static_cast<int64_t>(ti.e) * g.n_out : nullptr;
            if constexpr (EPI == EPI_SWIGLU) {
                float *h = acc;
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    h[i] = silu_approx(acc[i]) * acc[64 + i];
                    m = max(m, abs_bits(h[i]));
                }
                if (!exchange_amax(&ctl->exchange, m, xphase, quarter, half, lane, abort_flag, g.status)) break;
                xphase ^= 1u;
                const float2 s = fp8_scale(m);
                if (row < row_end) {
                    uint8_t *out = static_cast<uint8_t *>(g.out) + row * g.n_out;
#pragma unroll
                    for (int c = 0; c < 2; ++c) store_h32(h + 32 * c, s.y, out, n0 + half * 64 + 32 * c, g.n_out);
                    if (half == 0) g.h_scales[static_cast<int64_t>(nb) * g.rows + row] = s.x;
                }
            } else if constexpr (EPI == EPI_GELU) {
                const int c0 = n0 + half * 128;
                if (c0 >= g.n_out) continue;
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float b[8];
                    bias8(bias, c0 + 8 * j, g.n_out, b);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        acc[8 * j + i] = gelu_erf(acc[8 * j + i] + b[i]);
                        m = max(m, abs_bits(acc[8 * j + i]));
                    }
                }
                const float2 s = fp8_scale(m);
                if (row < row_end) {
                    uint8_t *out = static_cast<uint8_t *>(g.out) + row * g.n_out;
#pragma unroll
                    for (int c = 0; c < 4; ++c) store_h32(acc + 32 * c, s.y, out, c0 + 32 * c, g.n_out);
                    g.h_scales[static_cast<int64_t>(nb) * g.rows + row] = s.x;
                }
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int col = n0 + half * 128 + c * 32;
                    if (col >= g.n_out) break;
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = acc[c * 32 + i];
                    store_columns<EPI>(v, bias, g, col, row_first, row_end, stage, lane);
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
    const GemmArgs g = gemm_args(a, out_cols<EPI>());
    // every slice may end inside a tile
    const int64_t most = (a.rows / BM + min64(a.E, a.rows)) * g.n_tiles;
    if (most > (static_cast<int64_t>(1) << 30)) return cudaErrorInvalidValue;  // tile numbers and a step
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
