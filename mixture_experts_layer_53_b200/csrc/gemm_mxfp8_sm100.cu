// gemm_mxfp8_sm100.cu -- ragged grouped GEMM on e4m3 operands whose block
// scales are powers of two (tcgen05 kind::mxf8f6f4: the tensor core applies
// the scales, one 8-bit exponent per row and 32 values of the reduction).
//
// For row r of expert e (rows offsets[e] .. offsets[e+1]-1):
//   y[r, c] = sum_kb sA[kb, r] sW[e, c / 128, kb] sum_{k in kb} a[r, k] w[e, c, k]
// A power of two is its exponent, and a fp32 scale's exponent field is the
// hardware's UE8M0 code (255 for NaN), so the fp32 scale tensors are read as
// they are.  The whole reduction accumulates in TMEM in fp32; nothing is
// added on the CUDA cores (gemm_fp8_sm100.cu, for other scales, does that and
// spends more time on it than the tensor core on the products).
//
// Tiles are 128 rows x 256 columns on one CTA, or 256 x 256 on a CTA pair
// (cta_group::2), in which a weight tile crosses L2 -> SM once per pair; the
// pair is taken when experts average more than 192 rows, as in the bf16 FFN,
// since with fewer rows its second half would mostly compute rows of the next
// expert.  Tile list (expert, n-tile, m-tile), m-tiles innermost: CTAs that
// run at the same time share an expert's weight tile through L2.
//
// Warp roles (384 threads, one CTA per SM, persistent):
//   warp 0      TMA producer: per k-block of 128 values A (16 KB) and W
//               (32 KB; 16 KB per CTA of a pair), 192 KB of stages
//   warp 1      allocates TMEM; one lane issues the MMAs (K = 32), four
//               to a k-block
//   warps 2, 3  scales: pack four k-blocks' exponents into a word per row,
//               in the [row % 32][row / 32] order that tcgen05.cp spreads
//               over the TMEM lanes; alternate groups of four k-blocks,
//               the next group's scales on their way while one is packed
//   warps 4-11  epilogue: a warp owns 32 rows (its TMEM lane quarter) and
//               half of the columns
//
// TMEM: 512 columns hold two accumulators of 256 and, for two groups of
// k-blocks, 4 columns of A's and 8 of W's scales.  The accumulators overlap
// by those 24 columns (0-255 and 232-487): the epilogue reads the shared
// columns first and signals them free, and the next tile's MMAs start then.
//
// SwiGLU: accumulator columns 0-127 are the gate and 128-255 the up
// projection of the same 128 hidden units, one scale block of h: the
// epilogue quantises them on the spot.  GELU: two scale blocks per tile.
#include "gemm_fp8.cuh"
#include "host_util.h"

namespace moe {
namespace {

using namespace fp8;

// The epilogue holds a thread's 128 accumulator values, more than the 168
// registers that 384 threads launch with have room for beside the rest: the
// first warpgroup hands registers over (128 x 88 + 256 x 208 = 384 x 168).
constexpr int ROLE_REGS = 88, SUM_REGS = 208;
static_assert(32 * FIRST_SUM_WARP * ROLE_REGS + 32 * SUM_WARPS * SUM_REGS <= THREADS * LAUNCH_REGS, "register split");
constexpr int GROUP = 4;                     // k-blocks of one scale word
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t ACC_STEP = 232;           // second accumulator's first column
constexpr uint32_t SCALE_COL = 488;          // + 12 per group slot: 4 of A, 8 of W
constexpr int SCALE_BYTES = 3 * 512;         // A's 128 rows, W's 256
constexpr int SLOTS = 4;                     // groups of scales in shared memory
constexpr int A_BYTES = BM * BK;

template <bool PAIR> constexpr int w_bytes() { return (PAIR ? BN / 2 : BN) * BK; }
template <bool PAIR> constexpr int stage_bytes() { return A_BYTES + w_bytes<PAIR>(); }
template <bool PAIR> constexpr int stages() { return PAIR ? 6 : 4; }

template <bool PAIR> struct Ctl {
    alignas(1024) uint8_t stage[SUM_WARPS][CHUNK_BYTES];
    alignas(128) uint8_t scales[SLOTS][SCALE_BYTES];
    Exchange exchange;
    // a pair's barriers: full, sfull, tempty and shared_free are the even
    // CTA's (both CTAs' arrivals); empty, sempty, tfull are signalled in both
    uint64_t full[stages<PAIR>()];
    uint64_t empty[stages<PAIR>()];
    uint64_t sfull[SLOTS];
    uint64_t sempty[SLOTS];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t shared_free;
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    Slices slices;
};

template <bool PAIR> constexpr size_t smem_bytes() { return 1024 + stages<PAIR>() * stage_bytes<PAIR>() + sizeof(Ctl<PAIR>); }
static_assert(smem_bytes<false>() <= 232448 && smem_bytes<true>() <= 232448, "shared memory per CTA");

// Instruction descriptor of kind::mxf8f6f4: A and B e4m3 (0) and K-major, N >> 3
// at [17,23), UE8M0 scales (bit 23), M >> 4 at [24,29); the byte of the scale
// words that the MMA uses at [4,6) for B and [29,31) for A.
constexpr uint32_t idesc_mxf8(int M, int N, int byte)
{
    return (static_cast<uint32_t>(byte) << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
           (static_cast<uint32_t>(M >> 4) << 24) | (static_cast<uint32_t>(byte) << 29);
}

// D (+)= (A scaled) * (B scaled)^T; a pair's is issued by the even CTA.
template <bool PAIR>
__device__ __forceinline__ void umma_mxf8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                          uint32_t accumulate)
{
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
}

// 32 rows of 16 bytes from shared memory to four TMEM columns, repeated in
// every lane quarter (in both CTAs of a pair, each from its own memory).
template <bool PAIR> __device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc)
{
    if constexpr (PAIR)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Matrix descriptor of 32 unswizzled rows of 16 bytes (8-row groups 128
// bytes apart); fields as in desc_sw128.
__device__ __forceinline__ uint64_t desc_scales(uint32_t smem_addr)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(1) << 16;
    d |= static_cast<uint64_t>(128 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    return d;
}

// A load that stays where it is written: ahead of its use by a group.
__device__ __forceinline__ float load_ahead(const float *p)
{
    float v;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

template <bool PAIR> __device__ __forceinline__ void commit(uint64_t *bar)
{
    if constexpr (PAIR) umma_commit_pair(bar, 0x3);
    else umma_commit(bar);
}

template <int EPI, bool PAIR>
__device__ __forceinline__ void
    mxfp8_gemm(const CUtensorMap &tmA, const CUtensorMap &tmW, const CUtensorMap &tmW3, const GemmArgs &g)
{
    pdl_enter();
    extern __shared__ uint8_t smem_raw[];
    constexpr int CTAS = PAIR ? 2 : 1, TILE_M = BM * CTAS, NST = stages<PAIR>(), STAGE = stage_bytes<PAIR>();
    uint8_t *tiles = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                 ~static_cast<uintptr_t>(1023));
    Ctl<PAIR> *ctl = reinterpret_cast<Ctl<PAIR> *>(tiles + NST * STAGE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0;
    const bool leader = rank == 0;
    volatile int *abort_flag = &ctl->abort;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ctl->tfull[b], 1);
            mbar_init(&ctl->tempty[b], SUM_WARPS * CTAS);
        }
        for (int s = 0; s < SLOTS; ++s) {
            mbar_init(&ctl->sfull[s], CTAS);
            mbar_init(&ctl->sempty[s], 1);
        }
        for (int q = 0; q < 4; ++q) mbar_init(&ctl->exchange.there[q], 2);
        mbar_init(&ctl->shared_free, SUM_WARPS * CTAS);
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
        if constexpr (PAIR) {
            tmem_alloc_pair(&ctl->tmem_base, TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(&ctl->tmem_base, TMEM_COLS);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    load_slices<TILE_M>(&ctl->slices, g);
    // barriers of both CTAs are initialised before either signals the other
    if constexpr (PAIR) cluster_sync();
    tc_fence_after();

    const Slices *sl = &ctl->slices;
    const uint32_t tmem_base = ctl->tmem_base;
    const int total = sl->mt[g.E] * g.n_tiles;
    const int num_kb = (g.K + BK - 1) / BK;
    const int first = PAIR ? blockIdx.x >> 1 : blockIdx.x, step = PAIR ? gridDim.x >> 1 : gridDim.x;
    constexpr int TILE_N = out_cols<EPI>();

    if (warp < FIRST_SUM_WARP) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(ROLE_REGS));
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------ TMA producer
            int stage = 0;
            uint32_t phase = 0, armed = 0, armed_parity = 0;
            bool ok = true;
            for (int t = first; t < total && ok; t += step) {
                const Tile ti = decode_tile(t, sl, g.E, g.n_tiles);
                const int row0 = sl->off[ti.e] + ti.m_tile * TILE_M + static_cast<int>(rank) * BM;
                // a pair's W halves: SwiGLU W1 and W3, else the tile's columns
                const int n0 = ti.n_tile * TILE_N + (PAIR && EPI != EPI_SWIGLU ? static_cast<int>(rank) * (BN / 2) : 0);
                const CUtensorMap *tw = PAIR && EPI == EPI_SWIGLU && rank ? &tmW3 : &tmW;
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!mbar_wait(&ctl->empty[stage], phase ^ 1u, abort_flag, g.status)) {
                        ok = false;
                        break;
                    }
                    uint8_t *sA = tiles + stage * STAGE, *sW = sA + A_BYTES;
                    if (leader) {
                        mbar_arrive_expect_tx(&ctl->full[stage], CTAS * STAGE);
                        armed |= 1u << stage;
                        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
                    }
                    if constexpr (PAIR) {
                        const uint32_t full = mapa_shared(smem_u32(&ctl->full[stage]), 0);
                        tma_load_3d_pair(sA, &tmA, full, kb * BK, row0, 0);
                        tma_load_3d_pair(sW, tw, full, kb * BK, n0, ti.e);
                    } else {
                        tma_load_3d(sA, &tmA, &ctl->full[stage], kb * BK, row0, 0);
                        tma_load_3d(sW, &tmW, &ctl->full[stage], kb * BK, n0, ti.e);
                        if (EPI == EPI_SWIGLU)
                            tma_load_3d(sW + w_bytes<PAIR>() / 2, &tmW3, &ctl->full[stage], kb * BK, n0, ti.e);
                    }
                    if (++stage == NST) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (*abort_flag && leader) {
                // let every copy that lands on these barriers land before
                // the CTA exits
                for (int s = 0; s < NST; ++s)
                    if ((armed >> s) & 1u)
                        mbar_wait(&ctl->full[s], (armed_parity >> s) & 1u, abort_flag, g.status, false);
            }
        } else if (warp == 1 && lane == 0 && leader) {
            // -------------------------------------------------- MMA issuer
            int stage = 0, buf = 0;
            uint32_t phase = 0, tphase = 0, shared_phase = 1, group = 0;
            bool ok = true, issued = false;
            for (int t = first; t < total && ok; t += step) {
                // this accumulator's last tile has been read, and of the
                // other's the columns that both share
                if (!mbar_wait(&ctl->tempty[buf], tphase ^ 1u, abort_flag, g.status) ||
                    !mbar_wait(&ctl->shared_free, shared_phase, abort_flag, g.status))
                    break;
                shared_phase ^= 1u;
                tc_fence_after();
                const uint32_t d = tmem_base + (buf ? ACC_STEP : 0u);
                for (int kb0 = 0; kb0 < num_kb && ok; kb0 += GROUP) {
                    // The group's scales are there, and the MMAs of the
                    // group before the last, which read the same TMEM
                    // columns, are done.
                    const uint32_t slot = group % SLOTS, last = (group - 2) % SLOTS;
                    if (!mbar_wait<PAIR>(&ctl->sfull[slot], group / SLOTS & 1u, abort_flag, g.status) ||
                        (group >= 2 &&
                         !mbar_wait(&ctl->sempty[last], (group - 2) / SLOTS & 1u, abort_flag, g.status))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = tmem_base + SCALE_COL + (group & 1u) * 12u, sb = sa + 4u;
                    const uint32_t src = smem_u32(ctl->scales[slot]);
                    copy_scales<PAIR>(sa, desc_scales(src));
                    copy_scales<PAIR>(sb, desc_scales(src + 512));
                    copy_scales<PAIR>(sb + 4u, desc_scales(src + 1024));
                    issued = true;
                    const int kbs = min(GROUP, num_kb - kb0);
                    for (int j = 0; j < kbs; ++j) {
                        if (!mbar_wait(&ctl->full[stage], phase, abort_flag, g.status)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t a_addr = smem_u32(tiles + stage * STAGE), w_addr = a_addr + A_BYTES;
                        const uint32_t idesc = idesc_mxf8(TILE_M, BN, 0) | static_cast<uint32_t>(j) << 4 |
                                               static_cast<uint32_t>(j) << 29;
#pragma unroll
                        for (int kk = 0; kk < BK / 32; ++kk)
                            umma_mxf8<PAIR>(d, desc_sw128(a_addr + kk * 32), desc_sw128(w_addr + kk * 32), idesc, sa, sb,
                                            (kb0 | j | kk) != 0 ? 1u : 0u);
                        commit<PAIR>(&ctl->empty[stage]);
                        if (++stage == NST) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (!ok) break;
                    commit<PAIR>(&ctl->sempty[slot]);
                    ++group;
                }
                if (!ok) break;
                commit<PAIR>(&ctl->tfull[buf]);
                buf ^= 1;
                if (buf == 0) tphase ^= 1u;
            }
            if (*abort_flag && issued) {
                // wait for every MMA issued so far before TMEM is freed
                if constexpr (PAIR) umma_commit_pair(&ctl->drain, 0x1);
                else umma_commit(&ctl->drain);
                mbar_wait(&ctl->drain, 0, abort_flag, g.status, false);
            }
        } else if (warp >= 2) {
            // ------------------------------------------------------ scales
            const int nblocks = (g.n_out + kFp8Block - 1) / kFp8Block;
            const int groups = (num_kb + GROUP - 1) / GROUP;
            bool odd_scale = false;
            // a group of k-blocks and its values on their way from memory
            struct Fetch {
                int t, gi;        // tile, group of the tile
                float a[4][GROUP];  // rows lane, lane + 32, ... of four k-blocks
                float w;          // lanes 0-3, 4-7: the two 128-column halves of W
                uint32_t rows;    // bit i: row i of this lane is in the slice
            };
            Tile ti{};
            int decoded = -1;
            auto fetch = [&](Fetch &f) {
                if (f.t >= total) return;
                if (decoded != f.t) ti = decode_tile(f.t, sl, g.E, g.n_tiles);
                decoded = f.t;
                const int kb0 = f.gi * GROUP;
                const int64_t row0 = sl->off[ti.e] + static_cast<int64_t>(ti.m_tile) * TILE_M + rank * BM + lane;
                f.rows = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t row = row0 + 32 * i;
                    f.rows |= (row < sl->end[ti.e] ? 1u : 0u) << i;
                    const float *p = g.a_scales + min64(row, g.rows - 1) + static_cast<int64_t>(kb0) * g.rows;
#pragma unroll
                    for (int j = 0; j < GROUP; ++j)
                        f.a[i][j] = kb0 + j < num_kb ? load_ahead(p + static_cast<int64_t>(j) * g.rows) : 1.0f;
                }
                const int j = kb0 + (lane & 3), h = lane >> 2 & 1;
                const int nb = EPI == EPI_SWIGLU ? ti.n_tile : min(ti.n_tile * 2 + h, nblocks - 1);
                const float *p = (EPI == EPI_SWIGLU && h ? g.w3_scales : g.w_scales) +
                                 (static_cast<int64_t>(ti.e) * nblocks + nb) * num_kb;
                f.w = j < num_kb ? load_ahead(p + j) : 1.0f;
            };
            // exponent codes; a scale that is no power of two (zero,
            // negative, any mantissa) is reported
            auto code = [&](float v, bool counts) {
                const uint32_t b = __float_as_uint(v), e = b >> 23;
                odd_scale |= counts && (e == 0 || e > 255 || (e < 255 && (b & 0x7FFFFFu) != 0));
                return e & 255u;
            };
            auto next = [&](Fetch &f) {  // two groups on: the warps alternate
                f.gi += 2;
                while (f.gi >= groups) {
                    f.gi -= groups;
                    f.t += step;
                }
            };
            Fetch now, then;
            now.t = first;
            now.gi = warp - 4;
            next(now);
            fetch(now);
            for (uint32_t group = warp - 2; now.t < total; group += 2) {
                then.t = now.t;
                then.gi = now.gi;
                next(then);
                fetch(then);
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[i] = 0;
#pragma unroll
                    for (int j = 0; j < GROUP; ++j) w[i] |= code(now.a[i][j], now.rows >> i & 1u) << (8 * j);
                }
                uint32_t e = code(now.w, true) << (8 * (lane & 3));
                e |= __shfl_xor_sync(0xffffffffu, e, 1);
                e |= __shfl_xor_sync(0xffffffffu, e, 2);
                const uint32_t w0 = __shfl_sync(0xffffffffu, e, 0), w1 = __shfl_sync(0xffffffffu, e, 4);
                const uint32_t slot = group % SLOTS;
                if (!__all_sync(0xffffffffu,
                                mbar_wait(&ctl->sempty[slot], (group / SLOTS & 1u) ^ 1u, abort_flag, g.status)))
                    break;
                uint8_t *dst = ctl->scales[slot] + lane * 16;
                st16(dst, make_uint4(w[0], w[1], w[2], w[3]));
                st16(dst + 512, make_uint4(w0, w0, w0, w0));
                st16(dst + 1024, make_uint4(w1, w1, w1, w1));
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR) mbar_arrive_cluster(mapa_shared(smem_u32(&ctl->sfull[slot]), 0));
                    else mbar_arrive(&ctl->sfull[slot]);
                }
                now = then;
            }
            if (odd_scale) set_status(g.status, kDevBadArgument);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SUM_REGS));
        // ---------------------------------------------------- epilogue
        const int quarter = warp & 3, half = (warp - FIRST_SUM_WARP) >> 2;
        uint8_t *stage = ctl->stage[warp - FIRST_SUM_WARP];
        const int nblocks = (g.n_out + kFp8Block - 1) / kFp8Block;
        auto signal = [&](uint64_t *bar) {  // this warp's loads from TMEM have completed
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR) mbar_arrive_cluster_cta(mapa_shared(smem_u32(bar), 0));
                else mbar_arrive(bar);
            }
        };
        int buf = 0;
        uint32_t tphase = 0, xphase = 0;
        for (int t = first; t < total; t += step) {
            const Tile ti = decode_tile(t, sl, g.E, g.n_tiles);
            const int64_t row_first = sl->off[ti.e] + static_cast<int64_t>(ti.m_tile) * TILE_M + rank * BM + quarter * 32;
            const int64_t row_end = sl->end[ti.e], row = row_first + lane;
            const bool active = row_first < row_end;  // of the whole warp
            const int n0 = ti.n_tile * TILE_N;
            if (!__all_sync(0xffffffffu, mbar_wait(&ctl->tfull[buf], tphase, abort_flag, g.status))) break;
            tc_fence_after();
            const uint32_t tbase =
                tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + (buf ? ACC_STEP : 0u);
            // Chunks of 32 columns, the ones that the next tile's
            // accumulator shares (the first 24 columns or the last) in the
            // first step: the upper half goes downwards.  v: SwiGLU gate and
            // up of two chunks, else four chunks, in the order read.
            uint32_t v[4][32];
            auto chunk = [&](int c, int of) { return half ? of - 1 - c : c; };
            if (active) {
                if constexpr (EPI == EPI_SWIGLU) {
                    tmem_ld32(tbase + half * 64 + chunk(0, 2) * 32, v[0]);
                    tmem_ld32(tbase + 128 + half * 64 + chunk(0, 2) * 32, v[1]);
                    tmem_ld_wait(v[0]);
                    tmem_ld_wait(v[1]);
                } else {
                    tmem_ld32(tbase + half * 128 + chunk(0, 4) * 32, v[0]);
                    tmem_ld_wait(v[0]);
                }
            }
            signal(&ctl->shared_free);
            if (active) {
                if constexpr (EPI == EPI_SWIGLU) {
                    tmem_ld32(tbase + half * 64 + chunk(1, 2) * 32, v[2]);
                    tmem_ld32(tbase + 128 + half * 64 + chunk(1, 2) * 32, v[3]);
                    tmem_ld_wait(v[2]);
                    tmem_ld_wait(v[3]);
                } else {
                    tmem_ld32(tbase + half * 128 + chunk(1, 4) * 32, v[1]);
                    tmem_ld32(tbase + half * 128 + chunk(2, 4) * 32, v[2]);
                    tmem_ld32(tbase + half * 128 + chunk(3, 4) * 32, v[3]);
                    tmem_ld_wait(v[1]);
                    tmem_ld_wait(v[2]);
                    tmem_ld_wait(v[3]);
                }
            }
            signal(&ctl->tempty[buf]);
            buf ^= 1;
            if (buf == 0) tphase ^= 1u;
            if (!active) continue;

            const __nv_bfloat16 *bias = g.bias ? g.bias + static_cast<int64_t>(ti.e) * g.n_out : nullptr;
            if constexpr (EPI == EPI_SWIGLU) {
                float h[64];
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    h[i] = silu_approx(__uint_as_float(v[i / 32 * 2][i % 32])) * __uint_as_float(v[i / 32 * 2 + 1][i % 32]);
                    m = max(m, abs_bits(h[i]));
                }
                if (!exchange_amax(&ctl->exchange, m, xphase, quarter, half, lane, abort_flag, g.status)) break;
                xphase ^= 1u;
                const float2 s = fp8_scale(m);
                if (row < row_end) {
                    uint8_t *out = static_cast<uint8_t *>(g.out) + row * g.n_out;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        store_h32(h + 32 * c, s.y, out, n0 + half * 64 + chunk(c, 2) * 32, g.n_out);
                    if (half == 0) g.h_scales[static_cast<int64_t>(ti.n_tile) * g.rows + row] = s.x;
                }
            } else if constexpr (EPI == EPI_GELU) {
                const int c0 = n0 + half * 128;
                if (c0 >= g.n_out) continue;
                uint32_t m = 0;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float b[8];
                        bias8(bias, c0 + chunk(c, 4) * 32 + 8 * j, g.n_out, b);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float h = gelu_erf(__uint_as_float(v[c][8 * j + i]) + b[i]);
                            v[c][8 * j + i] = __float_as_uint(h);
                            m = max(m, abs_bits(h));
                        }
                    }
                }
                const float2 s = fp8_scale(m);
                if (row < row_end) {
                    uint8_t *out = static_cast<uint8_t *>(g.out) + row * g.n_out;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float h[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) h[i] = __uint_as_float(v[c][i]);
                        store_h32(h, s.y, out, c0 + chunk(c, 4) * 32, g.n_out);
                    }
                    g.h_scales[static_cast<int64_t>(min(ti.n_tile * 2 + half, nblocks - 1)) * g.rows + row] = s.x;
                }
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int col = n0 + half * 128 + chunk(c, 4) * 32;
                    if (col >= g.n_out) continue;
                    float f[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[c][i]);
                    store_columns<EPI>(f, bias, g, col, row_first, row_end, stage, lane);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    // neither CTA frees TMEM or leaves while its partner may still use it
    if constexpr (PAIR) cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        if constexpr (PAIR) tmem_dealloc_pair(tmem_base, TMEM_COLS);
        else tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

template <int EPI>
__global__ void __launch_bounds__(THREADS, 1)
    ffn_gemm_mxfp8_single_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
                                 const __grid_constant__ CUtensorMap tmW3, const GemmArgs g)
{
    mxfp8_gemm<EPI, false>(tmA, tmW, tmW3, g);
}

template <int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    ffn_gemm_mxfp8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
                               const __grid_constant__ CUtensorMap tmW3, const GemmArgs g)
{
    mxfp8_gemm<EPI, true>(tmA, tmW, tmW3, g);
}

template <int EPI, bool PAIR> cudaError_t launch(const Fp8GemmArgs &a, int num_sms, cudaStream_t s)
{
    CUtensorMap tmA, tmW, tmW3;
    constexpr bool kTwo = EPI == EPI_SWIGLU;
    constexpr uint32_t w_rows = PAIR || kTwo ? BN / 2 : BN;
    if (!make_tmap_u8(&tmA, a.a, a.k, a.rows, 1, BM) || !make_tmap_u8(&tmW, a.w, a.k, a.n, a.E, w_rows) ||
        !make_tmap_u8(&tmW3, kTwo ? a.w3 : a.w, a.k, a.n, a.E, w_rows))
        return cudaErrorInvalidValue;
    auto *kernel = PAIR ? ffn_gemm_mxfp8_pair_kernel<EPI> : ffn_gemm_mxfp8_single_kernel<EPI>;
    cudaError_t err = ensure_smem_attr(reinterpret_cast<const void *>(kernel), static_cast<int>(smem_bytes<PAIR>()));
    if (err != cudaSuccess) return err;
    const GemmArgs g = gemm_args(a, out_cols<EPI>());
    // every slice may end inside a tile
    constexpr int CTAS = PAIR ? 2 : 1;
    const int64_t most = (a.rows / (BM * CTAS) + min64(a.E, a.rows)) * g.n_tiles;
    if (most >= (static_cast<int64_t>(1) << 31)) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(min64(most, num_sms / CTAS) * CTAS));
    return launch_k(kernel, grid, dim3(THREADS), smem_bytes<PAIR>(), s, tmA, tmW, tmW3, g);
}

template <int EPI> cudaError_t by_rows(const Fp8GemmArgs &a, int num_sms, cudaStream_t s)
{
    return a.rows > 192 * static_cast<int64_t>(a.E) ? launch<EPI, true>(a, num_sms, s) : launch<EPI, false>(a, num_sms, s);
}

}  // namespace

cudaError_t launch_gemm_mxfp8(const Fp8GemmArgs &a, int num_sms, cudaStream_t s)
{
    if (a.rows == 0) return cudaSuccess;
    switch (a.epi) {
        case kFp8Swiglu: return by_rows<EPI_SWIGLU>(a, num_sms, s);
        case kFp8Gelu: return by_rows<EPI_GELU>(a, num_sms, s);
        case kFp8Bf16: return by_rows<EPI_BF16>(a, num_sms, s);
        default: return by_rows<EPI_F32>(a, num_sms, s);
    }
}

}  // namespace moe
