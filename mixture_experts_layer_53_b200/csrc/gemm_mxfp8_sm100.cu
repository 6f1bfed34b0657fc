// gemm_mxfp8_sm100.cu -- ragged grouped GEMM on e4m3 operands whose block
// scales are powers of two (tcgen05 kind::mxf8f6f4: the tensor core applies
// the scales, one 8-bit exponent per row and 32 values of the reduction).
//
// For row r of expert e (rows offsets[e] .. offsets[e+1]-1):
//   y[r, c] = sum_kb sA[kb, r] sW[e, c / 128, kb] sum_{k in kb} a[r, k] w[e, c, k]
// A power of two is its exponent, and a fp32 scale's exponent field is the
// hardware's UE8M0 code (255, NaN, for what is no such power), so the fp32
// scale tensors are read as they are.  The whole reduction accumulates in TMEM in fp32; nothing is
// added on the CUDA cores (gemm_fp8_sm100.cu, for other scales, does that and
// spends more time on it than the tensor core on the products).
//
// The weights are the MMA's M operand and the rows its N operand: a tile is
// 128 weight rows for each of its accumulators by up to NMAX of the expert's
// rows, and the MMA's N is the rows that the tile really has, rounded up to
// 16.  So a ragged slice costs what its rows cost (with the rows as M, a
// slice of 129 rows cost as much as one of 256), a slice of up to NMAX rows
// reads its weights once, and a result row's columns lie on the lanes of a
// warp: 32 consecutive columns a store, no detour through shared memory.
// Tile list (expert, weight tile, row tile), row tiles innermost: CTAs that
// run at the same time share an expert's weight tile through L2.
//
// Where arithmetic bounds it, it is shared memory that does: an MMA of N rows
// takes N / 2 cycles and reads 4 KB of weights and 32 N bytes of rows, and
// the next k-blocks are written meanwhile.  The shapes share 512 TMEM columns
// and 186 KB of stages:
//   Wide      two accumulators of 240 rows: fewest bytes from L2 and shared
//             memory per product.  The next tile's MMAs wait until its
//             epilogue has read it.
//   Tall      one accumulator of 240 rows, twice: the epilogue overlaps, and
//             there are twice as many tiles.
//   Few       two of 112 rows, twice, for slices of few rows: bound by reading
//             weights, with four stages instead of three.
//   Tiny, TinyTall  two or one of 32 rows, with five or nine stages.  With
//             tiles for a part of the SMs only, a cluster of two to eight
//             CTAs shares a tile's k-blocks; their accumulators are added
//             in rank order through distributed shared memory.
//
// Measured (events, short runs; 6.55 TB/s is this card's copy rate): 8 experts
// x 1024 rows, n = 8192, k = 4096: 234 us, 2.34 PFLOP/s (under the power cap,
// looped: 2.1); 512 tokens of DeepSeek-V3's FFN: 1.69 ms, 6.7 TB/s; 32 rows, n =
// 4096, k = 14336: 75 us, 6.2 TB/s; 131072 rows, n = 2048, k = 768, fp32: 303 us
// (370 in a loop).
//
// Warp roles (384 threads, one CTA per SM, persistent):
//   warp 0      TMA producer: per k-block of 128 values W (16 KB for each
//               accumulator) and the tile's rows, in boxes of 128, 64, 32 and 16
//   warp 1      allocates TMEM; one lane issues the MMAs (K = 32), four to a
//               k-block and accumulator
//   warps 2, 3  scales of 128 rows each (and the weights'): pack four
//               k-blocks' exponents into a word per row, in the [row % 32]
//               [row / 32] order that tcgen05.cp spreads over the TMEM lanes;
//               the next group's scales are on their way meanwhile
//   warps 4-11  epilogue: a warp owns 32 weight rows (its TMEM lane quarter)
//               of one of two accumulators, or every other 32 rows: of the
//               one, or with SwiGLU of both (gate and up of the same 128
//               hidden units)
//
// SwiGLU and GELU: the 128 hidden units of an accumulator are one scale block
// of h; the largest |h| of a row is reduced over the lanes and, through
// shared memory, over the four quarters, and h is quantised on the spot.
#include "gemm_fp8.cuh"
#include "host_util.h"

namespace moe {
namespace {

using namespace fp8;

// The epilogue holds up to 128 values of a thread and two chunks of 32 on
// their way from TMEM, more than the 168 registers that 384 threads launch
// with: the first warpgroup hands registers over (128 x 88 + 256 x 208 =
// 384 x 168).
constexpr int ROLE_REGS = 88, SUM_REGS = 208;
static_assert(32 * FIRST_SUM_WARP * ROLE_REGS + 32 * SUM_WARPS * SUM_REGS <= THREADS * LAUNCH_REGS, "register split");
constexpr int WM = 128;                      // weight rows of an accumulator
constexpr int GROUP = 4;                     // k-blocks of one scale word
constexpr int SLOTS = 4;                     // groups of scales in shared memory
constexpr int AHEAD = 4;                     // groups whose fp32 scales are on their way
constexpr int SCALE_BYTES = 4 * 512;         // W's two accumulators, rows 0-127 and 128-255
constexpr uint32_t TMEM_COLS = 512;

// A tile: accumulators of WM weight rows, their most rows, sets of them.
template <int ACC_, int NMAX_, int BUFS_> struct Shape {
    static constexpr int ACC = ACC_, NMAX = NMAX_, BUFS = BUFS_;
    static constexpr int ATOMS = NMAX > 128 ? 2 : 1;  // 128-row scale tiles of the rows
    static constexpr int W_BYTES = ACC * WM * BK;
    static constexpr int STAGE = W_BYTES + NMAX * BK;
    static constexpr int STAGES = 186 * 1024 / STAGE;
    static constexpr uint32_t SCALE_COL = ACC * BUFS * NMAX;
    static constexpr uint32_t SLOT_COLS = 4 * ACC + 4 * ATOMS;  // of the weights, of the rows; two slots
    static_assert(SCALE_COL + 2 * SLOT_COLS <= TMEM_COLS, "TMEM columns");
    static_assert(STAGE % 1024 == 0, "swizzled tiles start on 1024 bytes");
    static_assert(NMAX % 16 == 0, "the MMA's N");
};
using Wide = Shape<2, 240, 1>;
using Tall = Shape<1, 240, 2>;
using Few = Shape<2, 112, 2>;
using Tiny = Shape<2, 32, 2>;
using TinyTall = Shape<1, 32, 2>;
// Average rows of a slice up to which Tiny and Few are taken; slices of a
// random routing spread around the average.  n = 4096, k = 14336, 4 rows:
// 75.4 us Tiny, 77.2 Few; n = k = 4096, 32 rows: 46 Tiny, 28 Few; n = 8192, k =
// 4096 and 64 rows: 58 Few, 63 Wide, 112 rows: 79 Few, 65 Wide (8 slices).
constexpr int kTinyRows = 16, kFewRows = 80;

struct RowMaps {
    CUtensorMap box[4];  // 128, 64, 32, 16 rows
};

template <typename S> struct Ctl {
    alignas(128) uint8_t scales[SLOTS][SCALE_BYTES];
    // fp32 scales on their way: per scale warp and group, 17 values a lane
    // (written and read by the same lane)
    float ahead[S::ATOMS][AHEAD][4 * GROUP + 1][32];
    uint32_t amax[2][2][4][128];  // [phase][half][lane quarter][the half's rows]
    uint64_t full[S::STAGES];
    uint64_t empty[S::STAGES];
    uint64_t sfull[SLOTS];
    uint64_t sempty[SLOTS];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t there[2];            // per half: the four quarters' amax are there
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    Slices slices;
};

template <typename S> constexpr size_t smem_bytes() { return 1024 + S::STAGES * S::STAGE + sizeof(Ctl<S>); }
static_assert(smem_bytes<Wide>() <= 232448 && smem_bytes<Tall>() <= 232448 && smem_bytes<Few>() <= 232448 &&
                  smem_bytes<Tiny>() <= 232448 && smem_bytes<TinyTall>() <= 232448,
              "shared memory per CTA");

// Instruction descriptor of kind::mxf8f6f4: A and B e4m3 (0) and K-major, N >> 3
// at [17,23), UE8M0 scales (bit 23), M >> 4 at [24,29); the byte of the scale
// words that the MMA uses at [4,6) for B and [29,31) for A.
__device__ __forceinline__ uint32_t idesc_mxf8(int n, int byte)
{
    return (static_cast<uint32_t>(byte) << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) |
           (static_cast<uint32_t>(WM >> 4) << 24) | (static_cast<uint32_t>(byte) << 29);
}

// D (+)= (A scaled) * (B scaled)^T.
__device__ __forceinline__ void umma_mxf8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                          uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}

// 32 rows of 16 bytes from shared memory to four TMEM columns, repeated in
// every lane quarter.
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc)
{
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

// A copy of four bytes to shared memory that nobody waits for yet.
__device__ __forceinline__ void copy_ahead(float *dst, const float *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until all but this thread's last N groups of copies have landed.
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint32_t cluster_nctas()
{
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return n;
}
__device__ __forceinline__ float load_cluster(uint32_t cluster_addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr));
    return v;
}

// A predicated 4-byte store (a branch around a plain one costs the unrolled
// epilogues up to a third of their time).
__device__ __forceinline__ void store_if(bool p, void *dst, uint32_t v)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %0, 0;\n\t@q st.global.b32 [%1], %2;\n\t}\n" ::"r"(static_cast<int>(p)),
                 "l"(dst), "r"(v)
                 : "memory");
}

// Four lanes hold a column each, of the same four rows (a byte per row): lane
// r of them gets row r's four columns.
__device__ __forceinline__ uint32_t transpose4(uint32_t w, int lane)
{
    const uint32_t y = __shfl_xor_sync(0xffffffffu, w, 1);
    w = __byte_perm(w, y, lane & 1 ? 0x3715u : 0x6240u);
    const uint32_t z = __shfl_xor_sync(0xffffffffu, w, 2);
    return __byte_perm(w, z, lane & 2 ? 0x3276u : 0x5410u);
}

// Tiles at most: every slice may end inside one.
template <typename S> int64_t most_tiles(const Fp8GemmArgs &a, int64_t n_tiles)
{
    return (a.rows / S::NMAX + min64(a.E, a.rows)) * n_tiles;
}

// SPLIT: a cluster of CTAs per tile, each with its share of the k-blocks;
// one tile per cluster (the grid has room for all).
template <int EPI, typename S, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1)
    ffn_gemm_mxfp8_kernel(const __grid_constant__ RowMaps tmA, const __grid_constant__ CUtensorMap tmW,
                          const __grid_constant__ CUtensorMap tmW3, const GemmArgs g)
{
    constexpr bool kHidden = EPI == EPI_SWIGLU || EPI == EPI_GELU;
    // the epilogue's halves: an accumulator each, or every other 32 rows
    constexpr bool kHalfAcc = S::ACC == 2 && EPI != EPI_SWIGLU;
    static_assert(EPI != EPI_SWIGLU || S::ACC == 2, "gate and up");
    static_assert(EPI != EPI_GELU || S::ACC == 1, "a tile fits the epilogue's registers");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *tiles = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                 ~static_cast<uintptr_t>(1023));
    Ctl<S> *ctl = reinterpret_cast<Ctl<S> *>(tiles + S::STAGES * S::STAGE);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *abort_flag = &ctl->abort;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::STAGES; ++s) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        for (int s = 0; s < SLOTS; ++s) {
            mbar_init(&ctl->sfull[s], S::ATOMS);
            mbar_init(&ctl->sempty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ctl->tfull[b], 1);
            mbar_init(&ctl->tempty[b], SUM_WARPS);
            mbar_init(&ctl->there[b], SUM_WARPS / 2);
        }
        mbar_init(&ctl->drain, 1);
        ctl->abort = 0;
        fence_mbar_init();
    }
    if (threadIdx.x == 32) {
        for (int i = 0; i < 4; ++i) prefetch_tmap(&tmA.box[i]);
        prefetch_tmap(&tmW);
        if (EPI == EPI_SWIGLU) prefetch_tmap(&tmW3);
    }
    if (warp == 1) {
        tmem_alloc(&ctl->tmem_base, TMEM_COLS);
        tmem_relinquish();
    }
    // nothing above touches memory that an earlier kernel writes
    const int ranks = SPLIT ? static_cast<int>(cluster_nctas()) : 1, rank = SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
    // The stream's previous kernel may have written the slices and the weights
    // (then wait for it here) or, inside an FFN, only the rows: then what does
    // not depend on it starts now, and every warp waits before its part.
    if (!g.early) pdl_enter();
    auto begin = [&] {
        if (g.early) pdl_enter();
    };
    tc_fence_before();
    load_slices<S::NMAX>(&ctl->slices, g);
    tc_fence_after();

    const Slices *sl = &ctl->slices;
    const uint32_t tmem_base = ctl->tmem_base;
    const int total = sl->mt[g.E] * g.n_tiles;
    const int first = static_cast<int>(blockIdx.x) / ranks, step = static_cast<int>(gridDim.x) / ranks;
    const int num_kb = (g.K + BK - 1) / BK;
    const int kb_lo = SPLIT ? rank * num_kb / ranks : 0, kb_hi = SPLIT ? (rank + 1) * num_kb / ranks : num_kb;
    constexpr int TILE_N = EPI == EPI_SWIGLU ? WM : S::ACC * WM;  // result columns of a tile
    // A slice's rows in tiles of equal size (a multiple of 16): the tiles of a
    // wave then take equally long.
    struct Rows {
        int first, count;  // of all rows; rows of the tile
    };
    auto rows_of = [&](const Tile &ti) {
        const int rows = sl->end[ti.e] - sl->off[ti.e], tiles_e = sl->mt[ti.e + 1] - sl->mt[ti.e];
        const int size = ((rows - 1) / tiles_e + 16) & ~15;
        return Rows{sl->off[ti.e] + ti.m_tile * size, min(size, rows - ti.m_tile * size)};
    };

    if (warp < FIRST_SUM_WARP) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(ROLE_REGS));
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------ TMA producer
            int stage = 0, ahead = 0;  // ahead: stages whose weights are on their way
            uint32_t phase = 0, armed = 0, armed_parity = 0;
            bool ok = true;
            auto load_weights = [&](int e, int n0, int n, int kb, int to) {
                uint8_t *sW = tiles + to * S::STAGE;
                uint64_t *full = &ctl->full[to];
                mbar_arrive_expect_tx(full, static_cast<uint32_t>(S::W_BYTES + n * BK));
                armed |= 1u << to;
                armed_parity = (armed_parity & ~(1u << to)) | (phase << to);
                tma_load_3d(sW, &tmW, full, kb * BK, n0, e);
                if (EPI == EPI_SWIGLU) tma_load_3d(sW + WM * BK, &tmW3, full, kb * BK, n0, e);
            };
            if (g.early && first < total) {
                const Tile ti = decode_tile(first, sl, g.E, g.n_tiles);
                const int n = (rows_of(ti).count + 15) & ~15;
                for (; ahead < min(S::STAGES, kb_hi - kb_lo); ++ahead)
                    load_weights(ti.e, ti.n_tile * TILE_N, n, kb_lo + ahead, ahead);
            }
            begin();
            for (int t = first; t < total && ok; t += step) {
                const Tile ti = decode_tile(t, sl, g.E, g.n_tiles);
                const Rows tr = rows_of(ti);
                const int row0 = tr.first, n0 = ti.n_tile * TILE_N, n = (tr.count + 15) & ~15;
                for (int kb = kb_lo; kb < kb_hi; ++kb) {
                    if (ahead > 0) {
                        --ahead;
                    } else {
                        if (!mbar_wait(&ctl->empty[stage], phase ^ 1u, abort_flag, g.status)) {
                            ok = false;
                            break;
                        }
                        load_weights(ti.e, n0, n, kb, stage);
                    }
                    uint8_t *sA = tiles + stage * S::STAGE + S::W_BYTES;
                    uint64_t *full = &ctl->full[stage];
                    int r = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int rows = 128 >> i;
                        if (n & rows) {
                            tma_load_3d(sA + r * BK, &tmA.box[i], full, kb * BK, row0 + r, 0);
                            r += rows;
                        }
                    }
                    if (++stage == S::STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (*abort_flag) {
                // let every copy this thread started land before the CTA exits
                for (int s = 0; s < S::STAGES; ++s)
                    if ((armed >> s) & 1u)
                        mbar_wait(&ctl->full[s], (armed_parity >> s) & 1u, abort_flag, g.status, false);
            }
        } else if (warp == 1 && lane == 0) {
            // -------------------------------------------------- MMA issuer
            begin();
            int stage = 0, buf = 0;
            uint32_t phase = 0, tphase = 0, group = 0;
            bool ok = true, issued = false;
            for (int t = first; t < total && ok; t += step) {
                const Tile ti = decode_tile(t, sl, g.E, g.n_tiles);
                const int n = (rows_of(ti).count + 15) & ~15;
                const bool both = S::ACC == 2 && (EPI == EPI_SWIGLU || ti.n_tile * TILE_N + WM < g.n_out);
                if (!mbar_wait(&ctl->tempty[buf], tphase ^ 1u, abort_flag, g.status)) break;
                tc_fence_after();
                const uint32_t d = tmem_base + static_cast<uint32_t>(buf * S::ACC * S::NMAX);
                for (int kb0 = kb_lo; kb0 < kb_hi && ok; kb0 += GROUP) {
                    // The group's scales are there, and the MMAs of the
                    // group before the last, which read the same TMEM
                    // columns, are done.
                    const uint32_t slot = group % SLOTS, last = (group - 2) % SLOTS;
                    if (!mbar_wait(&ctl->sfull[slot], group / SLOTS & 1u, abort_flag, g.status) ||
                        (group >= 2 &&
                         !mbar_wait(&ctl->sempty[last], (group - 2) / SLOTS & 1u, abort_flag, g.status))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sw = tmem_base + S::SCALE_COL + (group & 1u) * S::SLOT_COLS, sr = sw + 4u * S::ACC;
                    const uint32_t src = smem_u32(ctl->scales[slot]);
                    copy_scales(sw, desc_scales(src));
                    if (S::ACC == 2) copy_scales(sw + 4u, desc_scales(src + 512));
                    copy_scales(sr, desc_scales(src + 1024));
                    if (S::ATOMS == 2) copy_scales(sr + 4u, desc_scales(src + 1536));
                    issued = true;
                    const int kbs = min(GROUP, kb_hi - kb0);
                    for (int j = 0; j < kbs; ++j) {
                        if (!mbar_wait(&ctl->full[stage], phase, abort_flag, g.status)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t w_addr = smem_u32(tiles + stage * S::STAGE), a_addr = w_addr + S::W_BYTES;
                        const uint32_t idesc = idesc_mxf8(n, j), add = kb0 + j != kb_lo ? 1u : 0u;
#pragma unroll
                        for (int kk = 0; kk < BK / 32; ++kk)
                            umma_mxf8(d, desc_sw128(w_addr + kk * 32), desc_sw128(a_addr + kk * 32), idesc, sw, sr,
                                      kk ? 1u : add);
                        if (both) {
#pragma unroll
                            for (int kk = 0; kk < BK / 32; ++kk)
                                umma_mxf8(d + S::NMAX, desc_sw128(w_addr + WM * BK + kk * 32),
                                          desc_sw128(a_addr + kk * 32), idesc, sw + 4u, sr, kk ? 1u : add);
                        }
                        umma_commit(&ctl->empty[stage]);
                        if (++stage == S::STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (!ok) break;
                    umma_commit(&ctl->sempty[slot]);
                    ++group;
                }
                if (!ok) break;
                umma_commit(&ctl->tfull[buf]);
                if (++buf == S::BUFS) {
                    buf = 0;
                    tphase ^= 1u;
                }
            }
            if (*abort_flag && issued) {
                // wait for every MMA issued so far before TMEM is freed
                umma_commit(&ctl->drain);
                mbar_wait(&ctl->drain, 0, abort_flag, g.status, false);
            }
        } else if (warp >= 2 && warp - 2 < S::ATOMS) {
            // ------------------------------------------------------ scales
            begin();
            const int atom = warp - 2;
            const int nblocks = (g.n_out + kFp8Block - 1) / kFp8Block;
            bool odd_scale = false;
            // Copies of a group's values on their way: rows lane, lane + 32,
            // ... of four k-blocks; lanes 0-3 and 4-7: the two accumulators'
            // weights.  1 where there is none.
            Tile ti{};
            Rows tr{};
            int t_ahead = first, kb_ahead = kb_lo, decoded = -1;
            auto fetch = [&](float (&to)[4 * GROUP + 1][32]) {
                if (t_ahead < total) {
                    if (decoded != t_ahead) {
                        ti = decode_tile(t_ahead, sl, g.E, g.n_tiles);
                        tr = rows_of(ti);
                        decoded = t_ahead;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = atom * 128 + 32 * i + lane;
                        const float *p = g.a_scales + tr.first + r + static_cast<int64_t>(kb_ahead) * g.rows;
#pragma unroll
                        for (int j = 0; j < GROUP; ++j) {
                            float *dst = &to[i * GROUP + j][lane];
                            if (r < tr.count && kb_ahead + j < kb_hi) copy_ahead(dst, p + static_cast<int64_t>(j) * g.rows);
                            else *dst = 1.0f;
                        }
                    }
                    const int j = kb_ahead + (lane & 3), h = lane >> 2 & 1;
                    const int nb = EPI == EPI_SWIGLU ? ti.n_tile : min(ti.n_tile * S::ACC + h, nblocks - 1);
                    const float *p = (EPI == EPI_SWIGLU && h ? g.w3_scales : g.w_scales) +
                                     (static_cast<int64_t>(ti.e) * nblocks + nb) * num_kb;
                    float *dst = &to[4 * GROUP][lane];
                    if (atom == 0 && lane < 8 && j < kb_hi) copy_ahead(dst, p + j);
                    else *dst = 1.0f;
                }
                copy_commit();
                if ((kb_ahead += GROUP) >= kb_hi) {
                    kb_ahead = kb_lo;
                    t_ahead += step;
                }
            };
            // exponent codes; a scale that is neither a positive normal power
            // of two nor NaN is reported, and its products are NaN: whoever
            // does not look at the status sees it too
            auto code = [&](float v) {
                const uint32_t b = __float_as_uint(v), e = b >> 23;
                const bool nan = (b & 0x7FFFFFFFu) > 0x7F800000u, pow2 = e - 1u < 254u && (b & 0x7FFFFFu) == 0;
                odd_scale |= !nan && !pow2;
                return pow2 ? e : 255u;
            };
            for (int i = 0; i + 1 < AHEAD; ++i) fetch(ctl->ahead[atom][i]);
            uint32_t group = 0;
            bool ok = true;
            for (int t = first; t < total && ok; t += step) {
                for (int kb0 = kb_lo; kb0 < kb_hi; kb0 += GROUP, ++group) {
                    fetch(ctl->ahead[atom][(group + AHEAD - 1) % AHEAD]);
                    copy_wait<AHEAD - 1>();
                    const float(&a)[4 * GROUP + 1][32] = ctl->ahead[atom][group % AHEAD];
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        w[i] = 0;
#pragma unroll
                        for (int j = 0; j < GROUP; ++j) w[i] |= code(a[i * GROUP + j][lane]) << (8 * j);
                    }
                    uint32_t e = code(a[4 * GROUP][lane]) << (8 * (lane & 3));
                    e |= __shfl_xor_sync(0xffffffffu, e, 1);
                    e |= __shfl_xor_sync(0xffffffffu, e, 2);
                    const uint32_t w0 = __shfl_sync(0xffffffffu, e, 0), w1 = __shfl_sync(0xffffffffu, e, 4);
                    const uint32_t slot = group % SLOTS;
                    if (!__all_sync(0xffffffffu,
                                    mbar_wait(&ctl->sempty[slot], (group / SLOTS & 1u) ^ 1u, abort_flag, g.status))) {
                        ok = false;
                        break;
                    }
                    uint8_t *dst = ctl->scales[slot] + lane * 16;
                    st16(dst + 1024 + 512 * atom, make_uint4(w[0], w[1], w[2], w[3]));
                    if (atom == 0) {
                        st16(dst, make_uint4(w0, w0, w0, w0));
                        st16(dst + 512, make_uint4(w1, w1, w1, w1));
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl->sfull[slot]);
                }
            }
            copy_wait<0>();  // none of this thread's copies is left behind
            if (odd_scale) set_status(g.status, kDevBadArgument);
        }
        if constexpr (SPLIT) {
            __syncwarp();
            cluster_sync();  // the other warps' comes with the exchange of accumulators
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SUM_REGS));
        // ---------------------------------------------------- epilogue
        begin();
        const int quarter = warp & 3, half = (warp - FIRST_SUM_WARP) >> 2;
        int buf = 0;
        uint32_t tphase = 0, xphase = 0;
        bool met = false;
        // SPLIT: the others leave this thread's accumulator values of one
        // chunk of rows (accumulator i) in shared memory; after the cluster
        // has met, rank 0 adds them.
        float *part = reinterpret_cast<float *>(tiles) + quarter * 32 + lane;
        auto leave = [&](const uint32_t (&v)[32], int i, int rows) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (j < rows) part[(32 * i + j) * WM] = __uint_as_float(v[j]);
        };
        auto gather = [&](uint32_t (&v)[32], int i, int rows) {
            for (int r = 1; r < ranks; ++r) {
                const uint32_t from = mapa_shared(smem_u32(part + 32 * i * WM), static_cast<uint32_t>(r));
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (j < rows)
                        v[j] = __float_as_uint(__uint_as_float(v[j]) + load_cluster(from + static_cast<uint32_t>(j * WM * 4)));
            }
        };
        for (int t = first; t < total; t += step) {
            const Tile ti = decode_tile(t, sl, g.E, g.n_tiles);
            const Rows tr = rows_of(ti);
            const int rows = tr.count;
            const int64_t row0 = tr.first;
            if (!__all_sync(0xffffffffu, mbar_wait(&ctl->tfull[buf], tphase, abort_flag, g.status))) break;
            tc_fence_after();
            const uint32_t tbase =
                tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(buf * S::ACC * S::NMAX) +
                (kHalfAcc ? static_cast<uint32_t>(half * S::NMAX) : 0u);
            // this warp's loads from TMEM have completed
            auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->tempty[buf]);
                if (++buf == S::BUFS) {
                    buf = 0;
                    tphase ^= 1u;
                }
            };
            // the first of this warp's 32 result columns, and this lane's
            const int col0 = ti.n_tile * TILE_N + (kHalfAcc ? half * WM : 0) + quarter * 32, col = col0 + lane;
            // this warp's chunks of 32 rows
            constexpr int CH = (S::NMAX + (kHalfAcc ? 31 : 63)) / (kHalfAcc ? 32 : 64);
            auto first_row = [&](int i) { return kHalfAcc ? 32 * i : 64 * i + 32 * half; };
            float bias = 0.0f;
            if (EPI != EPI_SWIGLU && g.bias && col < g.n_out)
                bias = to_f32(g.bias[static_cast<int64_t>(ti.e) * g.n_out + col]);

            if constexpr (kHidden) {
                float h[CH][32];
                uint32_t m[CH];  // lane j: the largest |h| of the chunk's row j over this warp's lanes
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    m[i] = 0;
                    const int r0 = first_row(i);
                    if (r0 >= rows) continue;
                    uint32_t v[32], up[32];
                    if constexpr (EPI == EPI_SWIGLU) {
                        tmem_ld32(tbase + r0, v);
                        tmem_ld32(tbase + S::NMAX + r0, up);
                        tmem_ld_wait(v);
                        tmem_ld_wait(up);
                    } else {
                        tmem_ld32(tbase + r0, v);
                        tmem_ld_wait(v);
                    }
                    if constexpr (SPLIT) {  // one chunk, of the first half
                        if (rank != 0) {
                            leave(v, 0, rows);
                            if (EPI == EPI_SWIGLU) leave(up, 1, rows);
                        }
                        cluster_sync();
                        met = true;
                        if (rank != 0) break;
                        gather(v, 0, rows);
                        if (EPI == EPI_SWIGLU) gather(up, 1, rows);
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if constexpr (EPI == EPI_SWIGLU)
                            h[i][j] = silu_approx(__uint_as_float(v[j])) * __uint_as_float(up[j]);
                        else
                            h[i][j] = gelu_erf(__uint_as_float(v[j]) + bias);
                        const uint32_t top = __reduce_max_sync(0xffffffffu, abs_bits(h[i][j]));
                        m[i] = lane == j ? top : m[i];
                    }
                }
                release();
                if (SPLIT && rank != 0) break;
                // over the four lane quarters; two sets of values by phase: a
                // warp that is a tile ahead writes the other set, and it
                // cannot be two ahead
#pragma unroll
                for (int i = 0; i < CH; ++i) ctl->amax[xphase][half][quarter][32 * i + lane] = m[i];
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->there[half]);
                if (!__all_sync(0xffffffffu, mbar_wait(&ctl->there[half], xphase, abort_flag, g.status))) break;
                uint8_t *out = static_cast<uint8_t *>(g.out);
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const int r0 = first_row(i);
                    if (r0 >= rows) continue;
#pragma unroll
                    for (int q = 0; q < 4; ++q) m[i] = max(m[i], ctl->amax[xphase][half][q][32 * i + lane]);
                    const float2 s = fp8_scale(m[i]);
                    if (quarter == 0 && r0 + lane < rows)
                        g.h_scales[static_cast<int64_t>(ti.n_tile) * g.rows + row0 + r0 + lane] = s.x;
                    uint8_t *at = out + (row0 + r0 + (lane & 3)) * g.n_out + col0 + (lane & ~3);
                    const int left = col0 + (lane & ~3) < g.n_out ? rows - r0 - (lane & 3) : 0;
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        float x[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) x[u] = h[i][j + u] * __shfl_sync(0xffffffffu, s.y, j + u);
                        const uint32_t w = transpose4(cvt_e4m3x4(x[0], x[1], x[2], x[3]), lane);
                        store_if(left > j, at, w);
                        at += 4 * static_cast<int64_t>(g.n_out);
                    }
                }
                xphase ^= 1u;
            } else {
                if (col0 >= g.n_out) {
                    release();
                    continue;
                }
                // bf16: pairs of rows, packed; even lanes store two columns of
                // a pair's first row, odd lanes of its second.  fp32: a
                // column a lane.
                constexpr bool kBf16 = EPI == EPI_BF16;
                constexpr int PER = kBf16 ? 16 : 32, ROWS = kBf16 ? 2 : 1, ES = kBf16 ? 2 : 4;
                const uint32_t pick = lane & 1 ? 0x3276u : 0x5410u;
                const int sub = kBf16 ? lane & 1 : 0, c = col0 + lane - sub;
                const int64_t row_bytes = static_cast<int64_t>(g.n_out) * ES;
                uint8_t *out = static_cast<uint8_t *>(g.out) + (row0 + first_row(0) + sub) * row_bytes + static_cast<int64_t>(c) * ES;
                int left = c < g.n_out ? rows - first_row(0) - sub : 0;  // rows from `out` on
                auto store = [&](const uint32_t (&p)[PER]) {
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        uint32_t w = p[j];
                        if constexpr (kBf16) w = __byte_perm(w, __shfl_xor_sync(0xffffffffu, w, 1), pick);
                        store_if(left > 0, out, w);
                        out += ROWS * row_bytes;
                        left -= ROWS;
                    }
                    if (!kHalfAcc) {  // past the other half's chunk
                        out += 32 * row_bytes;
                        left -= 32;
                    }
                };
                // The tile is held in registers where they suffice, and
                // TMEM released before the first store.
                constexpr bool kHold = CH * PER <= 128;
                uint32_t v[2][32], p[kHold ? CH : 1][PER];
                if (first_row(0) < rows) tmem_ld32(tbase + first_row(0), v[0]);
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    if (first_row(i) < rows) {
                        uint32_t(&x)[32] = v[i & 1];
                        tmem_ld_wait(x);
                        if constexpr (SPLIT) {  // one chunk, of the first half
                            if (rank != 0) leave(x, 0, rows);
                            cluster_sync();
                            met = true;
                            if (rank != 0) break;
                            gather(x, 0, rows);
                        }
                        if (i + 1 < CH && first_row(i + 1) < rows) tmem_ld32(tbase + first_row(i + 1), v[(i + 1) & 1]);
                        else if (!kHold) release();
                        if (g.bias) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) + bias);
                        }
                        uint32_t(&q)[PER] = p[kHold ? i : 0];
#pragma unroll
                        for (int j = 0; j < PER; ++j) {
                            if constexpr (kBf16) q[j] = pack_bf16x2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]));
                            else q[j] = x[j];
                        }
                        if (!kHold) store(q);
                    }
                }
                if (SPLIT && rank != 0) break;
                if (kHold || first_row(0) >= rows) release();
                if constexpr (kHold) {
#pragma unroll
                    for (int i = 0; i < CH; ++i)
                        if (first_row(i) < rows) store(p[i]);
                }
            }
        }
        if (SPLIT && !met) {
            __syncwarp();
            cluster_sync();
        }
    }

    tc_fence_before();
    __syncthreads();
    // nobody's shared memory goes while rank 0 reads it
    if constexpr (SPLIT) cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

template <int EPI, typename S, bool SPLIT = false>
cudaError_t launch(const Fp8GemmArgs &a, int num_sms, cudaStream_t s, int ranks = 1)
{
    static_assert(!SPLIT || S::NMAX <= 32, "one chunk of rows is exchanged");
    RowMaps tmA;
    CUtensorMap tmW, tmW3;
    constexpr bool kTwo = EPI == EPI_SWIGLU;
    constexpr int TILE_N = kTwo ? WM : S::ACC * WM;
    for (int i = 0; i < 4; ++i)
        if (!make_tmap_u8(&tmA.box[i], a.a, a.k, a.rows, 1, 128u >> i)) return cudaErrorInvalidValue;
    if (!make_tmap_u8(&tmW, a.w, a.k, a.n, a.E, TILE_N) || !make_tmap_u8(&tmW3, kTwo ? a.w3 : a.w, a.k, a.n, a.E, TILE_N))
        return cudaErrorInvalidValue;
    auto *kernel = ffn_gemm_mxfp8_kernel<EPI, S, SPLIT>;
    cudaError_t err = ensure_smem_attr(reinterpret_cast<const void *>(kernel), static_cast<int>(smem_bytes<S>()));
    if (err != cudaSuccess) return err;
    const GemmArgs g = gemm_args(a, TILE_N);
    const int64_t most = most_tiles<S>(a, g.n_tiles);
    if (most * ranks > (static_cast<int64_t>(1) << 30)) return cudaErrorInvalidValue;  // tile numbers and a step
    const dim3 grid(static_cast<unsigned>(SPLIT ? most * ranks : min64(most, num_sms)));
    return launch_clusters(kernel, grid, dim3(THREADS), ranks, smem_bytes<S>(), s, tmA, tmW, tmW3, g);
}

// The small shapes, with a tile's k-blocks split where all tiles leave at
// least half of the SMs idle and every part keeps two groups of k-blocks.
template <int EPI, typename S> cudaError_t launch_split(const Fp8GemmArgs &a, int num_sms, cudaStream_t s)
{
    constexpr int TILE_N = EPI == EPI_SWIGLU ? WM : S::ACC * WM;
    const int64_t most = most_tiles<S>(a, (a.n + TILE_N - 1) / TILE_N);
    const int num_kb = (a.k + BK - 1) / BK;
    for (int ranks = 8; ranks > 1; ranks /= 2)
        if (most * ranks <= num_sms && num_kb >= 2 * GROUP * ranks) return launch<EPI, S, true>(a, num_sms, s, ranks);
    return launch<EPI, S>(a, num_sms, s);
}

// Which shape: by the average rows of a slice, and where few waves of tiles
// fill the SMs, by how many there are.
enum { WIDE, TALL, FEW, TINY, TINY_TALL };
int shape_of(const Fp8GemmArgs &a, int num_sms)
{
    const int64_t each = (a.rows + a.E - 1) / a.E;
    auto tiles = [&](int64_t slices, int64_t tile_n) { return slices * ((a.n + tile_n - 1) / tile_n); };
    // fewer weight tiles than half the SMs: smaller ones keep more SMs reading
    // (one row, n = k = 4096: 25 us by 16 tiles, 18 by 32; 128 tiles: equal)
    if (each <= kTinyRows) return tiles(min64(a.rows, a.E), WM) <= num_sms ? TINY_TALL : TINY;
    if (each <= kFewRows) return FEW;
    // A wave of tall tiles takes about 0.59 of one of wide tiles (735 against
    // 1230 cycles a k-block, by the bytes of shared memory), so twice as many
    // of them can fill the SMs better.  8 x 600 rows, n = k = 2048: 28 us tall,
    // 31 wide; 4096 rows of one expert, n = k = 4096: 63 and 56.
    const int64_t slices = (each + Wide::NMAX - 1) / Wide::NMAX * a.E;
    auto waves = [&](int64_t tile_n) { return (tiles(slices, tile_n) + num_sms - 1) / num_sms; };
    return 100 * waves(2 * WM) > 59 * waves(WM) ? TALL : WIDE;
}

template <int EPI> cudaError_t launch_rows(const Fp8GemmArgs &a, int num_sms, cudaStream_t s)
{
    switch (shape_of(a, num_sms)) {
        case WIDE: return launch<EPI, Wide>(a, num_sms, s);
        case TALL: return launch<EPI, Tall>(a, num_sms, s);
        case FEW: return launch<EPI, Few>(a, num_sms, s);
        case TINY: return launch<EPI, Tiny>(a, num_sms, s);  // more tiles than SMs
        default: return launch_split<EPI, TinyTall>(a, num_sms, s);
    }
}

}  // namespace

cudaError_t launch_gemm_mxfp8(const Fp8GemmArgs &a, int num_sms, cudaStream_t s)
{
    if (a.rows == 0) return cudaSuccess;
    const int64_t each = (a.rows + a.E - 1) / a.E;
    switch (a.epi) {
        case kFp8Swiglu:  // always two accumulators, gate and up
            return each <= kTinyRows  ? launch_split<EPI_SWIGLU, Tiny>(a, num_sms, s)
                   : each <= kFewRows ? launch<EPI_SWIGLU, Few>(a, num_sms, s)
                                      : launch<EPI_SWIGLU, Wide>(a, num_sms, s);
        case kFp8Gelu:  // always one: a thread holds its values
            return each <= kTinyRows ? launch_split<EPI_GELU, TinyTall>(a, num_sms, s) : launch<EPI_GELU, Tall>(a, num_sms, s);
        case kFp8Bf16: return launch_rows<EPI_BF16>(a, num_sms, s);
        default: return launch_rows<EPI_F32>(a, num_sms, s);
    }
}

}  // namespace moe
