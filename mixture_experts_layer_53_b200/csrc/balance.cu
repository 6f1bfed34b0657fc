// balance.cu -- balance loss over sequences, per-expert counts, and the
// gradient of the router's logits.
//
// With T_s valid tokens in sequence s, scores p_n = softmax(z_n) or
// sigmoid(z_n) / sum_j sigmoid(z_{n,j}), cnt_{s,e} the assignments to e and
// P_{s,e} = sum_n p_{n,e} over the sequence's valid tokens:
//   L = 1/S' sum_{s: T_s > 0} E / T_s^2 sum_e cnt_{s,e} P_{s,e}
//   dL/dz_{n,e} = p_{n,e} m_{n,e} (c_{s,e} - sum_j p_{n,j} c_{s,j}),
//   c_{s,e} = cnt_{s,e} E / (S' T_s^2), m = 1 (softmax), 1 - sigmoid(z_{n,e}),
// S' the sequences with a valid token (course module "Mixture of Experts",
// sec. 2.3, with the averages over one sequence instead of the batch).
//
// A token's E scores lie on G lanes, 4 * NV consecutive-by-four experts per
// lane, so that a lane keeps its experts for all tokens it visits and P_{s,e}
// is summed in its registers.  Both passes are bound by reading the logits
// (and writing the gradient); the exponentials run on the special-function
// unit.  Everything is summed in a fixed order (floats) or in integers: equal
// inputs give equal bits.  131072 tokens x 256 experts of fp32, sigmoid scores:
// the loss's two kernels 37 and 14 us (reading takes 21), the gradient 48 us (41);
// the step, whose kernels' starts and ends overlap, 86 us.
#include <cuda_runtime.h>

#include <type_traits>

#include "common.cuh"
#include "host_util.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Tokens a lane group handles at once; the next ones are on their way from
// memory meanwhile.  (At E = 256, 131072 tokens of fp32: one token 47 us for
// the gradient, two 52 us with more registers; the loss 46.9 and 44.9 us.)
constexpr int kForwardUnroll = 2, kBackwardUnroll = 1;
constexpr int kMinChunk = 32;
constexpr int kMaxChunks = 592;  // 148 SMs x 4 CTAs: one wave
// Scores of one expert that a lane adds in fp32, one after another, before
// the sum goes on to fp64; more tokens (from 450,000 of over 64 experts on)
// take more waves of chunks.  Equal scores round the same way, so a run's
// error can grow with its length: 1700 additions (8M tokens of 100 experts)
// were 2e-5 off.
constexpr int kMaxRun = 96;
constexpr int kBadId = 1, kBadCut = 2;  // flags of a segment or sequence

__host__ __device__ __forceinline__ int64_t align256(int64_t b) { return (b + 255) & ~static_cast<int64_t>(255); }

// Lanes that hold a token's E scores, and vectors of four experts per lane.
constexpr int lanes_of(int E) { return E <= 4 ? 1 : E <= 8 ? 2 : E <= 16 ? 4 : E <= 32 ? 8 : E <= 64 ? 16 : 32; }
constexpr int vectors_of(int E) { return E <= 128 ? 1 : 2; }

// Tokens [chunk c * C, (c + 1) * C) may touch several sequences.  The pairs
// (c, s) with common tokens increase in both, so c + s numbers them.
struct Plan {
    int64_t chunk, chunks, slots, ticket, psum, cnt, tok, tokens, dot, total;
    int groups;  // 32-expert groups of the second kernel
};

Plan make_plan(int64_t N, int E, int S)
{
    Plan p{};
    const int64_t most = kMaxRun * (kThreads / lanes_of(E));
    const int64_t ctas = kMaxChunks * max64(1, (N + kMaxChunks * most - 1) / (kMaxChunks * most));
    const int64_t even = (N + ctas - 1) / ctas;
    p.chunk = max64(kMinChunk, (even + 15) / 16 * 16);
    p.chunks = max64(1, (N + p.chunk - 1) / p.chunk);
    p.slots = p.chunks + S;
    p.groups = (E + 31) / 32;
    int64_t o = 0;
    auto take = [&o](int64_t bytes) {
        const int64_t at = o;
        o += align256(bytes);
        return at;
    };
    p.ticket = take(4);
    p.psum = take(p.slots * E * 4);
    p.cnt = take(p.slots * E * 4);
    p.tok = take(p.slots * 8);                        // int2: valid tokens, flags
    p.tokens = take(static_cast<int64_t>(S) * 8);     // int2
    p.dot = take(static_cast<int64_t>(S) * p.groups * 8);
    p.total = o;
    return p;
}

struct Seqs {
    const int32_t *off;
    int64_t N;
    // boundary i of the sequences, held inside 0 .. N
    __device__ __forceinline__ int64_t at(int i) const
    {
        if (!off) return i == 0 ? 0 : N;
        return min64(max64(__ldg(off + i), 0), N);
    }
    // the last sequence that starts at or before token n (0 if none does)
    __device__ __forceinline__ int find(int64_t n, int S) const
    {
        int lo = 0, hi = S - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (at(mid) <= n) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    }
};

// Loads that stay where they are written: one step ahead of their use.  The
// first pass leaves the logits in L2 for the second (the gradient's), which
// reads them last.
template <bool LAST> __device__ __forceinline__ float4 load_vec(const float4 *p)
{
    float4 v;
    if (LAST)
        asm volatile("ld.global.cs.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    else
        asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    return v;
}
template <bool LAST> __device__ __forceinline__ uint2 load_vec(const uint2 *p)
{
    uint2 v;
    if (LAST) asm volatile("ld.global.cs.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    else asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

// Four consecutive logits as loaded: fp32 values, or pairs of bf16.
template <typename T> struct Raw;
template <> struct Raw<float> {
    float4 v;
    __device__ __forceinline__ void none() { v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); }
    template <bool LAST> __device__ __forceinline__ void load(const float *p) { v = load_vec<LAST>(reinterpret_cast<const float4 *>(p)); }
    __device__ __forceinline__ void set(float a, float b, float c, float d) { v = make_float4(a, b, c, d); }
    __device__ __forceinline__ float4 get() const { return v; }
};
template <> struct Raw<__nv_bfloat16> {
    uint2 v;
    __device__ __forceinline__ void none() { v = make_uint2(0xFF80FF80u, 0xFF80FF80u); }
    template <bool LAST> __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = load_vec<LAST>(reinterpret_cast<const uint2 *>(p)); }
    __device__ __forceinline__ void set(float a, float b, float c, float d) { v = make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d)); }
    __device__ __forceinline__ float4 get() const
    {
        return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                           __uint_as_float(v.y & 0xFFFF0000u));
    }
};

// This lane's experts of a token: NV times four consecutive ones; -inf past E
// and for a token that is not used.
template <typename T, int NV> using Row = Raw<T>[NV];
template <bool LAST, int G, int NV, typename T>
__device__ __forceinline__ void load_token(Row<T, NV> &r, const T *row, bool use, int q, int E, bool vec)
{
    const float ninf = -INFINITY;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int e = (j * G + q) * 4;
        r[j].none();
        if (use && e < E) {
            if (vec) r[j].template load<LAST>(row + e);
            else
                r[j].set(to_f32(row[e]), e + 1 < E ? to_f32(row[e + 1]) : ninf, e + 2 < E ? to_f32(row[e + 2]) : ninf,
                         e + 3 < E ? to_f32(row[e + 3]) : ninf);
        }
    }
}
template <int NV, typename T> __device__ __forceinline__ void unpack(float (&z)[4 * NV], const Row<T, NV> &r)
{
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const float4 v = r[j].get();
        z[4 * j] = v.x;
        z[4 * j + 1] = v.y;
        z[4 * j + 2] = v.z;
        z[4 * j + 3] = v.w;
    }
}

// U values summed (or their maxima taken) over the G lanes of a group, the
// independent shuffles of the U next to each other.
template <int G, int U> __device__ __forceinline__ void group_sum(float (&v)[U])
{
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) {
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] += __shfl_xor_sync(0xffffffffu, v[u], o);
    }
}
template <int G, int U> __device__ __forceinline__ void group_max(float (&v)[U])
{
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) {
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = fmaxf(v[u], __shfl_xor_sync(0xffffffffu, v[u], o));
    }
}

constexpr float kLog2e = 1.44269504f;

// min that keeps a NaN
__device__ __forceinline__ float min_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Normalised scores of U tokens in place of their logits z; with SLOPE also m
// = 1 - sigmoid(z).  Every lane of the warp takes part.  A token whose logits
// are all -inf (or that is not used) has p = 0.  The exponent is the rounded
// product of z - max (or z) and log2 e, so its error is relative to it: about
// 1e-7 for the scores that matter, 6e-8 |z - max| for small ones.  `again`
// loads token u's logits once more, for the rare path that needs them.
template <int G, int NV, bool SIGMOID, bool SLOPE, int U, typename Again>
__device__ __forceinline__ void scores(float (&z)[U][4 * NV], float (&m)[SLOPE ? U : 1][4 * NV], const bool (&use)[U],
                                       Again &&again)
{
    constexpr int N = 4 * NV;
    float sum[U];
    if constexpr (!SIGMOID) {
        float top[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            top[u] = -INFINITY;
#pragma unroll
            for (int i = 0; i < N; ++i) top[u] = fmaxf(top[u], z[u][i]);
        }
        group_max<G>(top);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            top[u] = top[u] == -INFINITY ? 0.0f : top[u];
            sum[u] = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                z[u][i] = ex2_approx((z[u][i] - top[u]) * kLog2e);
                sum[u] += z[u][i];
            }
        }
        group_sum<G>(sum);
    } else {
        // sigma(z) = 1 / (1 + e), m = e sigma(z) with e = e^-z, held below
        // 2^127: the reciprocal is then 0 (a sigmoid under 2^-126), and
        // e times it no NaN.
#pragma unroll
        for (int u = 0; u < U; ++u) {
            sum[u] = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float e = ex2_approx(min_nan(z[u][i] * -kLog2e, 127.0f));
                z[u][i] = rcp_approx(1.0f + e);
                if constexpr (SLOPE) m[u][i] = e * z[u][i];
                sum[u] += z[u][i];
            }
        }
        group_sum<G>(sum);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool low = use[u] && sum[u] < 1e-6f;
            if (!__any_sync(0xffffffffu, low)) continue;
            // Every logit of a token is far below zero: the sigmoids underflow
            // but their ratios, those of e^z, do not.
            float x[N], top[1] = {-INFINITY}, ratios[1] = {0.0f};
            again(x, u);
#pragma unroll
            for (int i = 0; i < N; ++i) top[0] = fmaxf(top[0], x[i]);
            group_max<G>(top);
            if (top[0] == -INFINITY) top[0] = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                x[i] = ex2_approx((x[i] - top[0]) * kLog2e);
                ratios[0] += x[i];
                if (low) {
                    z[u][i] = x[i];
                    if constexpr (SLOPE) m[u][i] = 1.0f;
                }
            }
            group_sum<G>(ratios);
            if (low) sum[u] = ratios[0];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const float inv = sum[u] == 0.0f ? 0.0f : rcp_approx(sum[u]);
#pragma unroll
        for (int i = 0; i < N; ++i) z[u][i] *= inv;
    }
}

template <typename T, int G, int NV, bool SIGMOID>
__global__ void __launch_bounds__(kThreads, 4) balance_partial_kernel(const BalanceArgs a, const Plan p)
{
    pdl_enter();
    __shared__ float red[kWarps][G * 4 * NV];
    __shared__ int cnt[kMaxE];
    __shared__ int valid, bad;
    constexpr int GROUPS = kThreads / G;
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = threadIdx.x / G, q = threadIdx.x % G;
    if (blockIdx.x == 0 && threadIdx.x == 0) *reinterpret_cast<uint32_t *>(ws + p.ticket) = 0;
    const Seqs seqs{a.seq_offsets, a.N};
    const T *logits = static_cast<const T *>(a.logits);
    const bool vec = a.E % 4 == 0;
    const int64_t c = blockIdx.x, begin = c * p.chunk, end = min64(begin + p.chunk, a.N);
    for (int s = seqs.find(begin, a.S); s < a.S; ++s) {
        const int64_t lo = max64(seqs.at(s), begin), hi = min64(seqs.at(s + 1), end);
        if (lo >= end) break;
        if (lo >= hi) continue;
        __syncthreads();  // the last segment's shared sums have been read
        for (int i = threadIdx.x; i < a.E; i += kThreads) cnt[i] = 0;
        if (threadIdx.x == 0) valid = bad = 0;
        __syncthreads();
        float sum[4 * NV];
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) sum[i] = 0.0f;
        int mine = 0;
        constexpr int U = kForwardUnroll;
        Row<T, NV> next[U];
        bool used[U];
        auto load = [&](Row<T, NV> &r, int64_t n, bool use) {
            load_token<false, G, NV>(r, logits + n * a.E, use, q, a.E, vec);
        };
        auto fetch = [&](int64_t n0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t n = n0 + u * GROUPS + group;
                used[u] = n < hi && (!a.mask || a.mask[n] != 0);
                load(next[u], n, used[u]);
            }
        };
        fetch(lo);
        // counts, several ids of a thread on their way at once
        constexpr int IDS = 8;
        const int64_t ids = (hi - lo) * a.k;
        for (int64_t i0 = threadIdx.x; i0 < ids; i0 += kThreads * IDS) {
            int e[IDS];
            bool count[IDS];
#pragma unroll
            for (int i = 0; i < IDS; ++i) {
                const int64_t at = i0 + i * kThreads;
                count[i] = at < ids;
                e[i] = count[i] ? __ldg(a.ids + lo * a.k + at) : 0;
                if (a.mask && count[i]) count[i] = a.mask[lo + static_cast<int>(at) / a.k] != 0;
            }
#pragma unroll
            for (int i = 0; i < IDS; ++i) {
                if (!count[i]) continue;
                if (static_cast<unsigned>(e[i]) < static_cast<unsigned>(a.E)) atomicAdd(&cnt[e[i]], 1);
                else bad = kBadId;
            }
        }
        for (int64_t n0 = lo; n0 < hi; n0 += GROUPS * U) {
            float z[U][4 * NV], none[1][4 * NV];
            bool use[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                use[u] = used[u];
                mine += use[u] && q == 0;
                unpack<NV, T>(z[u], next[u]);
            }
            fetch(n0 + GROUPS * U);
            scores<G, NV, SIGMOID, false>(z, none, use, [&](float (&x)[4 * NV], int u) {
                Row<T, NV> r;
                load(r, n0 + u * GROUPS + group, use[u]);
                unpack<NV, T>(x, r);
            });
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int i = 0; i < 4 * NV; ++i) sum[i] += z[u][i];
            }
        }
        if (mine) atomicAdd(&valid, mine);
        // over the warp's lane groups, then over the warps
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) {
#pragma unroll
            for (int o = G; o < 32; o <<= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
        }
        if (lane < G) {
#pragma unroll
            for (int i = 0; i < 4 * NV; ++i) red[warp][(i / 4 * G + q) * 4 + i % 4] = sum[i];
        }
        __syncthreads();
        const int64_t slot = c + s;
        for (int e = threadIdx.x; e < a.E; e += kThreads) {
            float t = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) t += red[w][e];
            reinterpret_cast<float *>(ws + p.psum)[slot * a.E + e] = t;
            reinterpret_cast<int *>(ws + p.cnt)[slot * a.E + e] = cnt[e];
        }
        if (threadIdx.x == 0) reinterpret_cast<int2 *>(ws + p.tok)[slot] = make_int2(valid, bad);
    }
}

// One CTA per (sequence, 32 experts): its slots summed in fp64 (scores) and
// integers, counts written, its share of sum_e cnt P kept; the last CTA to
// finish forms the loss and the sequences' weights.
__global__ void __launch_bounds__(1024) balance_finish_kernel(const BalanceArgs a, const Plan p)
{
    pdl_enter();
    __shared__ double dsum[32][33];
    __shared__ int isum[32][33];
    __shared__ bool last;
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    const float *psum = reinterpret_cast<const float *>(ws + p.psum);
    const int *cnt = reinterpret_cast<const int *>(ws + p.cnt);
    const int2 *tok = reinterpret_cast<const int2 *>(ws + p.tok);
    int2 *tokens = reinterpret_cast<int2 *>(ws + p.tokens);
    double *dot = reinterpret_cast<double *>(ws + p.dot);
    uint32_t *ticket = reinterpret_cast<uint32_t *>(ws + p.ticket);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const Seqs seqs{a.seq_offsets, a.N};
    const int s = static_cast<int>(blockIdx.x / p.groups), gr = static_cast<int>(blockIdx.x % p.groups);
    const int e = gr * 32 + lane;
    const int64_t lo = seqs.at(s), hi = seqs.at(s + 1);
    const int64_t c0 = lo / p.chunk, c1 = hi > lo ? (hi - 1) / p.chunk + 1 : c0;
    double P = 0.0;
    int n = 0, T = 0, odd = 0;
    if (e < a.E) {
#pragma unroll 8
        for (int64_t c = c0 + warp; c < c1; c += warps) {
            P += psum[(c + s) * a.E + e];
            n += cnt[(c + s) * a.E + e];
        }
    }
    if (gr == 0)
        for (int64_t c = c0 + threadIdx.x; c < c1; c += blockDim.x) {
            const int2 t = tok[c + s];
            T += t.x;
            odd |= t.y;
        }
    dsum[warp][lane] = P;
    isum[warp][lane] = n;
    __syncthreads();
    if (warp == 0) {
        for (int w = 1; w < warps; ++w) {
            P += dsum[w][lane];
            n += isum[w][lane];
        }
        if (e < a.E) a.counts[static_cast<int64_t>(s) * a.E + e] = n;
        double d = e < a.E ? P * n : 0.0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        if (lane == 0) dot[static_cast<int64_t>(s) * p.groups + gr] = d;
    }
    __syncthreads();
    T = __reduce_add_sync(0xffffffffu, T);
    odd = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(odd));
    if (lane == 0) {
        isum[warp][0] = T;
        isum[warp][1] = odd;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        if (gr == 0) {
            int2 all = make_int2(0, 0);
            for (int w = 0; w < warps; ++w) {
                all.x += isum[w][0];
                all.y |= isum[w][1];
            }
            // offsets that decrease or leave 0 .. N
            if (a.seq_offsets && (a.seq_offsets[s] < 0 || a.seq_offsets[s + 1] < a.seq_offsets[s] || a.seq_offsets[s + 1] > a.N))
                all.y |= kBadCut;
            tokens[s] = all;
        }
        __threadfence();
        last = atomicAdd(ticket, 1u) + 1u == gridDim.x;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    // sequences with tokens
    int full = 0;
    odd = 0;
    for (int i = threadIdx.x; i < a.S; i += blockDim.x) {
        const int2 t = __ldcg(tokens + i);
        full += t.x > 0;
        odd |= t.y;
    }
    full = __reduce_add_sync(0xffffffffu, full);
    odd = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(odd));
    if (lane == 0) {
        isum[warp][0] = full;
        isum[warp][1] = odd;
    }
    __syncthreads();
    full = odd = 0;
    for (int w = 0; w < warps; ++w) {
        full += isum[w][0];
        odd |= isum[w][1];
    }
    double L = 0.0;
    for (int i = threadIdx.x; i < a.S; i += blockDim.x) {
        const double t = __ldcg(tokens + i).x;
        double d = 0.0;
        for (int j = 0; j < p.groups; ++j) d += __ldcg(dot + static_cast<int64_t>(i) * p.groups + j);
        const double w = t > 0.0 ? a.E / (t * t * full) : 0.0;
        a.seq_weight[i] = static_cast<float>(w);
        if (t > 0.0) L += w * d;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    __syncthreads();
    if (lane == 0) dsum[warp][0] = L;
    __syncthreads();
    if (threadIdx.x == 0) {
        L = 0.0;
        for (int w = 0; w < warps; ++w) L += dsum[w][0];
        *a.loss = static_cast<float>(L);
        if (a.status) *a.status = odd & kBadCut ? kDevBadArgument : odd & kBadId ? kDevBadExpertId : kDevOk;
    }
}

template <typename T, int G, int NV, bool SIGMOID>
__global__ void __launch_bounds__(kThreads, 4) balance_backward_kernel(const BalanceArgs a, int64_t per_cta)
{
    pdl_enter();
    constexpr int GROUPS = kThreads / G;
    const int group = threadIdx.x / G, q = threadIdx.x % G;
    const Seqs seqs{a.seq_offsets, a.N};
    const T *logits = static_cast<const T *>(a.logits);
    const bool vec = a.E % 4 == 0;
    const int64_t begin = blockIdx.x * per_cta, end = min64(begin + per_cta, a.N);
    const float scale = a.dloss ? a.coef * *a.dloss : a.coef;
    int s = seqs.find(min64(begin, a.N - 1), a.S), loaded = -1;
    int64_t lo = seqs.at(s), hi = seqs.at(s + 1);
    float c[4 * NV];
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) c[i] = 0.0f;
    constexpr int U = kBackwardUnroll;
    Row<T, NV> next[U];
    bool used[U];
    auto load = [&](Row<T, NV> &r, int64_t n, bool use) {
        load_token<true, G, NV>(r, logits + n * a.E, use, q, a.E, vec);
    };
    auto fetch = [&](int64_t n0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t n = n0 + u * GROUPS + group;
            used[u] = n < end && (!a.mask || a.mask[n] != 0);
            load(next[u], n, used[u]);
        }
    };
    fetch(begin);
    for (int64_t n0 = begin; n0 < end; n0 += GROUPS * U) {
        float z[U][4 * NV], m[SIGMOID ? U : 1][4 * NV];
        bool use[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            use[u] = used[u];
            unpack<NV, T>(z[u], next[u]);
        }
        fetch(n0 + GROUPS * U);
        scores<G, NV, SIGMOID, SIGMOID>(z, m, use, [&](float (&x)[4 * NV], int u) {
            Row<T, NV> r;
            load(r, n0 + u * GROUPS + group, use[u]);
            unpack<NV, T>(x, r);
        });
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t n = n0 + u * GROUPS + group;
            if (n < end) {
                while (n >= hi && s + 1 < a.S) {
                    ++s;
                    lo = hi;
                    hi = seqs.at(s + 1);
                }
            }
            const bool in = n >= lo && n < hi;
            if (in && n < end && loaded != s) {
                loaded = s;
                const float w = scale * a.seq_weight[s];
                const int32_t *cs = a.counts + static_cast<int64_t>(s) * a.E;
#pragma unroll
                for (int i = 0; i < 4 * NV; ++i) {
                    const int e = (i / 4 * G + q) * 4 + i % 4;
                    c[i] = e < a.E ? w * static_cast<float>(__ldg(cs + e)) : 0.0f;
                }
            }
            float dot[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < 4 * NV; ++i) dot[0] = fmaf(z[u][i], c[i], dot[0]);
            group_sum<G>(dot);
            if (n >= end) continue;
            const bool real = use[u] && in;
            float *out = a.dlogits + n * a.E;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int e = (j * G + q) * 4;
                float o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float g = z[u][4 * j + i] * (c[4 * j + i] - dot[0]);
                    if constexpr (SIGMOID) g *= m[u][4 * j + i];
                    o[i] = real ? g : 0.0f;
                }
                if (vec) {
                    if (e < a.E) __stcs(reinterpret_cast<float4 *>(out + e), make_float4(o[0], o[1], o[2], o[3]));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (e + i < a.E) out[e + i] = o[i];
                }
            }
        }
    }
}

// Calls f with the lanes per token and the vectors per lane for E experts.
template <int W, typename F> cudaError_t of_width(F &&f)
{
    return f(std::integral_constant<int, lanes_of(W)>{}, std::integral_constant<int, vectors_of(W)>{});
}
template <typename F> cudaError_t by_width(int E, F &&f)
{
    if (E <= 4) return of_width<4>(f);
    if (E <= 8) return of_width<8>(f);
    if (E <= 16) return of_width<16>(f);
    if (E <= 32) return of_width<32>(f);
    if (E <= 64) return of_width<64>(f);
    if (E <= 128) return of_width<128>(f);
    return of_width<kMaxE>(f);
}

template <typename T, bool SIGMOID> cudaError_t forward(const BalanceArgs &a, const Plan &p, cudaStream_t s)
{
    return by_width(a.E, [&](auto g, auto nv) {
        return launch_k(balance_partial_kernel<T, decltype(g)::value, decltype(nv)::value, SIGMOID>,
                        dim3(static_cast<unsigned>(p.chunks)), dim3(kThreads), 0, s, a, p);
    });
}

template <typename T, bool SIGMOID>
cudaError_t backward(const BalanceArgs &a, int64_t ctas, int64_t per_cta, cudaStream_t s)
{
    return by_width(a.E, [&](auto g, auto nv) {
        return launch_k(balance_backward_kernel<T, decltype(g)::value, decltype(nv)::value, SIGMOID>,
                        dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, s, a, per_cta);
    });
}

}  // namespace

size_t balance_workspace(int64_t N, int E, int S) { return static_cast<size_t>(make_plan(N, E, S).total); }

cudaError_t launch_balance_loss(const BalanceArgs &a, cudaStream_t s)
{
    const Plan p = make_plan(a.N, a.E, a.S);
    cudaError_t err;
    if (a.dtype == kF32) err = a.sigmoid ? forward<float, true>(a, p, s) : forward<float, false>(a, p, s);
    else err = a.sigmoid ? forward<__nv_bfloat16, true>(a, p, s) : forward<__nv_bfloat16, false>(a, p, s);
    if (err != cudaSuccess) return err;
    // four chunks of a sequence to a warp, as far as 32 warps go
    const int64_t each = p.chunks / a.S + 1;
    const int warps = static_cast<int>(min64(32, max64(2, each / 4)));
    const int64_t ctas = static_cast<int64_t>(a.S) * p.groups;
    if (ctas >= (static_cast<int64_t>(1) << 31)) return cudaErrorInvalidValue;
    return launch_k(balance_finish_kernel, dim3(static_cast<unsigned>(ctas)), dim3(32 * warps), 0, s, a, p);
}

cudaError_t launch_balance_backward(const BalanceArgs &a, int num_sms, cudaStream_t s)
{
    if (a.N == 0) return cudaSuccess;
    const int64_t most = static_cast<int64_t>(num_sms) * 8;
    const int64_t per_cta = max64(kMinChunk, (a.N + most - 1) / most), ctas = (a.N + per_cta - 1) / per_cta;
    if (a.dtype == kF32)
        return a.sigmoid ? backward<float, true>(a, ctas, per_cta, s) : backward<float, false>(a, ctas, per_cta, s);
    return a.sigmoid ? backward<__nv_bfloat16, true>(a, ctas, per_cta, s)
                     : backward<__nv_bfloat16, false>(a, ctas, per_cta, s);
}

}  // namespace moe
