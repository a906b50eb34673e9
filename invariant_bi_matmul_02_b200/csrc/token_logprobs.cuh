// token_logprobs.cuh -- per row of logits: the log-probability of a given token, the entropy, the log of
// the sum of exponentials and the k best alternatives, in one pass that writes no probabilities.
//
// With z = scale * x, m = max x, d = z - scale m and e = exp(d):
//   S = sum e,  T = sum e d,  logsumexp = scale m + log S,  logprob(t) = d_t - log S,
//   entropy = log S - T / S   (a term with e = 0 adds nothing, so -inf logits are allowed).
//
// Order (fixed by V and the type alone): the row is cut into pieces; in a piece each thread of the
// block owns 64 consecutive bytes (32 bf16 or 16 fp32 elements, a group).  A warp takes the maximum of
// its elements, then every thread's sums of e and e d over its group (two interleaved chains), then a
// fixed butterfly: one (m, S, T) per (piece, warp).  These are folded at the end by one warp: against the
// row's maximum, lane j adds triples j, j + 32, ... in order, then a fixed butterfly.  A row is taken by one block or
// by a cluster of 2, 4 or 8 that share its pieces; the triples, and so the bits, are the same.
//
// Many rows are bound by memory and by the issue slots (2.4 of 4 instructions a cycle, beside the special-function
// unit's half): 1024 rows of 151936 bf16 take 53 us, 5.9 TB/s, and fp32 96 us, 6.5 TB/s; with the 5 best 59 and
// 103 (from a replayed graph; as one call among others 64.5).  One row is bound by latency: 5.1 us, 8.0 to 8.4 with the 20
// best.
//
// The k best: only the groups' maxima are kept during the pass.  The k best elements lie in the k best groups (larger
// maximum first, lower group first among equals, as groups are consecutive), so the end of the row reads a few
// groups again instead of sorting.  What is compared are 64-bit keys (ordered value, inverted index): ties go to the
// lowest token, and the result does not depend on the order in which keys are met.  NaN counts as less than every number.
#pragma once

#include <cooperative_groups.h>
#include <cstdint>
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "rowops.cuh"

namespace bi {

constexpr int kTlThreads = 256;
constexpr int kTlBlocks = 4;                        // resident per SM, a bound on registers
constexpr int kTlWarps = kTlThreads / 32;
constexpr int kTlWords = 16;                        // 32-bit words per thread and piece
constexpr int kTlMaxV = 262144;
constexpr int kTlMaxTop = 32;
constexpr int kTlMaxCluster = 8;

__host__ __device__ constexpr int tl_group(bool bf16) { return bf16 ? 2 * kTlWords : kTlWords; }
__host__ __device__ constexpr int tl_piece(bool bf16) { return kTlThreads * tl_group(bf16); }  // 8192 or 4096
constexpr int kTlMaxPieces = kTlMaxV / tl_piece(false);

struct TlParams {
    const void *x;
    int64_t ldx;
    const int32_t *tokens;  // may be null
    float scale;            // multiplies the logits
    float scale_log2;       // scale * log2(e)
    int32_t V, top, pieces, cluster;
    float *logprobs, *entropy, *logsumexp;  // each may be null
    float *top_logprobs;    // [M, top]
    int32_t *top_tokens;
    int32_t *status;
};

struct TlTriple {
    float m, s, t;  // maximum of x, sum of e, sum of e * d in units of log2
};

__device__ __forceinline__ float tl_logprob(float x, float m, float scale, float log_s)
{
    return __fsub_rn(__fmul_rn(x - m, scale), log_s);
}

// Ascending with the value; -0 as +0, NaN below everything.
__device__ __forceinline__ uint32_t tl_order(float v)
{
    const uint32_t u = __float_as_uint(v + 0.0f);
    if (v != v) return 0u;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float tl_value(uint32_t o)
{
    return __uint_as_float(o == 0u ? 0x7fffffffu : o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint64_t tl_key(float v, uint32_t index)
{
    return (uint64_t)tl_order(v) << 32 | (uint32_t)~index;  // never 0: indices are below 2^31
}

// The warp's list of the largest keys, one per lane, descending (0: none yet); `k` of them count.
struct TlList {
    uint64_t mine = 0, kth = 0;
    // Offers one key per lane (0: none).
    __device__ __forceinline__ void offer(uint64_t key, int k)
    {
        const int lane = threadIdx.x & 31;
        unsigned better = __ballot_sync(0xffffffffu, key > kth);
        while (better) {
            const int src = __ffs(better) - 1;
            const uint64_t b = __shfl_sync(0xffffffffu, key, src);
            const int rank = __popc(__ballot_sync(0xffffffffu, mine > b));
            const uint64_t up = __shfl_up_sync(0xffffffffu, mine, 1);
            if (lane == rank) mine = b;
            else if (lane > rank) mine = up;
            kth = __shfl_sync(0xffffffffu, mine, k - 1);
            if (lane == src) key = 0;
            better = __ballot_sync(0xffffffffu, key > kth);
        }
    }
};

// A thread's group as it sits in memory.
template <bool BF16>
struct TlGroup {
    static constexpr int kSize = tl_group(BF16);
    uint32_t w[kTlWords];

    // Elements e0 .. e0 + kSize - 1 of a row of V; elements past V are -inf.  VEC: rows are 16-byte
    // aligned.  Otherwise a group inside the row is cut out of the five aligned 16-byte pieces around it
    // (all of them within the row), and the row's first and last groups are read by element.
    template <bool VEC>
    __device__ __forceinline__ void load(const void *row, int e0, int V)
    {
        constexpr int kBytes = BF16 ? 2 : 4, kPer16 = 16 / kBytes;
        const uint8_t *at = static_cast<const uint8_t *>(row) + (int64_t)e0 * kBytes;
        if (VEC && e0 + kSize <= V) {
            // A lane's pieces are 64 bytes from the next lane's: 32-byte loads take each sector once, 16-byte
            // ones leave its other half to the L1.
            if ((reinterpret_cast<uintptr_t>(at) & 31u) == 0) {
#pragma unroll
                for (int i = 0; i < kTlWords / 8; ++i) load_32(at + 32 * i, w + 8 * i);
            } else {
#pragma unroll
                for (int i = 0; i < kTlWords / 4; ++i) put(i, __ldcs(reinterpret_cast<const uint4 *>(at) + i));
            }
            return;
        }
        if (!VEC && e0 > 0 && e0 + kSize + kPer16 <= V) {
            const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(at) & 15u);  // the same for every group of the row
            const uint4 *src = reinterpret_cast<const uint4 *>(at - off);
            uint32_t x[kTlWords + 4];
#pragma unroll
            for (int i = 0; i < kTlWords / 4 + 1; ++i) {
                const uint4 v = src[i];
                x[4 * i] = v.x;
                x[4 * i + 1] = v.y;
                x[4 * i + 2] = v.z;
                x[4 * i + 3] = v.w;
            }
            if (off & 8u)
#pragma unroll
                for (int i = 0; i < kTlWords + 2; ++i) x[i] = x[i + 2];
            if (off & 4u)
#pragma unroll
                for (int i = 0; i < kTlWords + 1; ++i) x[i] = x[i + 1];
            if (BF16 && (off & 2u))
#pragma unroll
                for (int i = 0; i < kTlWords; ++i) x[i] = __funnelshift_r(x[i], x[i + 1], 16);
#pragma unroll
            for (int i = 0; i < kTlWords; ++i) w[i] = x[i];
            return;
        }
#pragma unroll
        for (int i = 0; i < kTlWords; ++i) {
            if (BF16) {
                const uint16_t *src = static_cast<const uint16_t *>(row) + e0 + 2 * i;
                const uint32_t a = e0 + 2 * i < V ? src[0] : 0xff80u, b = e0 + 2 * i + 1 < V ? src[1] : 0xff80u;
                w[i] = a | b << 16;
            } else {
                w[i] = e0 + i < V ? static_cast<const uint32_t *>(row)[e0 + i] : 0xff800000u;
            }
        }
    }
    __device__ __forceinline__ void put(int i, uint4 v)
    {
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
    }
    __device__ __forceinline__ uint64_t less(int i, float ref) const  // elements 2 i and 2 i + 1, less ref
    {
        if (!BF16) return f2_add(f2_pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])), f2_pack(-ref, -ref));
        float lo, hi;
        sub_bf16x2(w[i], ref, lo, hi);
        return f2_pack(lo, hi);
    }
    __device__ __forceinline__ float max() const
    {
        if (BF16) {
            __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162 *>(&w[0]);
#pragma unroll
            for (int i = 1; i < kTlWords; ++i) m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
            return fmaxf(__low2float(m), __high2float(m));
        }
        float m = __uint_as_float(w[0]);
#pragma unroll
        for (int i = 1; i < kTlWords; ++i) m = fmaxf(m, __uint_as_float(w[i]));
        return m;
    }
    // The maximum of the first n elements (1 .. kSize); NaN where no number is among them.
    __device__ __forceinline__ float max_below(int n) const
    {
        float m = __int_as_float(0x7fffffff);
#pragma unroll
        for (int i = 0; i < kSize; ++i) {
            const uint32_t bits = !BF16 ? w[i] : i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16;
            if (i < n) m = fmaxf(m, __uint_as_float(bits));
        }
        return m;
    }
    // Sums of e = 2^((x - ref) c) and of e (x - ref) c over the group, in two interleaved chains.  A logit of
    // -inf has e = 0 and would make 0 * -inf: CLAMP keeps the factor finite (below -1000 e is 0 already).
    template <bool CLAMP>
    __device__ __forceinline__ void sums(float ref, float c, float &s, float &t) const
    {
        const uint64_t c2 = f2_pack(c, c);
        uint64_t s2 = 0, t2 = 0;
#pragma unroll
        for (int i = 0; i < kSize / 2; ++i) {
            uint64_t d2 = f2_mul(less(i, ref), c2);
            const float2 d = f2_unpack(d2);
            const uint64_t e2 = f2_pack(ex2(d.x), ex2(d.y));
            if (CLAMP) d2 = f2_pack(fmaxf(d.x, -1000.0f), fmaxf(d.y, -1000.0f));
            s2 = f2_add(s2, e2);
            t2 = f2_fma(e2, d2, t2);
        }
        const float2 sv = f2_unpack(s2), tv = f2_unpack(t2);
        s = __fadd_rn(sv.x, sv.y);
        t = __fadd_rn(tv.x, tv.y);
    }
};

// Sums of s and of t over the warp in a fixed tree, both at once: s in lanes 0 .. 15, t in lanes 16 .. 31.
__device__ __forceinline__ float tl_warp_sums(float s, float t)
{
    const bool low = (threadIdx.x & 16) == 0;
    float v = __fadd_rn(low ? s : t, __shfl_xor_sync(0xffffffffu, low ? t : s, 16));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// A group's maximum as it is kept during the pass, in 16 bits: itself for bf16; for fp32 the next bf16 value at or
// above it, which selects the same groups and now and then one more.  (At 32 bits the maxima of 1024 rows of 151936
// fp32 left the L1 too little room for the loads in flight: 121.6 us with top 5, 104.4 with 16 bits.)
__device__ __forceinline__ uint16_t tl_keep(float m)
{
    const uint32_t u = __float_as_uint(m);
    return (uint16_t)((m != m ? 0x7fc00000u : u & 0x80000000u ? u : u + 0xffffu) >> 16);
}
__device__ __forceinline__ uint32_t tl_kept(uint16_t k) { return tl_order(__uint_as_float((uint32_t)k << 16)); }

template <bool BF16>
__device__ __forceinline__ float tl_element(const void *row, int e)
{
    if (BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(row)[e]);
    return static_cast<const float *>(row)[e];
}

constexpr int kTlColumns = 128;  // candidate threads, groups and elements of the short way
constexpr int kTlGroups = 128;
constexpr int kTlKeys = kTlMaxTop + kTlWarps * 32;
constexpr int kTlCrowd = (kTlMaxTop - 1) * kTlMaxPieces;  // groups above the k-th thread's best, at most

struct TlScratch {
    uint64_t keys[kTlKeys];
    uint16_t groups[kTlCrowd];  // numbers i: piece i / kTlThreads of the block, thread i % kTlThreads
    uint16_t columns[kTlColumns];
    uint32_t range[2][kTlWarps];
    int32_t n_columns, n_groups, n_keys;
};

// The block's `top` best keys, in order, to out[] (places without an element: 0).  tl_max holds its `local`
// pieces' group maxima, one column per thread; `mine` is the ordered largest of the thread's own (0: NaN or none).
//   1. A bound that at least `top` groups reach: bisection over the ordered values of the threads' best
//      groups, until few more than `top` threads reach it (or it is exact).
//   2. The groups of those threads that reach it are listed, read again, and their elements
//      that reach it listed: at least `top` elements do, so the best are among them.
//   3. An element's place is the number of larger keys.
// Where a list overflows (many equal values around the k-th, such as a mask's), the long way: with the bound
// exact, fewer than `top` threads have a group above it.  The elements above the bound are read from those groups (more
// than fit: each warp keeps a sorted list of its share), and one warp takes the first `top` elements that equal it, in
// index order.
template <bool BF16>
__device__ __forceinline__ void tl_best_groups(const TlParams &p, const void *row, int rank, int local,
                                               const uint16_t *tl_max, uint32_t mine, TlScratch &s, uint64_t *out)
{
    constexpr int kGroup = tl_group(BF16), kPiece = tl_piece(BF16);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto first = [&](int i) { return (i / kTlThreads * p.cluster + rank) * kPiece + kGroup * (i % kTlThreads); };
    const uint32_t top_of_warp = __reduce_max_sync(0xffffffffu, mine), low_of_warp = __reduce_min_sync(0xffffffffu, mine);
    if (lane == 0) {
        s.range[0][warp] = low_of_warp;
        s.range[1][warp] = top_of_warp;
    }
    for (int j = tid; j < kTlKeys; j += kTlThreads) s.keys[j] = 0;
    if (tid < kTlMaxTop) out[tid] = 0;
    if (tid == 0) s.n_columns = s.n_groups = s.n_keys = 0;
    __syncthreads();
    // Invariant: at least `top` threads reach lo (or lo is the least of all: every group is a candidate), fewer reach hi.
    uint32_t lo = s.range[0][0], hi = s.range[1][0];
#pragma unroll
    for (int w = 1; w < kTlWarps; ++w) {
        lo = min(lo, s.range[0][w]);
        hi = max(hi, s.range[1][w]);
    }
    ++hi;
    auto halve = [&](int enough) {
        while (hi - lo > 1) {
            const uint32_t mid = lo + (hi - lo) / 2;
            const int n = __syncthreads_count(mine >= mid);
            if (n >= p.top) lo = mid;
            else hi = mid;
            if (n >= p.top && n <= enough) break;
        }
    };
    // Thirty binary orders between the bests (or their signs) are most often a mask's doing: where fewer than `top` threads
    // are clear of it, it is the bound, which bisection would take 32 steps to find (one masked row of 50257 fp32, top 8:
    // 9.8 us without, 7.8 with; 11.2 before the long way's keys were counted).
    if (hi - lo > 30u << 23 && __syncthreads_count(mine > lo) < p.top) hi = lo + 1;
    halve(p.top + p.top / 2 + 6);
    if (mine >= lo) {
        const int at = atomicAdd(&s.n_columns, 1);
        if (at < kTlColumns) s.columns[at] = (uint16_t)tid;
    }
    __syncthreads();
    const int n_columns = s.n_columns;
    int n = kTlKeys + 1;  // keys listed; more than fit: the long way
    if (n_columns <= kTlColumns) {
        for (int j = tid; j < n_columns * local; j += kTlThreads) {
            const int i = j % local * kTlThreads + s.columns[j / local];
            if (tl_kept(tl_max[i]) >= lo && first(i) < p.V) {
                const int at = atomicAdd(&s.n_groups, 1);
                if (at < kTlGroups) s.groups[at] = (uint16_t)i;
            }
        }
        __syncthreads();
        const int n_groups = s.n_groups;
        if (n_groups <= kTlGroups) {
            constexpr int kBatch = 6;  // elements a thread has in flight
            for (int i0 = tid; i0 - tid < n_groups * kGroup; i0 += kBatch * kTlThreads) {
                float v[kBatch];
                int e[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int i = i0 + k * kTlThreads;
                    e[k] = i < n_groups * kGroup ? first(s.groups[i / kGroup]) + i % kGroup : p.V;
                    v[k] = e[k] < p.V ? tl_element<BF16>(row, e[k]) : 0.0f;
                }
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
                    if (e[k] < p.V && tl_order(v[k]) >= lo) {
                        const int at = atomicAdd(&s.n_keys, 1);
                        if (at < kTlKeys) s.keys[at] = tl_key(v[k], (uint32_t)e[k]);
                    }
            }
            __syncthreads();
            n = s.n_keys;
        }
    }
    if (n > kTlKeys) {
        halve(0);
        __syncthreads();
        if (tid == 0) s.n_groups = 0;
        __syncthreads();
        if (mine > lo)
            for (int i = tid; i < local * kTlThreads; i += kTlThreads)
                if (first(i) < p.V && tl_kept(tl_max[i]) > lo) s.groups[atomicAdd(&s.n_groups, 1)] = (uint16_t)i;
        __syncthreads();
        const int n_groups = s.n_groups;
        constexpr int kBatch = 4;  // groups a warp has in flight
        for (int j = tid; j < kTlKeys; j += kTlThreads) s.keys[j] = 0;
        if (tid == 0) s.n_keys = 0;
        __syncthreads();
        if (warp == 0) {
            int more = p.top;
            for (int i0 = 0; i0 < local * kTlThreads && more > 0; i0 += 32) {
                const int i = i0 + lane;
                unsigned reach = __ballot_sync(0xffffffffu, first(i) < p.V && tl_kept(tl_max[i]) >= lo);
                while (reach && more > 0) {
                    uint32_t o[kBatch];
                    int e[kBatch];
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        e[k] = reach && lane < kGroup ? first(i0 + __ffs(reach) - 1) + lane : p.V;
                        o[k] = e[k] < p.V ? tl_order(tl_element<BF16>(row, e[k])) : 0u;
                        reach &= reach - 1;
                    }
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        const unsigned same = __ballot_sync(0xffffffffu, e[k] < p.V && o[k] == lo);
                        const int at = p.top - more + __popc(same & ((1u << lane) - 1));
                        if ((same >> lane & 1u) && at < p.top) s.keys[at] = (uint64_t)lo << 32 | (uint32_t)~e[k];
                        more -= __popc(same);
                    }
                }
            }
        } else {
            // Above the bound: straight into the keys, as long as they fit.
            for (int g = warp - 1; g < n_groups; g += kTlWarps - 1) {
                const int e = lane < kGroup ? first(s.groups[g]) + lane : p.V;
                const float v = e < p.V ? tl_element<BF16>(row, e) : 0.0f;
                if (e < p.V && tl_order(v) > lo) {
                    const int at = kTlMaxTop + atomicAdd(&s.n_keys, 1);
                    if (at < kTlKeys) s.keys[at] = tl_key(v, (uint32_t)e);
                }
            }
        }
        __syncthreads();
        n = kTlMaxTop + s.n_keys;
        if (n > kTlKeys) {
            TlList list;
            for (int g0 = warp; g0 < n_groups; g0 += kBatch * kTlWarps) {
                float v[kBatch];
                int e[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int g = g0 + k * kTlWarps;
                    e[k] = g < n_groups && lane < kGroup ? first(s.groups[g]) + lane : p.V;
                    v[k] = e[k] < p.V ? tl_element<BF16>(row, e[k]) : 0.0f;
                }
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
                    list.offer(e[k] < p.V && tl_order(v[k]) > lo ? tl_key(v[k], (uint32_t)e[k]) : 0, p.top);
            }
            s.keys[kTlMaxTop + tid] = list.mine;
            __syncthreads();
            n = kTlKeys;
        }
    }
    for (int i = tid; i < n; i += kTlThreads) {
        const uint64_t key = s.keys[i];
        int place = 0;
        if (key != 0)
            for (int j = 0; j < n; j += 4)
#pragma unroll
                for (int k = 0; k < 4; ++k) place += s.keys[j + k] > key;  // 0 past the n-th
        if (key != 0 && place < p.top) out[place] = key;
    }
}

// Grid M * cluster blocks of kTlThreads; block r of a row's cluster takes pieces r, r + cluster, ...
// Dynamic shared memory: the block's group maxima, kTlThreads per piece (top > 0 only).
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kTlThreads, kTlBlocks) token_logprobs_kernel(const TlParams p)
{
    namespace cg = cooperative_groups;
    constexpr int kGroup = tl_group(BF16), kPiece = tl_piece(BF16);
    extern __shared__ uint16_t tl_max[];  // [pieces of this block][kTlThreads]
    __shared__ TlTriple triple[kTlMaxPieces * kTlWarps];
    __shared__ uint64_t best[kTlMaxCluster][kTlMaxTop];
    __shared__ TlScratch scratch;
    __shared__ float row_m, row_log_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)(blockIdx.x % (unsigned)p.cluster);
    const int64_t r = blockIdx.x / (unsigned)p.cluster;
    const void *row = static_cast<const uint8_t *>(p.x) + r * p.ldx * (BF16 ? 2 : 4);
    TlTriple *triples = triple;
    uint64_t(*bests)[kTlMaxTop] = best;
    if (p.cluster > 1) {
        triples = cg::this_cluster().map_shared_rank(triple, 0);
        bests = reinterpret_cast<uint64_t(*)[kTlMaxTop]>(cg::this_cluster().map_shared_rank(&best[0][0], 0));
        cluster_sync_all();  // every block of the cluster runs before its shared memory is written
    }
    griddep_wait();
    griddep_launch_dependents();

    // The scored logit is on its way while the row is read.
    int32_t tok = -1;
    float tok_x = 0.0f;
    if (rank == 0 && tid == 0 && p.logprobs != nullptr) {
        tok = p.tokens[r];
        if (tok >= 0 && tok < p.V) tok_x = tl_element<BF16>(row, tok);
    }
    TlGroup<BF16> g, next;
    int local = 0;
    bool masked = false;
    float thread_best = __int_as_float(0x7fffffff);  // NaN: none yet
    if (rank < p.pieces) g.template load<VEC>(row, rank * kPiece + kGroup * tid, p.V);
    for (int piece = rank; piece < p.pieces; piece += p.cluster, ++local) {
        const int ahead = piece + p.cluster;
        if (ahead < p.pieces) next.template load<VEC>(row, ahead * kPiece + kGroup * tid, p.V);
        const float gm = g.max(), m = warp_max(gm);
        if (p.top > 0) {
            tl_max[local * kTlThreads + tid] = tl_keep(gm);
            if (ahead < p.pieces) {
                thread_best = fmaxf(thread_best, gm);
            } else {
                // The row may end here.  The -inf past its end are no elements: a group that it cuts and that holds NaN
                // only does not reach -inf.
                const int left = p.V - (piece * kPiece + kGroup * tid);
                const float own = gm == kNegInf && left < kGroup && left > 0 ? g.max_below(left) : gm;
                if (left > 0) thread_best = fmaxf(thread_best, own);
            }
        }
        const float ref = m == kNegInf ? 0.0f : m;
        float s, t;
        if (!masked) {
            g.template sums<false>(ref, p.scale_log2, s, t);
            masked = __any_sync(0xffffffffu, t != t);  // a mask of -inf (or a NaN): once more, and from now on
        }
        if (masked) g.template sums<true>(ref, p.scale_log2, s, t);
        const float v = tl_warp_sums(s, t);
        TlTriple &to = triples[piece * kTlWarps + warp];
        if (lane == 0) {
            to.m = m;
            to.s = v;
        } else if (lane == 16) {
            to.t = v;
        }
        g = next;
    }
    __syncthreads();

    if (p.top > 0)
        tl_best_groups<BF16>(p, row, rank, local, tl_max, tl_order(thread_best), scratch, bests[rank]);
    if (p.cluster > 1) {
        cluster_sync_all();
        if (rank != 0) return;
    } else {
        __syncthreads();
    }

    // A key's place is the number of larger ones: its own list is in order (unused places hold 0), in every other
    // list it is searched for.
    constexpr int kLists = (kTlMaxCluster + kTlWarps - 1) / kTlWarps;  // of a warp
    uint64_t key[kLists];
    int place[kLists];
#pragma unroll
    for (int i = 0; i < kLists; ++i) {
        const int q = warp + i * kTlWarps;
        key[i] = q < p.cluster && lane < p.top ? best[q][lane] : 0;
        place[i] = lane;
        if (key[i] != 0)
#pragma unroll
            for (int o = 0; o < kTlMaxCluster; ++o)
                if (o < p.cluster && o != q) {
                    int n = 0;
#pragma unroll
                    for (int step = 16; step > 0; step >>= 1) n += best[o][n + step - 1] > key[i] ? step : 0;
                    place[i] += n + (best[o][n] > key[i]);
                }
    }
    if (warp == 0) {
        // Fold the triples: the maximum is exact in any order; lane j adds triples j, j + 32, ... in order.
        const int n = p.pieces * kTlWarps;
        float m = kNegInf;
        for (int i = lane; i < n; i += 32) m = fmaxf(m, triple[i].m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float ref = m == kNegInf ? 0.0f : m;
        float s = 0.0f, t = 0.0f;
        for (int i = lane; i < n; i += 32) {
            const TlTriple v = triple[i];
            // Against the row's maximum the triple's d all grow by d: S' = f S, T' = f (T + S d).  A triple without
            // finite elements has S = T = 0; where f is 0 its terms are.
            const float d = v.m == kNegInf ? 0.0f : __fmul_rn(v.m - ref, p.scale_log2), f = exp2f(d);
            s = __fadd_rn(s, __fmul_rn(f, v.s));
            t = __fadd_rn(t, f == 0.0f ? 0.0f : __fmul_rn(f, __fadd_rn(v.t, __fmul_rn(v.s, d))));
        }
        const float sums = tl_warp_sums(s, t);
        TlTriple a{m, __shfl_sync(0xffffffffu, sums, 0), __shfl_sync(0xffffffffu, sums, 16)};
        // A row without a finite maximum has no distribution: all its values are NaN.
        const float log_s = logf(a.s);
        if (lane == 0) {
            row_m = a.m;
            row_log_s = log_s;
            if (p.logprobs != nullptr) {
                float v = 0.0f;  // a negative token: the row is not scored
                if (tok >= p.V) {
                    record_error(p.status, 1);  // BI_ERR_INVALID_ARG
                    v = __int_as_float(0x7fffffff);
                } else if (tok >= 0) {
                    v = tl_logprob(tok_x, a.m, p.scale, log_s);
                }
                p.logprobs[r] = v;
            }
            if (p.entropy != nullptr) p.entropy[r] = __fsub_rn(log_s, __fmul_rn(0.693147180559945309f, a.t / a.s));
            if (p.logsumexp != nullptr) p.logsumexp[r] = __fmaf_rn(a.m, p.scale, log_s);
        }
    }
    if (p.top == 0) return;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kLists; ++i)
        if (key[i] != 0 && place[i] < p.top) {
            p.top_logprobs[r * p.top + place[i]] = tl_logprob(tl_value((uint32_t)(key[i] >> 32)), row_m, p.scale, row_log_s);
            p.top_tokens[r * p.top + place[i]] = (int32_t)~(uint32_t)key[i];
        }
}

}  // namespace bi
