// rope.cuh -- rotary positions, and appending keys and values to a paged cache with the rotation
// applied on the way.
//
// Entry pair (a, b) number i < R/2 of a head at position p becomes
//   (a cos t - b sin t, b cos t + a sin t),  t = p * inv_freq[i],
// times a scale; entries R .. D-1 are copied.  The angle is a product in fp64, reduced to a fraction
// of a turn before it is rounded to fp32 (an fp32 angle of 10^6 radians would be off by 0.06), and
// each output is one fp32 expression rounded once.  The work is elementwise, so every launch shape
// gives the same bits.
//
// Bound by memory for many tokens and by latency for few.  A block takes a few tokens, so that each
// token's R/2 sines and cosines are computed once and read from shared memory by every head.  A
// thread's unit is W entries a and their W partners b (16-byte pieces where sizes, strides and
// addresses allow it, single entries otherwise; the arithmetic is the same), and it has the first
// units' loads in flight before the angles are worked out.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "rowops.cuh"

namespace bi {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;    // tokens per block when there are many
constexpr int kRopeMaxDim = 1024; // head size limit: kRopeTokens * D/2 cosines and sines are 16 KB
constexpr int kRopeUnits = 4;     // units a thread has in flight

// W consecutive entries (16 bytes for W > 1) as they sit in memory.
template <typename E, int W>
struct alignas(W * sizeof(E)) Piece {
    E e[W];
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f32(float v, float &o) { o = v; }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16 &o) { o = __float2bfloat16_rn(v); }

// (cos, sin) of pos * inv_freq, times scale.
__device__ __forceinline__ float2 rope_angle(int32_t pos, double inv_freq, float scale, bool inverse)
{
    const double turns = (double)pos * (inv_freq * 0.15915494309189533576888);
    const float f = (float)(turns - rint(turns));  // in [-1/2, 1/2]
    float s, c;
    sincospif(2.0f * f, &s, &c);
    if (inverse) s = -s;
    return make_float2(__fmul_rn(c, scale), __fmul_rn(s, scale));
}

// Rotates the pairs of one unit.  HALF: a holds entries i .. i+W-1 and b their partners
// i + R/2 ..; otherwise a and b are 2W consecutive entries, pairs side by side.
template <typename E, int W, bool HALF>
__device__ __forceinline__ void rope_unit(Piece<E, W> &a, Piece<E, W> &b, const float2 *cs)
{
#pragma unroll
    for (int j = 0; j < W; ++j) {
        E *pa, *pb;
        if (HALF) {
            pa = &a.e[j];
            pb = &b.e[j];
        } else {
            pa = 2 * j < W ? &a.e[2 * j] : &b.e[2 * j - W];
            pb = 2 * j + 1 < W ? &a.e[2 * j + 1] : &b.e[2 * j + 1 - W];
        }
        const float x = to_f32(*pa), y = to_f32(*pb), c = cs[j].x, s = cs[j].y;
        from_f32(__fmaf_rn(x, c, -__fmul_rn(y, s)), *pa);
        from_f32(__fmaf_rn(y, c, __fmul_rn(x, s)), *pb);
    }
}

// Where a unit's entries sit in its head.  Units 0 .. R/2W-1 are pairs, the rest copies of one piece.
template <int W, bool HALF>
struct RopeUnit {
    int a, b;   // entry offsets of the two pieces (b < 0: one piece, copied)
    int pair;   // first pair number
    __device__ __forceinline__ RopeUnit(int u, int R)
    {
        const int np = R / (2 * W);
        if (u < np) {
            pair = u * W;
            a = HALF ? u * W : 2 * u * W;
            b = HALF ? R / 2 + u * W : a + W;
        } else {
            pair = 0;
            a = R + (u - np) * W;
            b = -1;
        }
    }
};

struct RopeParams {
    const void *x;
    void *y;
    int64_t x_token, x_head, y_token, y_head;  // strides in entries
    const int32_t *pos;
    const double *inv_freq;
    int64_t T;
    int32_t H, D, R;
    float scale;
    int32_t inverse;
};

template <typename E, int W, bool HALF>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p, int tokens)
{
    extern __shared__ float2 rope_cs[];  // [tokens][R/2]
    const int tid = threadIdx.x, half = p.R / 2;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int nt = (int)(p.T - t0 < tokens ? p.T - t0 : tokens);
    const int per_head = p.R / (2 * W) + (p.D - p.R) / W;
    const int per_token = per_head * p.H, units = per_token * nt;
    const E *x = static_cast<const E *>(p.x) + t0 * p.x_token;
    E *y = static_cast<E *>(p.y) + t0 * p.y_token;
    const bool in_place = p.x == p.y;
    griddep_wait();
    griddep_launch_dependents();

    Piece<E, W> a[kRopeUnits], b[kRopeUnits];
    for (int u0 = tid; u0 - tid < units; u0 += kRopeUnits * kRopeThreads) {
#pragma unroll
        for (int k = 0; k < kRopeUnits; ++k) {
            const int u = u0 + k * kRopeThreads;
            if (u < units) {
                const int t = u / per_token, r = u - t * per_token, h = r / per_head;
                const RopeUnit<W, HALF> w(r - h * per_head, p.R);
                const E *src = x + t * p.x_token + h * p.x_head;
                a[k] = *reinterpret_cast<const Piece<E, W> *>(src + w.a);
                if (w.b >= 0) b[k] = *reinterpret_cast<const Piece<E, W> *>(src + w.b);
            }
        }
        if (u0 == tid) {  // the first units' loads are in flight
            for (int i = tid; i < nt * half; i += kRopeThreads) {
                const int t = i / half;
                rope_cs[i] = rope_angle(p.pos[t0 + t], p.inv_freq[i - t * half], p.scale, p.inverse != 0);
            }
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < kRopeUnits; ++k) {
            const int u = u0 + k * kRopeThreads;
            if (u < units) {
                const int t = u / per_token, r = u - t * per_token, h = r / per_head;
                const RopeUnit<W, HALF> w(r - h * per_head, p.R);
                E *dst = y + t * p.y_token + h * p.y_head;
                if (w.b >= 0) {
                    rope_unit<E, W, HALF>(a[k], b[k], rope_cs + t * half + w.pair);
                    *reinterpret_cast<Piece<E, W> *>(dst + w.a) = a[k];
                    *reinterpret_cast<Piece<E, W> *>(dst + w.b) = b[k];
                } else if (!in_place) {
                    *reinterpret_cast<Piece<E, W> *>(dst + w.a) = a[k];
                }
            }
        }
    }
}

// ------------------------------------------------------------------------------- paged append

// Number of entries of the ascending v[0 .. n) that are <= t, by a warp: 32 probes a step.  For any
// contents of v the result is in 0 .. n.
__device__ __forceinline__ int warp_count_le(const int32_t *v, int n, int t)
{
    const int lane = threadIdx.x & 31;
    int lo = 0;
    while (n > 0) {
        const int step = (n + 31) / 32, last = (lane + 1) * step - 1;
        const bool le = last < n && v[lo + last] <= t;
        const int full = __popc(__ballot_sync(0xffffffffu, le));
        lo += full * step;
        if (step == 1) break;
        n = n - full * step < step ? n - full * step : step;
    }
    return lo;
}

struct AppendParams {
    const __nv_bfloat16 *k, *v, *q;  // q may be null
    __nv_bfloat16 *q_out, *k_cache, *v_cache;
    int64_t k_token, k_head, v_token, v_head, q_token, q_head, qo_token, qo_head;
    int64_t c_page, c_token, c_head;  // cache strides
    const int32_t *table;             // [B, max_pages], rows table_row apart
    int64_t table_row;
    const int32_t *lens;       // [B] lengths with the new tokens
    const int32_t *cu;         // [B+1] first new token of each sequence, or null: one each
    const int32_t *positions;  // [T] or null: the place in the sequence
    const double *inv_freq;    // null when R = 0
    int64_t T, pages;
    int32_t B, Hq, Hkv, D, R, page_size, max_pages;
    float scale;
    int32_t *status;
};

// Where one new token goes.
struct AppendSlot {
    int64_t cache;  // offset of its row in the cache (head 0), or -1: the token is skipped
    int32_t pos;    // position that turns it
};

// One warp works out token t's slot.
__device__ __forceinline__ AppendSlot append_slot(const AppendParams &p, int64_t t)
{
    int b = (int)t, left = 1;  // tokens of the sequence from t on
    if (p.cu != nullptr) {
        b = warp_count_le(p.cu, p.B + 1, (int)t) - 1;
        if (b < 0 || b >= p.B) return {-1, 0};  // before the first sequence or behind the last: not ours
        left = p.cu[b + 1] - (int)t;
    }
    const int32_t len = p.lens[b];
    if (len == 0) return {-1, 0};  // an empty place of a padded batch
    const int64_t at = (int64_t)len - left;
    int32_t page = -1;
    if (left >= 1 && at >= 0 && at / p.page_size < p.max_pages) page = p.table[b * p.table_row + at / p.page_size];
    if (page < 0 || page >= p.pages) {
        *reinterpret_cast<volatile int32_t *>(p.status) = 1;  // BI_ERR_INVALID_ARG
        return {-1, 0};
    }
    return {page * p.c_page + (at % p.page_size) * p.c_token, p.positions ? p.positions[t] : (int32_t)at};
}

template <int W, bool HALF>
__global__ void __launch_bounds__(kRopeThreads) paged_append_kernel(const AppendParams p, int tokens)
{
    using E = __nv_bfloat16;
    extern __shared__ float2 rope_cs[];  // [tokens][R/2]
    __shared__ AppendSlot slot[kRopeTokens];
    const int tid = threadIdx.x, half = p.R / 2;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int nt = (int)(p.T - t0 < tokens ? p.T - t0 : tokens);
    const int per_head = p.R / (2 * W) + (p.D - p.R) / W, per_v = p.D / W;
    const int hq = p.q ? p.Hq : 0, turned = per_head * (hq + p.Hkv);
    const int per_token = turned + per_v * p.Hkv, units = per_token * nt;
    griddep_wait();
    griddep_launch_dependents();

    // Unit u: a piece (or pair of pieces) of a query head, a key head or a value head of token t.
    struct At {
        int t, head, a, b, pair;
        int kind;  // 0 query, 1 key, 2 value
    };
    auto locate = [&](int u) -> At {
        const int t = u / per_token, r = u - t * per_token;
        if (r >= turned) {
            const int w = r - turned, h = w / per_v;
            return {t, h, (w - h * per_v) * W, -1, 0, 2};
        }
        const int h = r / per_head;
        const RopeUnit<W, HALF> w(r - h * per_head, p.R);
        return {t, h < hq ? h : h - hq, w.a, w.b, w.pair, h < hq ? 0 : 1};
    };

    Piece<E, W> a[kRopeUnits], b[kRopeUnits];
    for (int u0 = tid; u0 - tid < units; u0 += kRopeUnits * kRopeThreads) {
#pragma unroll
        for (int k = 0; k < kRopeUnits; ++k) {
            const int u = u0 + k * kRopeThreads;
            if (u < units) {
                const At w = locate(u);
                const int64_t t = t0 + w.t;
                const E *src = w.kind == 0   ? p.q + t * p.q_token + w.head * p.q_head
                               : w.kind == 1 ? p.k + t * p.k_token + w.head * p.k_head
                                             : p.v + t * p.v_token + w.head * p.v_head;
                a[k] = *reinterpret_cast<const Piece<E, W> *>(src + w.a);
                if (w.b >= 0) b[k] = *reinterpret_cast<const Piece<E, W> *>(src + w.b);
            }
        }
        if (u0 == tid) {  // the first units' loads are in flight
            if ((tid >> 5) < nt) {
                const AppendSlot s = append_slot(p, t0 + (tid >> 5));
                if ((tid & 31) == 0) slot[tid >> 5] = s;
            }
            __syncthreads();
            for (int i = tid; i < nt * half; i += kRopeThreads) {
                const int t = i / half;
                rope_cs[i] = rope_angle(slot[t].pos, p.inv_freq[i - t * half], p.scale, false);
            }
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < kRopeUnits; ++k) {
            const int u = u0 + k * kRopeThreads;
            if (u < units) {
                const At w = locate(u);
                const int64_t t = t0 + w.t, row = slot[w.t].cache;
                if (row < 0) continue;
                E *dst = w.kind == 0   ? p.q_out + t * p.qo_token + w.head * p.qo_head
                         : w.kind == 1 ? p.k_cache + row + w.head * p.c_head
                                       : p.v_cache + row + w.head * p.c_head;
                if (w.b >= 0) {
                    rope_unit<E, W, HALF>(a[k], b[k], rope_cs + w.t * half + w.pair);
                    *reinterpret_cast<Piece<E, W> *>(dst + w.b) = b[k];
                }
                *reinterpret_cast<Piece<E, W> *>(dst + w.a) = a[k];
            }
        }
    }
}

}  // namespace bi
