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
// Bound by memory for many tokens and by latency for few.  A warp takes a token (or a share of its heads
// where there are few tokens): it works out the token's R/2 sines and cosines once, into its own piece of
// shared memory, and its lanes keep a fixed place in the head while they walk the heads.  A lane's unit
// is W entries a and their W partners b (16-byte pieces where sizes, strides and addresses allow it, single
// entries otherwise; the arithmetic is the same), and kRopeUnits heads' loads are in flight before
// the first angle is needed.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "rowops.cuh"

namespace bi {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRopeMaxDim = 1024;  // head size limit: kRopeWarps * D/2 cosines and sines are 32 KB
constexpr int kRopeUnits = 4;      // heads a lane has in flight

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

// A lane's place in the heads its warp walks.  A head has R/2W units of pairs and then (D - R)/W single
// pieces that are copied; 32 / units heads are taken at a time (or one head 32 units at a time).
template <int W, bool HALF>
struct RopeLane {
    int units, heads;  // units per head; heads the warp takes at a time
    int head, unit;    // this lane's first head and unit (unit >= units: the lane idles)
    __device__ __forceinline__ RopeLane(int D, int R)
    {
        const int lane = threadIdx.x & 31;
        units = R / (2 * W) + (D - R) / W;
        heads = units < 32 ? 32 / units : 1;
        head = units < 32 ? lane / units : 0;
        unit = lane - head * units;
        if (head >= heads) unit = units;
    }
    // Entry offsets of unit u's two pieces (b < 0: one piece, copied) and its first pair.
    static __device__ __forceinline__ void place(int u, int R, int &a, int &b, int &pair)
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

// The warp's token's cosines and sines into cs[R/2].
__device__ __forceinline__ void rope_angles(float2 *cs, const double *inv_freq, int half, int32_t pos, float scale, bool inverse)
{
    for (int i = threadIdx.x & 31; i < half; i += 32) cs[i] = rope_angle(pos, inv_freq[i], scale, inverse);
    __syncwarp();
}

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

// `shares` warps take a token's heads in turn.
template <typename E, int W, bool HALF>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p, int shares)
{
    extern __shared__ float2 rope_cs[];  // [kRopeWarps][R/2]
    const int half = p.R / 2;
    float2 *cs = rope_cs + (threadIdx.x >> 5) * half;
    const int64_t gw = (int64_t)blockIdx.x * kRopeWarps + (threadIdx.x >> 5), t = gw / shares;
    griddep_wait();
    griddep_launch_dependents();
    if (t >= p.T) return;
    const RopeLane<W, HALF> me(p.D, p.R);
    const int h_first = me.head + (int)(gw - t * shares) * me.heads, h_step = me.heads * shares;
    const E *x = static_cast<const E *>(p.x) + t * p.x_token;
    E *y = static_cast<E *>(p.y) + t * p.y_token;
    const bool in_place = p.x == p.y;
    bool ready = false;
    for (int u0 = 0; u0 < me.units; u0 += 32) {
        const int u = me.unit + u0;
        const bool on = u < me.units;
        int ea, eb, pair;
        RopeLane<W, HALF>::place(u, p.R, ea, eb, pair);
        for (int h0 = h_first; h0 - me.head < p.H; h0 += kRopeUnits * h_step) {
            Piece<E, W> a[kRopeUnits], b[kRopeUnits];
#pragma unroll
            for (int k = 0; k < kRopeUnits; ++k) {
                const int h = h0 + k * h_step;
                if (on && h < p.H) {
                    const E *src = x + h * p.x_head;
                    a[k] = *reinterpret_cast<const Piece<E, W> *>(src + ea);
                    if (eb >= 0) b[k] = *reinterpret_cast<const Piece<E, W> *>(src + eb);
                }
            }
            if (!ready) {  // the first loads are in flight
                if (half > 0) rope_angles(cs, p.inv_freq, half, p.pos[t], p.scale, p.inverse != 0);
                ready = true;
            }
            float2 c[W];
            if (on && eb >= 0)
#pragma unroll
                for (int j = 0; j < W; ++j) c[j] = cs[pair + j];
#pragma unroll
            for (int k = 0; k < kRopeUnits; ++k) {
                const int h = h0 + k * h_step;
                if (on && h < p.H) {
                    E *dst = y + h * p.y_head;
                    if (eb >= 0) {
                        rope_unit<E, W, HALF>(a[k], b[k], c);
                        *reinterpret_cast<Piece<E, W> *>(dst + eb) = b[k];
                    }
                    if (eb >= 0 || !in_place) *reinterpret_cast<Piece<E, W> *>(dst + ea) = a[k];
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

// `shares` warps take a token's query and key heads, and then its values, in turn.
template <int W, bool HALF>
__global__ void __launch_bounds__(kRopeThreads) paged_append_kernel(const AppendParams p, int shares)
{
    using E = __nv_bfloat16;
    extern __shared__ float2 rope_cs[];  // [kRopeWarps][R/2]
    const int half = p.R / 2, lane = threadIdx.x & 31;
    float2 *cs = rope_cs + (threadIdx.x >> 5) * half;
    const int64_t gw = (int64_t)blockIdx.x * kRopeWarps + (threadIdx.x >> 5), t = gw / shares;
    griddep_wait();
    griddep_launch_dependents();
    if (t >= p.T) return;
    const int share = (int)(gw - t * shares);
    const RopeLane<W, HALF> me(p.D, p.R);
    const int hq = p.q ? p.Hq : 0, H = hq + p.Hkv;  // heads 0 .. hq-1 query, then key
    const int h_first = me.head + share * me.heads, h_step = me.heads * shares;
    const E *q = p.q + t * p.q_token, *kk = p.k + t * p.k_token, *vv = p.v + t * p.v_token;
    E *qo = p.q_out + t * p.qo_token;
    AppendSlot slot{-1, 0};
    bool ready = false;
    for (int u0 = 0; u0 < me.units; u0 += 32) {
        const int u = me.unit + u0;
        const bool on = u < me.units;
        int ea, eb, pair;
        RopeLane<W, HALF>::place(u, p.R, ea, eb, pair);
        for (int h0 = h_first; h0 - me.head < H; h0 += kRopeUnits * h_step) {
            Piece<E, W> a[kRopeUnits], b[kRopeUnits];
#pragma unroll
            for (int k = 0; k < kRopeUnits; ++k) {
                const int h = h0 + k * h_step;
                if (on && h < H) {
                    const E *src = h < hq ? q + h * p.q_head : kk + (h - hq) * p.k_head;
                    a[k] = *reinterpret_cast<const Piece<E, W> *>(src + ea);
                    if (eb >= 0) b[k] = *reinterpret_cast<const Piece<E, W> *>(src + eb);
                }
            }
            if (!ready) {  // the first loads are in flight
                slot = append_slot(p, t);
                if (slot.cache < 0) return;
                if (half > 0) rope_angles(cs, p.inv_freq, half, slot.pos, p.scale, false);
                ready = true;
            }
            float2 c[W];
            if (on && eb >= 0)
#pragma unroll
                for (int j = 0; j < W; ++j) c[j] = cs[pair + j];
#pragma unroll
            for (int k = 0; k < kRopeUnits; ++k) {
                const int h = h0 + k * h_step;
                if (on && h < H) {
                    E *dst = h < hq ? qo + h * p.qo_head : p.k_cache + slot.cache + (h - hq) * p.c_head;
                    if (eb >= 0) {
                        rope_unit<E, W, HALF>(a[k], b[k], c);
                        *reinterpret_cast<Piece<E, W> *>(dst + eb) = b[k];
                    }
                    *reinterpret_cast<Piece<E, W> *>(dst + ea) = a[k];
                }
            }
        }
    }
    if (!ready) {  // a share without a head
        slot = append_slot(p, t);
        if (slot.cache < 0) return;
    }
    const int per_v = p.D / W, pieces = per_v * p.Hkv;
    for (int i0 = share * 32 + lane; i0 - lane < pieces; i0 += kRopeUnits * 32 * shares) {
        Piece<E, W> a[kRopeUnits];
#pragma unroll
        for (int k = 0; k < kRopeUnits; ++k) {
            const int i = i0 + k * 32 * shares, h = i / per_v;
            if (i < pieces) a[k] = *reinterpret_cast<const Piece<E, W> *>(vv + h * p.v_head + (i - h * per_v) * W);
        }
#pragma unroll
        for (int k = 0; k < kRopeUnits; ++k) {
            const int i = i0 + k * 32 * shares, h = i / per_v;
            if (i < pieces)
                *reinterpret_cast<Piece<E, W> *>(p.v_cache + slot.cache + h * p.c_head + (i - h * per_v) * W) = a[k];
        }
    }
}

}  // namespace bi
