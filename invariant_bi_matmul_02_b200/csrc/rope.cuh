// rope.cuh -- rotary positions, and appending keys and values to a paged cache with the rotation
// applied on the way.
//
// Entry pair (a, b) number i < R/2 of a head at position p becomes
//   (a cos t - b sin t, b cos t + a sin t),  t = p * inv_freq[i],
// times a scale; entries R .. D-1 are copied.  The angle is a product in fp64, reduced to a fraction
// of a turn before it is rounded to fp32 (an fp32 angle of 10^6 radians would be off by 0.06), what that rounding leaves
// out is put back to first order, and each output is one fp32 expression rounded once.  The work is elementwise, so every launch shape
// gives the same bits.
//
// Bound by memory for many tokens (B200: 40 heads of 128 of 8192 tokens, bf16, 28.9 us or 5.8 TB/s; 9734 tokens
// appended with 32 query and 8 key and value heads 42.5 us, 5.6 TB/s) and by latency for few (one token 2.1 us, 64
// appended 3.8).  A warp takes a token (or a share of its heads where there are few tokens): it works out the token's R/2
// sines and cosines once, into its own piece of shared memory, and its lanes keep a fixed place in the head while
// they walk the heads.  A lane's unit is W entries a and their W partners b (16-byte pieces where sizes, strides and
// addresses allow it, else two entries or one; the arithmetic is the same).
// Walks of 16-byte pieces are streamed: copies to shared memory bring up to kRopeStages steps of the queries, the keys
// and the values at once, with entries that are only copied as units of their own, so that most of a token's 10 KB is
// on its way while the angles are worked out (with two steps in registers instead: 31.2 and 45.8 us).  Heads of
// 16-byte pieces that the pairs do not fill are turned in shared memory (rope_staged_kernel).  Else narrower pieces go
// through registers, and the entries that are only copied go apart, in the widest pieces that they allow.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "rowops.cuh"

namespace bi {

constexpr int kRopeThreads = 128;
constexpr int kRopeBlocks = 7;  // resident per SM, a bound on registers (4096 x 40 x 128: 17.5 us with 6, 15.5 with 7)
constexpr int kRopeStagedBlocks = 10;  // the same of the staged walk, as its 44 registers allow (9 for the append's 56)
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRopeMaxDim = 1024;  // head size limit: kRopeWarps * D/2 cosines and sines are 16 KB
constexpr int kRopeCopies = 4;     // value pieces a lane has in flight

// W consecutive entries as they sit in memory: 16 bytes, two entries or one.
template <typename E, int W>
struct alignas(16) Piece {
    uint32_t w[4];
};
template <typename E>
struct Piece<E, 1> {
    E e;
};
template <typename E>
struct alignas(2 * sizeof(E)) Piece<E, 2> {
    E e[2];
};

// Buffers of a lane that walks through registers: one head is turned while the others are on their way.  More for
// smaller pieces, as registers allow (8284 tokens of 19 heads of 192, 74 bf16 entries turned one by one: 88.8 us with 2,
// 57.7 with 6; 20 by twos: 37.8 with 2, 35.2 with 4; both before kRopeBlocks was 7, 46.5 and 30.8 since).
template <typename E, int W>
__host__ __device__ constexpr int rope_buffers()
{
    return W == 1 ? 6 : W == 2 ? 4 : 2;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f32(float v, float &o) { o = v; }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16 &o) { o = __float2bfloat16_rn(v); }

// Cosine and sine of pos * inv_freq, times scale.
__device__ __forceinline__ void rope_angle(int32_t pos, double inv_freq, float scale, bool inverse, float &c, float &s)
{
    const double turns = (double)pos * (inv_freq * 0.15915494309189533576888);
    const double part = turns - rint(turns);  // in [-1/2, 1/2]
    const float f = (float)part, r = 6.2831853f * (float)(part - (double)f);
    float c0, s0;
    sincospif(2.0f * f, &s0, &c0);
    // The angle that the rounding of f left out, at most 2^-23.3 radians: its square is below any bit.
    c = __fmaf_rn(-r, s0, c0);
    s = __fmaf_rn(r, c0, s0);
    if (inverse) s = -s;
    c = __fmul_rn(c, scale);
    s = __fmul_rn(s, scale);
}

// The cosines and sines of a unit's W pairs.
template <int W>
struct RopeTurn {
    float c[W], s[W];
    __device__ __forceinline__ void load(const float *cs, int half, int pair)
    {
#pragma unroll
        for (int j = 0; j < W; ++j) {
            c[j] = cs[pair + j];
            s[j] = cs[half + pair + j];
        }
    }
    // The first half of the pairs from `pair` on, the second from `pair2` on.
    __device__ __forceinline__ void load2(const float *cs, int half, int pair, int pair2)
    {
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const int at = j < W / 2 ? pair + j : pair2 + j - W / 2;
            c[j] = cs[at];
            s[j] = cs[half + at];
        }
    }
    // Pairs j and j + 1: (x, y) to (x c - y s, y c + x s), each one product and one fused sum.
    __device__ __forceinline__ void turn2(int j, uint64_t &x, uint64_t &y) const
    {
        const uint64_t c2 = f2_pack(c[j], c[j + 1]);
        const uint64_t s2 = f2_pack(s[j], s[j + 1]), u = f2_fma(x, c2, f2_mul(y, s2) ^ 0x8000000080000000ull);
        y = f2_fma(y, c2, f2_mul(x, s2));
        x = u;
    }
};

// Rotates the W pairs of one unit in place.  HALF: a holds entries i .. i+W-1 and b their partners i + R/2 ..;
// otherwise a and b are 2W consecutive entries, pairs side by side.
template <typename E, int W, bool HALF>
__device__ __forceinline__ void rope_unit(Piece<E, W> &a, Piece<E, W> &b, const RopeTurn<W> &t)
{
    if constexpr (W == 1) {
        const float x = to_f32(a.e), y = to_f32(b.e);
        from_f32(__fmaf_rn(x, t.c[0], -__fmul_rn(y, t.s[0])), a.e);
        from_f32(__fmaf_rn(y, t.c[0], __fmul_rn(x, t.s[0])), b.e);
    } else if constexpr (W == 2) {
        E &x0 = a.e[0], &x1 = HALF ? a.e[1] : b.e[0], &y0 = HALF ? b.e[0] : a.e[1], &y1 = b.e[1];
        uint64_t x = f2_pack(to_f32(x0), to_f32(x1)), y = f2_pack(to_f32(y0), to_f32(y1));
        t.turn2(0, x, y);
        const float2 u = f2_unpack(x), v = f2_unpack(y);
        from_f32(u.x, x0);
        from_f32(u.y, x1);
        from_f32(v.x, y0);
        from_f32(v.y, y1);
    } else if constexpr (W == 8 && HALF) {  // bf16: a word holds entries 2j and 2j + 1
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint64_t x = f2_pack(bf16lo(a.w[j]), bf16hi(a.w[j])), y = f2_pack(bf16lo(b.w[j]), bf16hi(b.w[j]));
            t.turn2(2 * j, x, y);
            const float2 u = f2_unpack(x), v = f2_unpack(y);
            a.w[j] = pack_bf16x2(u.x, u.y);
            b.w[j] = pack_bf16x2(v.x, v.y);
        }
    } else if constexpr (W == 8) {  // bf16: a word holds a pair
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            uint32_t &w0 = j < 4 ? a.w[j] : b.w[j - 4], &w1 = j < 4 ? a.w[j + 1] : b.w[j - 3];
            uint64_t x = f2_pack(bf16lo(w0), bf16lo(w1)), y = f2_pack(bf16hi(w0), bf16hi(w1));
            t.turn2(j, x, y);
            const float2 u = f2_unpack(x), v = f2_unpack(y);
            w0 = pack_bf16x2(u.x, v.x);
            w1 = pack_bf16x2(u.y, v.y);
        }
    } else {  // fp32: four entries a piece
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            uint32_t &x0 = HALF ? a.w[j] : j == 0 ? a.w[0] : b.w[0], &x1 = HALF ? a.w[j + 1] : j == 0 ? a.w[2] : b.w[2];
            uint32_t &y0 = HALF ? b.w[j] : j == 0 ? a.w[1] : b.w[1], &y1 = HALF ? b.w[j + 1] : j == 0 ? a.w[3] : b.w[3];
            uint64_t x = f2_pack(__uint_as_float(x0), __uint_as_float(x1)), y = f2_pack(__uint_as_float(y0), __uint_as_float(y1));
            t.turn2(j, x, y);
            const float2 u = f2_unpack(x), v = f2_unpack(y);
            x0 = __float_as_uint(u.x);
            x1 = __float_as_uint(u.y);
            y0 = __float_as_uint(v.x);
            y1 = __float_as_uint(v.y);
        }
    }
}

// A lane's place in the heads its warp walks: a head has R/2W units; 32 / units heads are taken at a time (or one
// head 32 units at a time).
template <int W>
struct RopeLane {
    int units, heads;  // units per head; heads the warp takes at a time
    int head, unit;    // this lane's first head and unit (unit >= units: the lane idles)
    __device__ __forceinline__ explicit RopeLane(int R)
    {
        const int lane = threadIdx.x & 31;
        units = R / (2 * W);
        heads = units > 0 && units < 32 ? 32 / units : 1;
        head = units > 0 && units < 32 ? lane / units : 0;
        unit = lane - head * units;
        if (head >= heads) unit = units;
    }
};

// Steps of a warp that a streamed walk has on their way at once (8192 x 40 x 128: 29.3 us with 4, 28.9 with 6; 8 and 10
// leave room for fewer warps: 29.3, 30.6).
constexpr int kRopeStages = 6;

// One of a token's tensors (queries, keys or values) in a streamed walk: H heads, src_head and dst_head entries apart.
template <typename E>
struct RopeStretch {
    const E *src;
    int64_t src_head, dst_head;
    int H;
};

// How a streamed walk splits a head and a token: units of 2W entries, the first R/2W turned and the others copied;
// 32 / units heads to a step (or one head, 32 units at a time); steps numbered through the N stretches.
template <int W>
struct RopeSteps {
    int units, heads;
    __host__ __device__ RopeSteps(int R, int rest) : units(R / (2 * W) + (rest + 2 * W - 1) / (2 * W))
    {
        heads = units > 0 && units < 32 ? 32 / units : 1;
    }
    __host__ __device__ int steps(int H) const { return units > 0 ? (H + heads - 1) / heads : 0; }
};

// Turns (stretches below `turned`) or copies the heads of one token's N stretches, every `shares`-th step from
// `share` on.  rest: entries R .. R + rest - 1 of each head are copied.  ring: `stages` steps of the warp, each 64
// pieces; as many as it takes, or kRopeStages if those are fewer.  ready() is called once the first loads are
// in flight and before cs or dst(i), stretch i's place, is needed; false ends the walk.
template <typename E, int W, bool HALF, int N, typename Ready, typename Dst>
__device__ __forceinline__ bool rope_stream(const RopeStretch<E> (&st)[N], int turned, int R, int rest, int share,
                                            int shares, uint4 *ring, int stages, const float *cs, Ready ready, Dst dst)
{
    const RopeSteps<W> shape(R, rest);
    const int lane = threadIdx.x & 31, half = R / 2, turning = R / (2 * W);
    int first[N + 1];  // first step of each stretch
    first[0] = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) first[i + 1] = first[i] + shape.steps(st[i].H);
    if (share >= first[N]) return true;
    const int mine = (first[N] - share + shares - 1) / shares;
    for (int u0 = 0; u0 < shape.units; u0 += 32) {
        const int my_head = shape.units < 32 ? lane / shape.units : 0, u = u0 + lane - my_head * shape.units;
        const bool on = my_head < shape.heads && u < shape.units, turns = u < turning;
        // Either layout's piece a is in the first half of the turned (or copied) entries and b in the second, so that
        // neighbouring lanes have neighbouring pieces.
        const int ea = turns ? u * W : R + (u - turning) * W, eb = ea + (turns ? half : (shape.units - turning) * W);
        const bool has_b = turns || eb < R + rest;
        // Stretch and head that step j of this warp gives the lane; head >= H: none.
        auto place = [&](int j, int &i, int &h) {
            const int g = share + j * shares;
            i = 0;
            int base = 0;
#pragma unroll
            for (int k = 1; k < N; ++k)
                if (g >= first[k]) {
                    i = k;
                    base = first[k];
                }
            h = my_head + (g - base) * shape.heads;
        };
        auto pick = [&](int i) {  // st[i] without an indexed array
            RopeStretch<E> v = st[0];
#pragma unroll
            for (int k = 1; k < N; ++k)
                if (i == k) v = st[k];
            return v;
        };
        auto load = [&](int j, int slot) {
            int i, h;
            place(j, i, h);
            const RopeStretch<E> v = pick(i);
            if (on && h < v.H) {
                const E *from = v.src + h * v.src_head;
                cp_async16(ring + slot * 64 + lane, from + ea, 16);
                if (has_b) cp_async16(ring + slot * 64 + 32 + lane, from + eb, 16);
            }
        };
#pragma unroll 1
        for (int k = 0; k < stages && k < mine; ++k) {
            load(k, k);
            cp_async_commit();
        }
        if (!ready()) {
            cp_async_wait_all();
            return false;
        }
        RopeTurn<W> turn;
        if (on && turns) HALF ? turn.load(cs, half, u * W) : turn.load2(cs, half, u * (W / 2), (half + u * W) / 2);
        int slot = 0;
#pragma unroll 1
        for (int j = 0; j < mine; ++j) {
            // Steps j .. min(j + stages, mine) - 1 are on their way.
            const int left = mine - j;
            if (left >= kRopeStages)
                cp_async_wait_pending<kRopeStages - 1>();
            else if (left >= kRopeStages / 2)
                cp_async_wait_pending<kRopeStages / 2 - 1>();
            else
                cp_async_wait_pending<0>();
            Piece<E, W> a, b;
            *reinterpret_cast<uint4 *>(&a) = ring[slot * 64 + lane];
            *reinterpret_cast<uint4 *>(&b) = ring[slot * 64 + 32 + lane];
            if (j + stages < mine) {
                load(j + stages, slot);
                cp_async_commit();
            }
            slot = slot + 1 == stages ? 0 : slot + 1;
            int i, h;
            place(j, i, h);
            const RopeStretch<E> v = pick(i);
            if (on && h < v.H) {
                if (turns && i < turned) rope_unit<E, W, HALF>(a, b, turn);
                E *to = dst(i) + h * v.dst_head;
                *reinterpret_cast<Piece<E, W> *>(to + ea) = a;
                if (has_b) *reinterpret_cast<Piece<E, W> *>(to + eb) = b;
            }
        }
    }
    return true;
}

// The same for heads of 16-byte pieces that their pairs do not fill (R/2 is not a multiple of a piece's entries): the
// first `pieces` pieces of a head (64 at most) are streamed as they lie, 64 / pieces heads to a step, and the pairs
// turned in shared memory one by one, across the lanes, before the pieces go out.
// (8284 tokens of 19 heads of 192 bf16 with 74 entries turned: 26.8 us, 46.7 when lanes read and wrote single entries; of
// 2 heads of 256, 254 turned: 9.5 and 15.9; 32 heads of 80, 20 turned: one token 2.4 and 2.7, 2048 5.6 and 6.2; 64
// sequences' tokens appended with 32 query and 32 key and value heads of 80, 20 turned: 3.4 and 5.7.)
template <typename E, bool HALF, int N, typename Ready, typename Dst>
__device__ __forceinline__ bool rope_staged(const RopeStretch<E> (&st)[N], int turned, int R, int pieces, int share, int shares,
                                            uint4 *ring, int stages, const float *cs, Ready ready, Dst dst)
{
    constexpr int W = 16 / (int)sizeof(E);
    const int lane = threadIdx.x & 31, half = R / 2, heads = 64 / pieces;
    int first[N + 1];  // first step of each stretch
    first[0] = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) first[i + 1] = first[i] + (st[i].H + heads - 1) / heads;
    if (share >= first[N]) return true;
    const int mine = (first[N] - share + shares - 1) / shares;
    int head[2], entry[2];  // of this lane's two pieces in a step
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int i = lane + 32 * k;
        head[k] = i / pieces;
        entry[k] = (i - head[k] * pieces) * W;
    }
    // Stretch of step j of this warp and its first head there.
    auto place = [&](int j, int &h0) {
        const int g = share + j * shares;
        int i = 0, base = 0;
#pragma unroll
        for (int k = 1; k < N; ++k)
            if (g >= first[k]) {
                i = k;
                base = first[k];
            }
        h0 = (g - base) * heads;
        return i;
    };
    auto pick = [&](int i) {  // st[i] without an indexed array
        RopeStretch<E> v = st[0];
#pragma unroll
        for (int k = 1; k < N; ++k)
            if (i == k) v = st[k];
        return v;
    };
    auto load = [&](int j, int slot) {
        int h0;
        const RopeStretch<E> v = pick(place(j, h0));
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (head[k] < heads && h0 + head[k] < v.H)
                cp_async16(ring + slot * 64 + lane + 32 * k, v.src + (h0 + head[k]) * v.src_head + entry[k], 16);
    };
#pragma unroll 1
    for (int k = 0; k < stages && k < mine; ++k) {
        load(k, k);
        cp_async_commit();
    }
    if (!ready()) {
        cp_async_wait_all();
        return false;
    }
    const float per_half = 1.0f / (float)half;
    int slot = 0;
#pragma unroll 1
    for (int j = 0; j < mine; ++j) {
        const int left = mine - j;  // as in rope_stream
        if (left >= kRopeStages)
            cp_async_wait_pending<kRopeStages - 1>();
        else if (left >= kRopeStages / 2)
            cp_async_wait_pending<kRopeStages / 2 - 1>();
        else
            cp_async_wait_pending<0>();
        __syncwarp();
        int h0;
        const int which = place(j, h0);
        const RopeStretch<E> v = pick(which);
        if (which < turned) {
            const int pairs = min(heads, v.H - h0) * half;
            E *at = reinterpret_cast<E *>(ring + slot * 64);
            for (int i = lane; i < pairs; i += 32) {
                const int h = (int)(((float)i + 0.5f) * per_half), k = i - h * half;  // i < 2^8: exact
                E *a = at + h * pieces * W + (HALF ? k : 2 * k), *b = a + (HALF ? half : 1);
                const float u = to_f32(*a), w = to_f32(*b), c = cs[k], s = cs[half + k];
                from_f32(__fmaf_rn(u, c, -__fmul_rn(w, s)), *a);
                from_f32(__fmaf_rn(w, c, __fmul_rn(u, s)), *b);
            }
            __syncwarp();
        }
        E *to = dst(which);
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (head[k] < heads && h0 + head[k] < v.H)
                *reinterpret_cast<uint4 *>(to + (h0 + head[k]) * v.dst_head + entry[k]) = ring[slot * 64 + lane + 32 * k];
        if (j + stages < mine) {
            load(j + stages, slot);
            cp_async_commit();
        }
        slot = slot + 1 == stages ? 0 : slot + 1;
    }
    return true;
}

// The warp's token's R/2 cosines, then R/2 sines, into cs.
__device__ __forceinline__ void rope_angles(float *cs, const double *inv_freq, int half, int32_t pos, float scale, bool inverse)
{
    for (int i = threadIdx.x & 31; i < half; i += 32) rope_angle(pos, inv_freq[i], scale, inverse, cs[i], cs[half + i]);
    __syncwarp();
}

// Turns heads 0 .. H-1 of one token, every `shares`-th group of them from group `group` on: src to the
// place that dst() gives.  ready() is called once the first loads are in flight and before cs or dst() is
// needed; false ends the walk.
template <typename E, int W, bool HALF, typename Ready, typename Dst>
__device__ __forceinline__ bool rope_walk(const RopeLane<W> &me, const E *src, int64_t src_head, int64_t dst_head, int H,
                                          int R, int group, int shares, const float *cs, Ready ready, Dst dst)
{
    const int h_step = me.heads * shares, half = R / 2;
    const int64_t src_step = h_step * src_head, dst_step = h_step * dst_head;
    for (int u0 = 0; u0 < me.units; u0 += 32) {
        const int u = me.unit + u0;
        const int ea = HALF ? u * W : 2 * u * W, eb = HALF ? half + u * W : ea + W;
        // Heads left for this lane, and for the warp's first lane (the loop's bound).
        const int h = me.head + group * me.heads;
        int left = u < me.units && h < H ? (H - h + h_step - 1) / h_step : 0;
        int turns = group * me.heads < H ? (H - group * me.heads + h_step - 1) / h_step : 0;
        if (turns == 0) continue;
        const E *from = src + h * src_head;
        constexpr int kBuffers = rope_buffers<E, W>();
        Piece<E, W> a[kBuffers], b[kBuffers];
        auto load = [&](int k, bool some) {
            if (some) {
                a[k] = *reinterpret_cast<const Piece<E, W> *>(from + ea);
                b[k] = *reinterpret_cast<const Piece<E, W> *>(from + eb);
            }
            from += src_step;
        };
#pragma unroll
        for (int k = 0; k + 1 < kBuffers; ++k) load(k, left > k);
        if (!ready()) return false;
        RopeTurn<W> turn;
        if (u < me.units) turn.load(cs, half, u * W);
        E *to = dst() + h * dst_head;
        while (turns > 0) {
#pragma unroll
            for (int k = 0; k < kBuffers; ++k) {
                load((k + kBuffers - 1) % kBuffers, left > kBuffers - 1);
                if (left > 0) {
                    rope_unit<E, W, HALF>(a[k], b[k], turn);
                    *reinterpret_cast<Piece<E, W> *>(to + ea) = a[k];
                    *reinterpret_cast<Piece<E, W> *>(to + eb) = b[k];
                }
                to += dst_step;
                --left;
                if (--turns == 0) break;
            }
        }
    }
    return true;
}

// Copies `bytes` bytes of each of H heads (strides in bytes) by pieces of type P, every `shares`-th 32 pieces from
// share `share` on.  ready() as in rope_walk.
template <typename P, typename Ready, typename Dst>
__device__ __forceinline__ bool copy_pieces(const uint8_t *src, int64_t src_head, int64_t dst_head, int H, int bytes,
                                            int share, int shares, Ready ready, Dst dst)
{
    const int per_head = bytes / (int)sizeof(P), pieces = per_head * H, lane = threadIdx.x & 31;
    for (int i0 = share * 32 + lane; i0 - lane < pieces; i0 += kRopeCopies * 32 * shares) {
        P a[kRopeCopies];
#pragma unroll
        for (int k = 0; k < kRopeCopies; ++k) {
            const int i = i0 + k * 32 * shares, h = i / per_head;
            if (i < pieces) a[k] = *reinterpret_cast<const P *>(src + h * src_head + (i - h * per_head) * (int)sizeof(P));
        }
        if (!ready()) return false;
        uint8_t *to = dst();
#pragma unroll
        for (int k = 0; k < kRopeCopies; ++k) {
            const int i = i0 + k * 32 * shares, h = i / per_head;
            if (i < pieces) *reinterpret_cast<P *>(to + h * dst_head + (i - h * per_head) * (int)sizeof(P)) = a[k];
        }
    }
    return true;
}

// The same with pieces of `piece` bytes (16, 8, 4 or 2), which the host has found to fit.
template <typename Ready, typename Dst>
__device__ __forceinline__ bool copy_heads(int piece, const void *src, int64_t src_head, int64_t dst_head, int H, int bytes,
                                           int share, int shares, Ready ready, Dst dst)
{
    const uint8_t *from = static_cast<const uint8_t *>(src);
    switch (piece) {
    case 16: return copy_pieces<uint4>(from, src_head, dst_head, H, bytes, share, shares, ready, dst);
    case 8: return copy_pieces<uint2>(from, src_head, dst_head, H, bytes, share, shares, ready, dst);
    case 4: return copy_pieces<uint32_t>(from, src_head, dst_head, H, bytes, share, shares, ready, dst);
    default: return copy_pieces<uint16_t>(from, src_head, dst_head, H, bytes, share, shares, ready, dst);
    }
}

struct RopeParams {
    const void *x;
    void *y;
    int64_t x_token, x_head, y_token, y_head;  // strides in entries
    const int32_t *pos;  // pos and inv_freq may be null when R = 0
    const double *inv_freq;
    int64_t T;
    int32_t H, D, R;
    float scale;
    int32_t inverse;
    int32_t copy_piece;  // bytes; 0: entries R .. D-1 are not copied (none, or y is x)
    int32_t pieces;      // rope_staged_kernel: 16-byte pieces of a head that are taken, 64 at most
};

// `shares` warps take a token's heads in turn, in a streamed walk or not.  (Two 16-byte buffers want more registers: 512
// tokens 4.3 us with kRopeBlocks, 3.8 with 6.)
template <typename E, int W, bool HALF, bool STREAM>
__global__ void __launch_bounds__(kRopeThreads, !STREAM && sizeof(Piece<E, W>) == 16 ? 6 : kRopeBlocks)
    rope_kernel(const RopeParams p, int shares, int stages)
{
    extern __shared__ __align__(16) uint8_t rope_smem[];  // [kRopeWarps][stages][64] pieces, [kRopeWarps][R] floats
    const int warp = threadIdx.x >> 5;
    uint4 *ring = reinterpret_cast<uint4 *>(rope_smem) + warp * stages * 64;
    float *cs = reinterpret_cast<float *>(rope_smem + kRopeWarps * stages * 1024) + warp * p.R;
    const int64_t gw = (int64_t)blockIdx.x * kRopeWarps + warp, t = gw / shares;
    griddep_wait();
    griddep_launch_dependents();
    if (t >= p.T) return;
    const int share = (int)(gw - t * shares);
    const E *x = static_cast<const E *>(p.x) + t * p.x_token;
    E *y = static_cast<E *>(p.y) + t * p.y_token;
    bool have = false;
    auto ready = [&] {
        if (!have && p.R > 0) rope_angles(cs, p.inv_freq, p.R / 2, p.pos[t], p.scale, p.inverse != 0);
        have = true;
        return true;
    };
    int copy_piece = p.copy_piece;
    if constexpr (STREAM) {
        const RopeStretch<E> st[1] = {{x, p.x_head, p.y_head, p.H}};
        rope_stream<E, W, HALF>(st, 1, p.R, copy_piece == 16 ? p.D - p.R : 0, share, shares, ring, stages, cs, ready,
                                [&](int) { return y; });
        if (copy_piece == 16) copy_piece = 0;
    } else {
        rope_walk<E, W, HALF>(RopeLane<W>(p.R), x, p.x_head, p.y_head, p.H, p.R, share, shares, cs, ready, [&] { return y; });
    }
    if (copy_piece)
        copy_heads(
            copy_piece, x + p.R, p.x_head * (int)sizeof(E), p.y_head * (int)sizeof(E), p.H, (p.D - p.R) * (int)sizeof(E),
            share, shares, [] { return true; }, [&] { return reinterpret_cast<uint8_t *>(y + p.R); });
}

// rope_kernel with the staged walk.
template <typename E, bool HALF>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks) rope_staged_kernel(const RopeParams p, int shares, int stages)
{
    extern __shared__ __align__(16) uint8_t rope_smem[];  // as in rope_kernel
    const int warp = threadIdx.x >> 5;
    uint4 *ring = reinterpret_cast<uint4 *>(rope_smem) + warp * stages * 64;
    float *cs = reinterpret_cast<float *>(rope_smem + kRopeWarps * stages * 1024) + warp * p.R;
    const int64_t gw = (int64_t)blockIdx.x * kRopeWarps + warp, t = gw / shares;
    griddep_wait();
    griddep_launch_dependents();
    if (t >= p.T) return;
    E *y = static_cast<E *>(p.y) + t * p.y_token;
    const RopeStretch<E> st[1] = {{static_cast<const E *>(p.x) + t * p.x_token, p.x_head, p.y_head, p.H}};
    rope_staged<E, HALF>(
        st, 1, p.R, p.pieces, (int)(gw - t * shares), shares, ring, stages, cs,
        [&] {
            rope_angles(cs, p.inv_freq, p.R / 2, p.pos[t], p.scale, p.inverse != 0);
            return true;
        },
        [&](int) { return y; });
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
    int32_t pieces;               // rope_staged: 16-byte pieces of a head
    int32_t rest_piece, v_piece;  // bytes per copied piece of entries R .. D-1 of queries and keys (0: none), and of values
    float scale;
    int32_t *status;
};

// The place in its sequence that new token t takes, by a warp.
struct AppendPlace {
    int64_t at;       // place in the sequence
    int32_t b;        // sequence, or -1: the token is skipped
    int32_t page;     // what the table says, -1 where it says nothing
};

__device__ __forceinline__ AppendPlace append_place(const AppendParams &p, int64_t t)
{
    int b = (int)t, left = 1;  // tokens of the sequence from t on
    if (p.cu != nullptr) {
        b = warp_count_le(p.cu, p.B + 1, (int)t) - 1;
        if (b < 0 || b >= p.B) return {0, -1, -1};  // before the first sequence or behind the last: not ours
        left = p.cu[b + 1] - (int)t;
    }
    const int32_t len = p.lens[b];
    if (len == 0) return {0, -1, -1};  // an empty place of a padded batch
    const int64_t at = (int64_t)len - left;
    int32_t page = -1;
    if (left >= 1 && at >= 0 && at / p.page_size < p.max_pages) page = p.table[b * p.table_row + at / p.page_size];
    return {at, b, page};
}

// What a streamed walk of 16-byte pieces takes with it: the entries that are only copied, and the values.
template <int W>
__host__ __device__ inline int append_rest(const AppendParams &p)
{
    return W == 8 && p.rest_piece == 16 ? p.D - p.R : 0;
}
template <int W>
__host__ __device__ inline bool append_values(const AppendParams &p)
{
    return W == 8 && p.v_piece == 16 && p.R + append_rest<W>(p) == p.D;
}

// `shares` warps take a token's query heads, key heads and values in turn.
template <int W, bool HALF, bool STAGED = false>
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks)
    paged_append_kernel(const AppendParams p, int shares, int stages)
{
    using E = __nv_bfloat16;
    extern __shared__ __align__(16) uint8_t rope_smem[];  // as in rope_kernel
    const int warp = threadIdx.x >> 5;
    uint4 *ring = reinterpret_cast<uint4 *>(rope_smem) + warp * stages * 64;
    float *cs = reinterpret_cast<float *>(rope_smem + kRopeWarps * stages * 1024) + warp * p.R;
    const int64_t gw = (int64_t)blockIdx.x * kRopeWarps + warp, t = gw / shares;
    griddep_wait();
    griddep_launch_dependents();
    if (t >= p.T) return;
    const int share = (int)(gw - t * shares);
    int64_t row = -1;  // offset of the token's row in the cache (head 0), or -1: the token is skipped
    bool have = false;
    auto ready = [&] {
        if (!have) {
            const AppendPlace w = append_place(p, t);
            have = true;
            if (w.b < 0) return false;
            // The angles do not need the page, which is still on its way.
            if (p.R > 0) rope_angles(cs, p.inv_freq, p.R / 2, p.positions ? p.positions[t] : (int32_t)w.at, p.scale, false);
            if (w.page < 0 || w.page >= p.pages)
                record_error(p.status, 1);  // BI_ERR_INVALID_ARG
            else
                row = w.page * p.c_page + (w.at % p.page_size) * p.c_token;
        }
        return row >= 0;
    };
    const E *q = p.q + t * p.q_token, *k = p.k + t * p.k_token, *v = p.v + t * p.v_token;
    E *qo = p.q_out + t * p.qo_token;
    auto bytes_at = [](E *e) { return reinterpret_cast<uint8_t *>(e); };
    constexpr int kE = sizeof(E);
    if constexpr (STAGED) {
        const RopeStretch<E> st[3] = {{q, p.q_head, p.qo_head, p.q != nullptr ? p.Hq : 0},
                                      {k, p.k_head, p.c_head, p.Hkv},
                                      {v, p.v_head, p.c_head, p.Hkv}};
        rope_staged<E, HALF>(st, 2, p.R, p.pieces, share, shares, ring, stages, cs, ready,
                             [&](int i) { return i == 0 ? qo : (i == 1 ? p.k_cache : p.v_cache) + row; });
        return;
    }
    int rest = p.rest_piece ? p.D - p.R : 0;  // entries left to copy after the walk
    if constexpr (W == 8) {
        const RopeStretch<E> st[3] = {{q, p.q_head, p.qo_head, p.q != nullptr ? p.Hq : 0},
                                      {k, p.k_head, p.c_head, p.Hkv},
                                      {v, p.v_head, p.c_head, append_values<W>(p) ? p.Hkv : 0}};
        if (!rope_stream<E, W, HALF>(st, 2, p.R, append_rest<W>(p), share, shares, ring, stages, cs, ready,
                                     [&](int i) { return i == 0 ? qo : (i == 1 ? p.k_cache : p.v_cache) + row; }))
            return;
        rest -= append_rest<W>(p);
    } else {
        const RopeLane<W> me(p.R);
        int group = share;  // the warp's next group of heads; the key heads go on where the query heads end
        if (p.q != nullptr) {
            if (!rope_walk<E, W, HALF>(me, q, p.q_head, p.qo_head, p.Hq, p.R, group, shares, cs, ready, [&] { return qo; }))
                return;
            group = (share + shares - (p.Hq + me.heads - 1) / me.heads % shares) % shares;
        }
        if (!rope_walk<E, W, HALF>(me, k, p.k_head, p.c_head, p.Hkv, p.R, group, shares, cs, ready,
                                   [&] { return p.k_cache + row; }))
            return;
    }
    if (rest > 0) {
        if (p.q != nullptr && !copy_heads(p.rest_piece, q + p.R, p.q_head * kE, p.qo_head * kE, p.Hq, rest * kE, share, shares,
                                          ready, [&] { return bytes_at(qo + p.R); }))
            return;
        if (!copy_heads(p.rest_piece, k + p.R, p.k_head * kE, p.c_head * kE, p.Hkv, rest * kE, share, shares, ready,
                        [&] { return bytes_at(p.k_cache + row + p.R); }))
            return;
    }
    if (!append_values<W>(p))
        copy_heads(p.v_piece, v, p.v_head * kE, p.c_head * kE, p.Hkv, p.D * kE, share, shares, ready,
                   [&] { return bytes_at(p.v_cache + row); });
}

}  // namespace bi
