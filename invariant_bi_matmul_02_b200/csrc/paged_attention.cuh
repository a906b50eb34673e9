// paged_attention.cuh -- batch-invariant decode attention over a paged cache (one query token per
// sequence).
//
// The cache is pages of P tokens; a sequence's block table names its pages in order.  A sequence of up to
// kPgWhole tokens is one split (no second launch: with splits of 256 the 5.5 us of 300 tokens were 1 us more), a
// longer one is cut into splits of kPgSplit tokens, and each split into tiles of kPgTile tokens: cuts fixed by
// the sequence's own length.  A (split, kv head) is taken by a group of four warps: warp w takes tiles w,
// w + 4, ..., with a running maximum; scores, weights and the weighted value sum never leave the warp.
// The four warps are then folded in order through shared memory; a sequence of one split is written out
// at once, the splits of a longer one go to scratch and are folded by the second launch in a tree fixed
// by the number of splits.  So a sequence's output depends on its own query, tokens and length only.
//
// Bound by the cache's bytes (B200: 64 sequences of 4096 tokens, 32 / 8 heads of 128, pages of 16, 170 us or
// 6.3 TB/s; 256 of 512 tokens 81.7 us, 6.6 TB/s) and, for a few short sequences, by latency: prefix sums, page
// table and first tile take about 2 us, a tile 0.7 us, the fold 0.7 us.  One persistent CTA per SM; the (split, kv
// head) items of the batch are numbered through the prefix sums of the sequences' split counts, so a CTA's share does not
// depend on how ragged the batch is; two consumer groups take alternate items, so that one's folding overlaps the
// other's arithmetic and loads.  The producers fill a ring of tiles (K and V of 32 tokens: 16 KB at
// head size 128, 8 tiles; 8 KB at 64, 20 tiles) by TMA: boxes of gcd(P, kPgTile) tokens x 64
// entries, each within one page and completing on the tile's mbarrier.  The lanes look pages up one chunk of
// 32 boxes ahead and each issues its own box.  Four producer warps issue alternate tiles: one warp needs about
// 1000 cycles a tile in pages of 16 (wait, barrier, 8 copies), more than a tile takes to arrive.
//
// Tensor-core work (mma.sync m16n8k16, bf16 in, fp32 accumulate): S^T = K Q^T with tokens on the 16
// rows and the group's heads on the 8 columns (two column tiles for groups of 9 to 16), then
// O^T += V^T P^T with the head's entries on the rows.  An fp32 weight enters as three bf16 terms, its upper 8, next 8
// and last 8 bits (pg_terms), whose sum it is, so the only rounding to fewer than 24 bits is the output's.  (Two
// terms, 16 bits, made one output in 500 round otherwise than in fp32.  The third costs nothing where memory bounds, 0.1 us of
// one sequence's 5.7, 0.4 of the ragged batch's 25, and with 16 query heads per kv head 112 us for 105 at 32 x 4096.)
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "attention.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace bi {

constexpr int kPgTile = 32;                      // tokens per ring stage, one consumer warp's
constexpr int kPgWarps = 8;                      // consumer warps
constexpr int kPgGroups = 2;                     // consumer groups, alternate items
constexpr int kPgGroupWarps = kPgWarps / kPgGroups;
constexpr int kPgSplit = 256;                    // tokens per split: two tiles for each warp of a group
constexpr int kPgWhole = 512;                    // a sequence of up to this many tokens is one split
constexpr int kPgProducers = 4;                  // producer warps
constexpr int kPgThreads = 32 * (kPgWarps + kPgProducers);
constexpr int kPgSeqs = 2048;                    // sequences per launch (their prefix sums are in shared memory)

template <int D>
struct PgShape {
    static constexpr int kHalves = D / 64;                  // 64-entry TMA boxes per token row
    static constexpr int kHalfBytes = kPgTile * 128;        // one half of a tile's K or V
    static constexpr int kKBytes = kHalves * kHalfBytes;    // K (or V) of a tile
    static constexpr int kStageBytes = 2 * kKBytes;
    static constexpr int kStages = D == 64 ? 20 : 8;        // 160 or 128 KB: what the fold's buffers leave, by fours
    static constexpr int kORow = D + 4;                     // floats between heads of a warp's sums: no bank conflicts
    static constexpr int kOFloats = kPgWarps * 8 * kORow;   // one buffer of the warps' sums, eight heads
    static_assert(kStages % kPgProducers == 0, "a stage is always filled by the same producer warp");
    static constexpr int kSmem = kStages * kStageBytes + 2 * kOFloats * 4 + 1024;  // + alignment slack
};

// Quotients of numbers below 2^31 by a divisor that the host knows: n / d = n * mul >> shift, with
// mul = ceil(2^shift / d) and shift = 31 + ceil(log2 d).
struct PgDivisor {
    uint32_t mul, shift, d;
    __host__ static PgDivisor of(uint32_t d)
    {
        uint32_t l = 0;
        while ((uint64_t(1) << l) < d) ++l;
        return {(uint32_t)(((uint64_t(1) << (31 + l)) + d - 1) / d), 31 + l, d};
    }
    __device__ __forceinline__ uint32_t quotient(uint32_t n) const { return (uint32_t)((uint64_t)n * mul >> shift); }
};

struct PgParams {
    const __nv_bfloat16 *q;
    int64_t q_row;  // entries between sequences
    const int32_t *table;
    int64_t table_row;
    const int32_t *lens;
    float *part_o;     // [B, Hq, S, D]
    float2 *part_ml;   // [B, Hq, S] (maximum in units of log2, sum)
    __nv_bfloat16 *out;  // [B, Hq, D]
    int32_t B, Hq, Hkv, G, S, pages, max_len;
    PgDivisor by_page, by_heads;  // page_size and Hkv
    int32_t box;          // tokens per TMA box: gcd(page_size, kPgTile)
    int32_t box_log2, boxes;  // boxes per tile: kPgTile / box
    int32_t chunk;        // tiles per 32 boxes
    int32_t heads_inner;  // dimension order of the tensor maps: (entry, head, token, page) or (entry, token, head, page)
    float scale_log2;     // score scale times log2(e)
    int32_t *status;
    uint64_t wait_limit_ns;
};

__host__ __device__ inline int64_t pg_splits(int64_t L)
{
    return L <= 0 ? 0 : L <= kPgWhole ? 1 : (L + kPgSplit - 1) / kPgSplit;
}

// Length as the kernels use it: outside 0 .. max_len it is clamped (and reported by the first launch).
__device__ __forceinline__ int pg_len(int L, int max_len)
{
    return L < 0 ? 0 : (L > max_len ? max_len : L);
}

// 8x8 b16 matrix in the mma register layout, transposed across the warp.
__device__ __forceinline__ uint32_t movm_trans(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Weights x and y as bf16 terms, each the upper half of what is left of its fp32 word (x low, y high in a register),
// turned so that tokens run along a thread's registers.  Every difference is exact; terms below 2^-133 are lost.
__device__ __forceinline__ void pg_terms(uint32_t (&t)[3], float x, float y)
{
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
        t[i] = movm_trans(__byte_perm(a, b, 0x7632));
        x = __fsub_rn(x, __uint_as_float(a & 0xffff0000u));
        y = __fsub_rn(y, __uint_as_float(b & 0xffff0000u));
    }
}

// Launch 1: grid = min(items, SMs).  Item i: kv head i % Hkv of the global split i / Hkv (kv head
// fastest, so neighbouring CTAs read neighbouring pieces of the same tokens' rows).
template <int D, int NT>  // NT column tiles of 8 query heads per kv head
__global__ void __launch_bounds__(kPgThreads, 1)
    paged_attention_split_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                                 const PgParams p)
{
    using C = PgShape<D>;
    extern __shared__ uint8_t pg_raw[];
    uint8_t *smem = pg_raw + ((1024u - (smem_addr(pg_raw) & 1023u)) & 1023u);
    float *so_all = reinterpret_cast<float *>(smem + C::kStages * C::kStageBytes);  // [2][warp][8 heads][kORow]
    __shared__ uint64_t full[C::kStages], empty[C::kStages];
    __shared__ float red_m[2][kPgWarps][8], red_l[2][kPgWarps][8];
    __shared__ int32_t first[kPgSeqs + 1];  // global number of each sequence's first split
    __shared__ int32_t lens_s[kPgSeqs];
    __shared__ int32_t warp_total[kPgThreads / 32];
    __shared__ int abort_flag_s;
    __shared__ int slot_use_s[C::kStages];  // uses of each stage that a consumer warp has passed
    volatile int *abort_flag = &abort_flag_s, *slot_use = slot_use_s;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            slot_use_s[s] = 0;
        }
        abort_flag_s = 0;
        fence_mbar_init();
    } else if (tid == 32 * kPgWarps) {
        prefetch_tensor_map(&tm_k);
        prefetch_tensor_map(&tm_v);
    }
    griddep_wait();  // the previous kernel's output (q, cache, lengths, table) is complete
    griddep_launch_dependents();

    // Prefix sums of the split counts (an empty sequence counts as one split, which writes its zeros).
    {
        const int per = (p.B + kPgThreads - 1) / kPgThreads, b0 = tid * per;
        int sum = 0;
        for (int j = 0; j < per && b0 + j < p.B; ++j) {
            const int given = p.lens[b0 + j], L = pg_len(given, p.max_len);
            if (blockIdx.x == 0 && L != given) record_error(p.status, 1);  // BI_ERR_INVALID_ARG
            lens_s[b0 + j] = L;
            const int n = (int)pg_splits(L);
            sum += n > 0 ? n : 1;
        }
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) warp_total[warp] = inc;
        __syncthreads();
        int at = inc - sum + (int)__reduce_add_sync(0xffffffffu, lane < warp ? (unsigned)warp_total[lane] : 0u);
        for (int j = 0; j < per && b0 + j < p.B; ++j) {
            first[b0 + j] = at;
            const int n = (int)pg_splits(lens_s[b0 + j]);
            at += n > 0 ? n : 1;
        }
        if (b0 < p.B && b0 + per >= p.B) first[p.B] = at;
    }
    __syncthreads();

    const uint32_t n_kv = (uint32_t)p.Hkv;
    const uint32_t items = (uint32_t)first[p.B] * n_kv;
    const uint64_t lim = p.wait_limit_ns;
    struct Item {
        int b, g, split, t0, n;  // n tokens from t0 on
    };
    // Items come in ascending order: the sequence is searched from the last one on, 32 at a time.
    int b = 0, first_b = 0;
    auto item = [&](uint32_t it) -> Item {
        const int sg = (int)p.by_heads.quotient(it), g = (int)(it - (uint32_t)sg * n_kv);
        int passed;
        do {
            const int v = b + 1 + lane < p.B ? first[b + 1 + lane] : 0x7fffffff;
            passed = __popc(__ballot_sync(0xffffffffu, v <= sg));
            if (passed > 0) first_b = __shfl_sync(0xffffffffu, v, passed - 1);
            b += passed;
        } while (passed == 32);
        const int split = sg - first_b, t0 = split * kPgSplit;
        const int L = lens_s[b], left = L - t0, most = L <= kPgWhole ? kPgWhole : kPgSplit;
        return {b, g, split, t0, left < most ? left : most};
    };

    if (warp >= kPgWarps) {
        // ------------------------------------------------------------------ producers
        // Tiles are numbered across the CTA's items; number n goes to stage n % kStages as its use n / kStages and
        // is issued by producer warp n % kPgProducers.  kStages is a multiple of kPgProducers, so a stage's uses
        // are issued by one warp in order, and its parity waits are exact.
        const uint32_t pw = (uint32_t)(warp - kPgWarps);
        const uint64_t policy = l2_policy_evict_first();  // every cache byte is read once
        const int nb = p.boxes, chunk_tiles = p.chunk;    // a chunk is 32 boxes, one per lane
        // A chunk of an item: its lane's box, the page it lies in and its first row there.
        struct Chunk {
            Item w;
            uint32_t it;    // the item's number (>= items: none left)
            int tile0;      // first tile of the chunk within the item
            int32_t page, row;
        };
        auto look_up = [&](Chunk &c) {
            const int k = c.tile0 * kPgTile + lane * p.box;  // token within the item
            c.page = c.row = 0;
            if (k < c.w.n) {
                const uint32_t t = (uint32_t)(c.w.t0 + k), at = p.by_page.quotient(t);
                c.page = p.table[c.w.b * p.table_row + at];
                c.row = (int32_t)(t - at * p.by_page.d);
            }
        };
        auto enter = [&](Chunk &c, uint32_t it) {  // the first chunk of the next item with tokens, from item `it` on
            for (c.it = it; c.it < items; c.it += gridDim.x) {
                c.w = item(c.it);
                if (c.w.n > 0) break;
            }
            c.tile0 = 0;
            if (c.it < items) look_up(c);
        };
        uint32_t base = 0, mine = 0;  // the item's first tile number; tiles this warp has issued
        bool ok = true;
        Chunk cur;
        enter(cur, blockIdx.x);
        while (ok && cur.it < items) {
            const int tiles = (cur.w.n + kPgTile - 1) / kPgTile, end = cur.tile0 + chunk_tiles;
            Chunk next = cur;
            auto look_ahead = [&] {
                if (end < tiles) {
                    next.tile0 = end;
                    look_up(next);
                } else {
                    enter(next, cur.it + gridDim.x);
                }
            };
            // The next chunk's pages are looked up while this one's boxes are issued (the first chunk's boxes go
            // first).
            const bool start = mine == 0 && cur.it == blockIdx.x;
            if (!start) look_ahead();
            const uint32_t n0 = base + (uint32_t)cur.tile0;
            for (int j = cur.tile0 + (int)((pw - n0) % kPgProducers); j < end && j < tiles; j += kPgProducers) {
                const uint32_t num = base + (uint32_t)j, stage = num % C::kStages, use = num / C::kStages;
                ok = __all_sync(0xffffffffu, wait_bounded(&empty[stage], (use & 1u) ^ 1u, abort_flag, p.status, lim));
                if (!ok) break;
                const int left = cur.w.n - kPgTile * j, cnt = left >= kPgTile ? nb : (left + p.box - 1) >> p.box_log2;
                if (lane == 0) mbar_arrive_expect_tx(&full[stage], (uint32_t)(cnt * p.box * D * 2 * 2));
                __syncwarp();
                const int x = lane - (j - cur.tile0) * nb;
                if (x >= 0 && x < cnt) {
                    int32_t pg = cur.page;
                    if (pg < 0 || pg >= p.pages) {  // no such page: recorded, and read as zeros (out of the map's range)
                        record_error(p.status, 1);  // BI_ERR_INVALID_ARG
                        pg = p.pages;
                    }
                    uint8_t *dst = smem + stage * C::kStageBytes + x * p.box * 128;
                    const int c1 = p.heads_inner ? cur.w.g : cur.row, c2 = p.heads_inner ? cur.row : cur.w.g;
#pragma unroll
                    for (int h = 0; h < C::kHalves; ++h)
                        tma_load_4d(dst + h * C::kHalfBytes, &tm_k, &full[stage], 64 * h, c1, c2, pg, policy);
#pragma unroll
                    for (int h = 0; h < C::kHalves; ++h)
                        tma_load_4d(dst + C::kKBytes + h * C::kHalfBytes, &tm_v, &full[stage], 64 * h, c1, c2, pg, policy);
                }
                ++mine;
            }
            if (start) look_ahead();
            if (next.it != cur.it) base += (uint32_t)tiles;
            cur = next;
        }
        if (!ok && lane == 0) {
            // A wait ran out: let every copy this warp has issued land before shared memory goes away.
            constexpr uint32_t kOwn = C::kStages / kPgProducers;  // its stages
            for (uint32_t i = mine > kOwn ? mine - kOwn : 0; i < mine; ++i) {
                const uint32_t num = i * kPgProducers + pw, stage = num % C::kStages;
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait(smem_addr(&full[stage]), (num / C::kStages) & 1u) && global_timer_ns() - t0 < lim) {
                }
            }
        }
    } else {
        // ------------------------------------------------------------------ consumers
        // Group grp takes the CTA's items grp, grp + 2, ...; its warp cw tiles cw, cw + 4, ... of each.  Tiles are
        // numbered across all of the CTA's items in the producer's order; tile number n is use n / kStages of stage
        // n % kStages.  A stage's uses are passed in order: once its previous use has been passed (slot_use, by
        // either group) its barrier is at most one phase from the one waited for, so a parity wait is exact.
        const int grp = warp / kPgGroupWarps, cw = warp % kPgGroupWarps, ct = tid % (32 * kPgGroupWarps);
        const int gid = lane >> 2, tig = lane & 3;
        uint32_t base = 0, local = 0;
        bool alive = true;
        const int w0 = grp * kPgGroupWarps;  // the group's first warp
        int buf = 0;
        for (uint32_t it = blockIdx.x; it < items; it += gridDim.x) {
            const Item w = item(it);
            const int tiles = (w.n + kPgTile - 1) / kPgTile;
            const int head0 = w.g * p.G;
            const uint32_t num0 = base;
            base += (uint32_t)tiles;
            if ((int)(local++ % kPgGroups) != grp) continue;
            if (w.n <= 0) {  // an empty sequence: its row is zeros
                __nv_bfloat16 *o = p.out + ((int64_t)w.b * p.Hq + head0) * D;
                for (int i = ct; i < p.G * D / 8; i += 32 * kPgGroupWarps) reinterpret_cast<uint4 *>(o)[i] = make_uint4(0, 0, 0, 0);
                continue;
            }
            const int warps = tiles < kPgGroupWarps ? tiles : kPgGroupWarps;  // with a tile of this item
            float m[NT][2], l[NT][2];  // of heads 8 nt + 2 tig and + 1; l of this thread's tokens only
            float o[NT][D / 16][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                m[nt][0] = m[nt][1] = kNegInf;
                l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.0f;
            }
            if (cw < warps) {
                // Q^T fragments: column n = head, rows k = entries 16 kk + 2 tig (+1) and + 8.
                uint32_t qf[NT][D / 16][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const bool live = 8 * nt + gid < p.G;
                    const __nv_bfloat16 *qr = p.q + w.b * p.q_row + (int64_t)(head0 + 8 * nt + gid) * D + 2 * tig;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        qf[nt][kk][0] = live ? *reinterpret_cast<const uint32_t *>(qr + 16 * kk) : 0u;
                        qf[nt][kk][1] = live ? *reinterpret_cast<const uint32_t *>(qr + 16 * kk + 8) : 0u;
                    }
                }
#pragma unroll 1
                for (int j = cw; j < tiles; j += kPgGroupWarps) {
                    const uint32_t num = num0 + (uint32_t)j, stage = num % C::kStages, use = num / C::kStages;
                    if (alive)
                        alive = __all_sync(0xffffffffu,
                                           wait_flag_at_least(&slot_use[stage], (int)use, abort_flag, p.status, lim) &&
                                               wait_bounded(&full[stage], use & 1u, abort_flag, p.status, lim));
                    if (!alive) break;
                    if (lane == 0) slot_use[stage] = (int)use + 1;
                    const uint8_t *ks = smem + stage * C::kStageBytes, *vs = ks + C::kKBytes;
                    const int n_tok = w.n - kPgTile * j < kPgTile ? w.n - kPgTile * j : kPgTile;
                    // 16-byte chunk c of token row r: 128-byte swizzle within each 64-entry half.
                    auto chunk = [&](const uint8_t *t, int r, int c) {
                        return t + (c >> 3) * C::kHalfBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4);
                    };
                    // ---- scores of tokens 16 mt + gid (+ 8) and heads 8 nt + 2 tig (+ 1)
                    float s[NT][2][4];
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) s[nt][mt][0] = s[nt][mt][1] = s[nt][mt][2] = s[nt][mt][3] = 0.0f;
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            uint32_t a[4];
                            ldsm_x4(a, chunk(ks, 16 * mt + (lane & 15), 2 * kk + (lane >> 4)));
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma_16816_bf16(s[nt][mt], a, qf[nt][kk][0], qf[nt][kk][1]);
                        }
                    }
                    // ---- running maximum, rescaled sums, weights; tokens past the sequence weigh nothing
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float f[2];
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float v = kNegInf;
#pragma unroll
                            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                                for (int r = 0; r < 2; ++r) {
                                    float &x = s[nt][mt][2 * r + c];
                                    x = 16 * mt + gid + 8 * r < n_tok ? __fmul_rn(x, p.scale_log2) : kNegInf;
                                    v = fmaxf(v, x);
                                }
                            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                            v = fmaxf(v, m[nt][c]);
                            const float ref = v == kNegInf ? 0.0f : v;
                            f[c] = ex2(m[nt][c] - ref);  // 0 at the first tile
                            m[nt][c] = v;
                            float sum = __fmul_rn(l[nt][c], f[c]);
#pragma unroll
                            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                                for (int r = 0; r < 2; ++r) {
                                    float &x = s[nt][mt][2 * r + c];
                                    x = ex2(x - ref);
                                    sum = __fadd_rn(sum, x);
                                }
                            l[nt][c] = sum;
                        }
                        if (j >= kPgGroupWarps) {
#pragma unroll
                            for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
                                for (int e = 0; e < 4; ++e) o[nt][mt][e] = __fmul_rn(o[nt][mt][e], f[e & 1]);
                        }
                    }
                    // ---- O^T += V^T P^T over two 16-token steps in ascending order, the larger terms first
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        uint32_t w[NT][2][3];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int r = 0; r < 2; ++r) pg_terms(w[nt][r], s[nt][mt][2 * r], s[nt][mt][2 * r + 1]);
                        // Value rows past the sequence hold anything: their bits are cleared.
                        const int ta = 16 * mt + 2 * tig;
                        uint32_t keep[2];
#pragma unroll
                        for (int r = 0; r < 2; ++r)
                            keep[r] = (ta + 8 * r < n_tok ? 0xffffu : 0u) | (ta + 8 * r + 1 < n_tok ? 0xffff0000u : 0u);
#pragma unroll
                        for (int dt = 0; dt < D / 8; dt += 2) {
                            uint32_t v[4];
                            ldsm_x4_trans(v, chunk(vs, 16 * mt + (lane & 15), dt + (lane >> 4)));
                            const uint32_t a[4] = {v[0] & keep[0], v[2] & keep[0], v[1] & keep[1], v[3] & keep[1]};
#pragma unroll
                            for (int i = 0; i < 3; ++i)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma_16816_bf16(o[nt][dt / 2], a, w[nt][0][i], w[nt][1][i]);
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty[stage]);
                }
            }
            // ---- fold the warps in order through shared memory, eight heads at a time.  Two buffers: a warp that
            // writes one has passed the barrier behind which the other was read.
            const bool last = first[w.b + 1] - first[w.b] == 1;  // the sequence's only split
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int heads = p.G - 8 * nt < 8 ? p.G - 8 * nt : 8;
                float(*gm)[8] = red_m[buf] + w0, (*gl)[8] = red_l[buf] + w0;
                float *so_grp = so_all + buf * C::kOFloats + w0 * 8 * C::kORow, *so = so_grp + cw * 8 * C::kORow;
                buf ^= 1;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float v = l[nt][c];
                    v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, 4));
                    v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, 8));
                    v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, 16));
                    if (gid == 0) {
                        gm[cw][2 * tig + c] = m[nt][c];
                        gl[cw][2 * tig + c] = v;
                    }
                }
                if (cw < warps) {
#pragma unroll
                    for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (2 * tig + (e & 1) < heads)
                                so[(2 * tig + (e & 1)) * C::kORow + 16 * mt + gid + 8 * (e >> 1)] = o[nt][mt][e];
                }
                consumers_sync(1 + grp);
                for (int i = ct; i < heads * (D / 4); i += 32 * kPgGroupWarps) {
                    const int h = i / (D / 4), d = 4 * (i % (D / 4));
                    // All loads at once; a warp without a tile counts with a maximum of -inf and zeros.
                    float mt[kPgGroupWarps], lt[kPgGroupWarps], mx = kNegInf, sum = 0.0f;
                    float4 v[kPgGroupWarps], r = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int t = 0; t < kPgGroupWarps; ++t) {
                        const bool some = t < warps;
                        mt[t] = some ? gm[t][h] : kNegInf;
                        lt[t] = some ? gl[t][h] : 0.0f;
                        v[t] = some ? *reinterpret_cast<const float4 *>(so_grp + (t * 8 + h) * C::kORow + d) : r;
                    }
#pragma unroll
                    for (int t = 0; t < kPgGroupWarps; ++t) mx = fmaxf(mx, mt[t]);
                    const float ref = mx == kNegInf ? 0.0f : mx;
#pragma unroll
                    for (int t = 0; t < kPgGroupWarps; ++t) {
                        const float f = ex2(mt[t] - ref);
                        sum = __fmaf_rn(lt[t], f, sum);
                        r.x = __fmaf_rn(v[t].x, f, r.x);
                        r.y = __fmaf_rn(v[t].y, f, r.y);
                        r.z = __fmaf_rn(v[t].z, f, r.z);
                        r.w = __fmaf_rn(v[t].w, f, r.w);
                    }
                    const int64_t bh = (int64_t)w.b * p.Hq + head0 + 8 * nt + h;
                    if (last) {
                        uint2 u;
                        u.x = pack_bf16(r.x / sum, r.y / sum);
                        u.y = pack_bf16(r.z / sum, r.w / sum);
                        *reinterpret_cast<uint2 *>(p.out + bh * D + d) = u;
                    } else {
                        *reinterpret_cast<float4 *>(p.part_o + (bh * p.S + w.split) * D + d) = r;
                        if (d == 0) p.part_ml[bh * p.S + w.split] = make_float2(mx, sum);
                    }
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------------------- launch 2
// Folds the splits of each (sequence, query head).  Up to kPgSerial splits run in ascending order; more are taken
// by 32 groups, group g splits g, g + 32, ..., folded in a fixed butterfly and then in order.  The cut depends on
// the sequence's own number of splits, so both kernels below give a sequence the same bits.
constexpr int kPgCombineThreads = 256;
constexpr int kPgSerial = 32;
constexpr int kPgAhead = 16;  // splits whose values a thread has in flight

// Splits s0, s0 + step, ... below n (at most kPgAhead): four columns of each and its maximum and sum.
struct PgBatch {
    float4 x[kPgAhead];
    float2 w[kPgAhead];
    __device__ __forceinline__ void load(const float2 *ml, const float4 *v, int row, int s0, int step, int n)
    {
#pragma unroll
        for (int k = 0; k < kPgAhead; ++k) {
            const int s = s0 + k * step;
            x[k] = s < n ? v[(int64_t)s * row] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            w[k] = s < n ? ml[s] : make_float2(kNegInf, 0.0f);
        }
    }
};

struct PgFold {
    float l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    __device__ __forceinline__ void add(float4 v, float2 ml, float ref)
    {
        const float f = ex2(ml.x - ref);  // 0 for the padding (maximum -inf)
        l = __fmaf_rn(ml.y, f, l);
        o.x = __fmaf_rn(v.x, f, o.x);
        o.y = __fmaf_rn(v.y, f, o.y);
        o.z = __fmaf_rn(v.z, f, o.z);
        o.w = __fmaf_rn(v.w, f, o.w);
    }
    // Splits first, first + step, ... below n in order; `batch` holds the first of them.
    __device__ __forceinline__ void run(PgBatch &batch, const float2 *ml, const float4 *v, int row, int first, int step, int n,
                                        float ref)
    {
        for (int s0 = first;;) {
#pragma unroll
            for (int k = 0; k < kPgAhead; ++k) add(batch.x[k], batch.w[k], ref);
            s0 += kPgAhead * step;
            if (s0 >= n) break;
            batch.load(ml, v, row, s0, step, n);
        }
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *out) const
    {
        uint2 u;
        u.x = pack_bf16(o.x / l, o.y / l);
        u.y = pack_bf16(o.z / l, o.w / l);
        *reinterpret_cast<uint2 *>(out) = u;
    }
};

__device__ __forceinline__ float pg_warp_max(float m)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// No sequence has more than kPgSerial splits: a warp takes 128 / D (sequence, head) pairs.
template <int D>
__global__ void __launch_bounds__(kPgCombineThreads)
    paged_attention_combine_kernel(const float2 *__restrict__ part_ml, const float *__restrict__ part_o,
                                   const int32_t *__restrict__ lens, __nv_bfloat16 *__restrict__ out, int Hq, int S,
                                   int max_len, int rows)
{
    constexpr int kLanes = D / 4;
    const int bh = (int)((blockIdx.x * (unsigned)kPgCombineThreads + threadIdx.x) / kLanes), c = threadIdx.x % kLanes;
    // Launch 1 lets this kernel start once all its blocks have seen the inputs complete, so the lengths, which it
    // does not write, need no wait.
    const int n = bh < rows ? (int)pg_splits(pg_len(lens[bh / Hq], max_len)) : 0;
    griddep_wait();
    griddep_launch_dependents();
    const float2 *ml = part_ml + (int64_t)bh * S;
    const float4 *po = reinterpret_cast<const float4 *>(part_o + (int64_t)bh * S * D) + c;
    PgBatch batch;  // on its way while the maximum (exact in any order) is found
    if (n > 1) batch.load(ml, po, kLanes, 0, 1, n);
    float m = kNegInf;
    for (int s = c; s < n; s += kLanes) m = fmaxf(m, ml[s].x);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (n <= 1) return;  // written by launch 1, or no such row
    PgFold f;
    f.run(batch, ml, po, kLanes, 0, 1, n, m == kNegInf ? 0.0f : m);
    f.store(out + (int64_t)bh * D + 4 * c);
}

// Grid (D / 32, Hq, B): 8 lanes of four columns, 32 groups.
template <int D>
__global__ void __launch_bounds__(kPgCombineThreads)
    paged_attention_combine_long_kernel(const float2 *__restrict__ part_ml, const float *__restrict__ part_o,
                                        const int32_t *__restrict__ lens, __nv_bfloat16 *__restrict__ out, int Hq, int S,
                                        int max_len)
{
    constexpr int kWarps = kPgCombineThreads / 32;
    __shared__ float red[kWarps], sl[kWarps];
    __shared__ float4 so[kWarps][8];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, grp = tid / 8, c = tid % 8 + 8 * blockIdx.x;
    const int h = blockIdx.y, b = blockIdx.z;
    const int n = (int)pg_splits(pg_len(lens[b], max_len));  // complete, as above
    griddep_wait();
    griddep_launch_dependents();
    if (n <= 1) return;  // written by launch 1
    const int64_t bh = (int64_t)b * Hq + h;
    const float2 *ml = part_ml + bh * S;
    const float4 *po = reinterpret_cast<const float4 *>(part_o + bh * S * D) + c;
    const bool serial = n <= kPgSerial;
    const int start = serial ? (grp == 0 ? 0 : n) : grp, step = serial ? 1 : kPgCombineThreads / 8;
    PgBatch batch;
    batch.load(ml, po, D / 4, start, step, n);
    float m = kNegInf;
    for (int s = tid; s < n; s += kPgCombineThreads) m = fmaxf(m, ml[s].x);
    m = pg_warp_max(m);
    if (lane == 0) red[warp] = m;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int k = 1; k < kWarps; ++k) m = fmaxf(m, red[k]);
    const float ref = m == kNegInf ? 0.0f : m;
    PgFold f;
    f.run(batch, ml, po, D / 4, start, step, n, ref);
    if (serial) {
        if (grp == 0) f.store(out + bh * D + 4 * c);
        return;
    }
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
        f.l = __fadd_rn(f.l, __shfl_xor_sync(0xffffffffu, f.l, o));
        f.o.x = __fadd_rn(f.o.x, __shfl_xor_sync(0xffffffffu, f.o.x, o));
        f.o.y = __fadd_rn(f.o.y, __shfl_xor_sync(0xffffffffu, f.o.y, o));
        f.o.z = __fadd_rn(f.o.z, __shfl_xor_sync(0xffffffffu, f.o.z, o));
        f.o.w = __fadd_rn(f.o.w, __shfl_xor_sync(0xffffffffu, f.o.w, o));
    }
    if (lane < 8) so[warp][lane] = f.o;
    if (lane == 0) sl[warp] = f.l;
    __syncthreads();
    if (tid < 8) {
        f.l = sl[0];
        f.o = so[0][tid];
        for (int w = 1; w < kWarps; ++w) {
            const float4 v = so[w][tid];
            f.l = __fadd_rn(f.l, sl[w]);
            f.o.x = __fadd_rn(f.o.x, v.x);
            f.o.y = __fadd_rn(f.o.y, v.y);
            f.o.z = __fadd_rn(f.o.z, v.z);
            f.o.w = __fadd_rn(f.o.w, v.w);
        }
        f.store(out + bh * D + 4 * c);
    }
}

}  // namespace bi
