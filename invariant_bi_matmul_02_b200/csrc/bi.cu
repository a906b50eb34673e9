// bi.cu -- host side of libbi.so: argument checks, TMA tensor-map encoding and
// stream-ordered launches behind the C ABI declared in include/bi.h.
//
// The library allocates no device memory.  Per device it caches the SM count, the
// address of its status word and the GEMM kernel's shared-memory attribute.  No
// launch decision depends on M except how the work is shared (how many CTAs walk the tile
// list, how many rows there are, how many blocks or warps take a row's or a token's
// pieces), which never changes a row's arithmetic.
#include "bi.h"

#include <algorithm>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstddef>
#include <cstdint>
#include <mutex>

#include "gemm.cuh"
#include "attention.cuh"
#include "gemm_pair.cuh"
#include "paged_attention.cuh"
#include "ptx.cuh"
#include "rope.cuh"
#include "rowops.cuh"
#include "token_logprobs.cuh"

// Per-device status word: 0, or the first error a kernel recorded (BI_ERR_TIMEOUT or BI_ERR_INVALID_ARG).
__device__ int32_t g_bi_status = 0;

namespace {

constexpr uint64_t kWaitLimitNs = 1000ull * 1000ull * 1000ull;  // 1 s per device-side wait
constexpr int kMaxDevices = 64;
constexpr int64_t kI32Max = 2147483647;

struct DeviceState {
    bool ready = false;
    int sms = 0;
    int gemm_clusters_wide = 0;    // CTA pairs of each GEMM configuration that fit on the device at once
    int gemm_clusters_narrow = 0;
    int gemm_clusters_mid = 0;
    int mean_rows_blocks_per_sm = 0;  // co-resident 1024-thread blocks of the persistent mean
    int32_t *status = nullptr;
};

std::mutex g_mu;
DeviceState g_dev[kMaxDevices];

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Opt the decode-attention kernels of head size D into their shared memory.
template <int D>
bi_status attn_smem_opt_in()
{
    const void *fns[4] = {reinterpret_cast<const void *>(bi::decode_attention_split_kernel<1, D>),
                          reinterpret_cast<const void *>(bi::decode_attention_split_kernel<2, D>),
                          reinterpret_cast<const void *>(bi::decode_attention_split_kernel<4, D>),
                          reinterpret_cast<const void *>(bi::decode_attention_split_kernel<8, D>)};
    for (const void *fn : fns)
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bi::kAttnSmem) != cudaSuccess)
            return BI_ERR_CUDA;
    return BI_OK;
}

// Opt the paged decode-attention kernels of head size D and the token log-probability kernels into theirs.
template <int D>
bi_status paged_smem_opt_in()
{
    const void *fns[2] = {reinterpret_cast<const void *>(bi::paged_attention_split_kernel<D, 1>),
                          reinterpret_cast<const void *>(bi::paged_attention_split_kernel<D, 2>)};
    for (const void *fn : fns)
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bi::PgShape<D>::kSmem) != cudaSuccess)
            return BI_ERR_CUDA;
    return BI_OK;
}

// Shared memory of a token_logprobs block that takes `pieces` pieces.
inline size_t token_logprobs_smem(int64_t pieces, int64_t top) { return top > 0 ? (size_t)pieces * bi::kTlThreads * sizeof(uint16_t) : 0; }

// With this much and its own 14.5 KB a block takes more than a quarter of an SM's 228 KB, and less than a third.
constexpr int kTlThirdOfSm = 43 * 1024;
static_assert(kTlThirdOfSm >= bi::kTlMaxPieces * bi::kTlThreads * (int)sizeof(uint16_t), "the longest row's group maxima fit");

bi_status token_logprobs_smem_opt_in()
{
    const void *fns[4] = {reinterpret_cast<const void *>(bi::token_logprobs_kernel<true, true>),
                          reinterpret_cast<const void *>(bi::token_logprobs_kernel<true, false>),
                          reinterpret_cast<const void *>(bi::token_logprobs_kernel<false, true>),
                          reinterpret_cast<const void *>(bi::token_logprobs_kernel<false, false>)};
    for (const void *fn : fns)
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kTlThirdOfSm) != cudaSuccess)
            return BI_ERR_CUDA;
    return BI_OK;
}

// Opt the GEMM configuration T into its shared memory and count the CTA pairs that fit at once.
template <typename T>
bi_status pair_clusters(int sms, int *out)
{
    const void *fn = reinterpret_cast<const void *>(bi::gemm_bf16_pair_kernel<T::kBN, T::kStageK>);
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, T::kSmem) != cudaSuccess)
        return BI_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * sms, 1, 1);
    cfg.blockDim = dim3(bi::kGemmThreads, 1, 1);
    cfg.dynamicSmemBytes = T::kSmem;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) return BI_ERR_CUDA;
    *out = n;
    return BI_OK;
}

bi_status device_state(DeviceState **out)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return BI_ERR_CUDA;
    if (dev < 0 || dev >= kMaxDevices) return BI_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(g_mu);
    DeviceState &d = g_dev[dev];
    if (!d.ready) {
        if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return BI_ERR_CUDA;
        void *sym = nullptr;
        if (cudaGetSymbolAddress(&sym, g_bi_status) != cudaSuccess) return BI_ERR_CUDA;
        d.status = static_cast<int32_t *>(sym);
        if (pair_clusters<bi::WideTile>(d.sms, &d.gemm_clusters_wide) != BI_OK ||
            pair_clusters<bi::NarrowTile>(d.sms, &d.gemm_clusters_narrow) != BI_OK ||
            pair_clusters<bi::MidTile>(d.sms, &d.gemm_clusters_mid) != BI_OK)
            return BI_ERR_CUDA;
        if (attn_smem_opt_in<64>() != BI_OK || attn_smem_opt_in<128>() != BI_OK) return BI_ERR_CUDA;
        if (paged_smem_opt_in<64>() != BI_OK || paged_smem_opt_in<128>() != BI_OK) return BI_ERR_CUDA;
        if (token_logprobs_smem_opt_in() != BI_OK) return BI_ERR_CUDA;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&d.mean_rows_blocks_per_sm, bi::mean_rows_kernel,
                                                          bi::kMeanRowsThreads, 0) !=
                cudaSuccess ||
            d.mean_rows_blocks_per_sm < 1)
            return BI_ERR_CUDA;
        if (cudaFuncSetAttribute(bi::log_softmax_stream_kernel<true>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, bi::kLsmSmem) != cudaSuccess ||
            cudaFuncSetAttribute(bi::log_softmax_stream_kernel<false>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, bi::kLsmSmem) != cudaSuccess ||
            cudaFuncSetAttribute(bi::log_softmax_cluster_kernel<true>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, bi::kClSliceBytesMax) != cudaSuccess ||
            cudaFuncSetAttribute(bi::log_softmax_cluster_kernel<false>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, bi::kClSliceBytesMax) != cudaSuccess)
            return BI_ERR_CUDA;
        if (bi::kRowCluster > 8 &&  // clusters above the portable size must be allowed per kernel
            (cudaFuncSetAttribute(bi::log_softmax_cluster_kernel<true>,
                                  cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
             cudaFuncSetAttribute(bi::log_softmax_cluster_kernel<false>,
                                  cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess))
            return BI_ERR_CUDA;
        d.ready = true;
    }
    *out = &d;
    return BI_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// 2-D bf16 tensor map over a row-major matrix: `inner` contiguous elements per row,
// `outer` rows `ld` elements apart, box inner x outer, 128-byte swizzle, zero fill.
bi_status encode_map_uncached(CUtensorMap *map, const void *base, uint64_t inner, uint64_t outer, uint64_t ld,
                              uint32_t box_inner, uint32_t box_outer)
{
    auto enc = tensor_map_encoder();
    if (!enc) return BI_ERR_CUDA;
    const cuuint64_t dims[2] = {inner, outer};
    const cuuint64_t strides[1] = {ld * 2};
    const cuuint32_t box[2] = {box_inner, box_outer};
    const cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides,
                     box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? BI_OK : BI_ERR_CUDA;
}

// Encoded tensor maps, keyed by everything the encoding reads (base address, extents, row
// stride, box).  A map is a pure function of its key, so a hit returns exactly the map a fresh
// encoding would; a freed and re-allocated buffer at the same address with the same shape gets
// the same, still correct, map.  Direct-mapped with kMapCacheSlots slots under one mutex: a
// colliding key replaces the slot.  A GEMM call looks up two maps.
struct MapKey {
    uint64_t base, inner, outer, ld;
    uint32_t box_inner, box_outer;
    bool operator==(const MapKey &o) const
    {
        return base == o.base && inner == o.inner && outer == o.outer && ld == o.ld &&
               box_inner == o.box_inner && box_outer == o.box_outer;
    }
};
struct MapSlot {
    bool used = false;
    MapKey key{};
    CUtensorMap map{};
};
constexpr int kMapCacheSlots = 256;
std::mutex g_map_mu;
MapSlot g_map_cache[kMapCacheSlots];
uint64_t g_map_hits = 0, g_map_misses = 0;

inline uint32_t map_slot(const MapKey &k)
{
    uint64_t h = 0x9E3779B97F4A7C15ull;
    for (uint64_t v : {k.base, k.inner, k.outer, k.ld, (uint64_t)k.box_inner << 32 | k.box_outer}) {
        h ^= v + 0x9E3779B97F4A7C15ull + (h << 6) + (h >> 2);
    }
    return (uint32_t)(h % kMapCacheSlots);
}

bi_status encode_map(CUtensorMap *map, const void *base, uint64_t inner, uint64_t outer, uint64_t ld,
                     uint32_t box_inner, uint32_t box_outer)
{
    const MapKey key{reinterpret_cast<uint64_t>(base), inner, outer, ld, box_inner, box_outer};
    const uint32_t slot = map_slot(key);
    std::lock_guard<std::mutex> lock(g_map_mu);
    MapSlot &e = g_map_cache[slot];
    if (e.used && e.key == key) {
        ++g_map_hits;
        *map = e.map;
        return BI_OK;
    }
    ++g_map_misses;
    const bi_status st = encode_map_uncached(map, base, inner, outer, ld, box_inner, box_outer);
    if (st != BI_OK) return st;
    e.used = true;
    e.key = key;
    e.map = *map;
    return BI_OK;
}

// 4-D bf16 tensor map over a decode cache [B, Lmax, Hkv, D] (row-major): dims innermost first
// (D, Hkv, Lmax, B); box 64 d x 1 head x 128 tokens x 1 sequence, 128-byte swizzle, zero fill
// past Lmax.
bi_status encode_kv_map(CUtensorMap *map, const void *base, uint64_t D, uint64_t Hkv, uint64_t Lmax, uint64_t B)
{
    auto enc = tensor_map_encoder();
    if (!enc) return BI_ERR_CUDA;
    const cuuint64_t dims[4] = {D, Hkv, Lmax, B};
    const cuuint64_t strides[3] = {D * 2, Hkv * D * 2, Lmax * Hkv * D * 2};
    const cuuint32_t box[4] = {64, 1, (cuuint32_t)bi::kAttnChunk, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? BI_OK : BI_ERR_CUDA;
}

// 4-D bf16 tensor map over one side of a paged cache: entries innermost, pages outermost, heads and rows
// of a page between them by ascending stride (heads_inner: heads first); box 64 entries x `box` rows of
// one head of one page, 128-byte swizzle, zero fill outside.  A dimension of one entry is never
// stepped over, so its stride is replaced by one the encoder accepts.
bi_status encode_page_map(CUtensorMap *map, const void *base, const bi_paged_cache &c, bool heads_inner, uint32_t box)
{
    auto enc = tensor_map_encoder();
    if (!enc) return BI_ERR_CUDA;
    const uint64_t D = (uint64_t)c.head_dim;
    const uint64_t head = c.heads > 1 ? (uint64_t)c.head_stride : D;
    const uint64_t token = c.page_size > 1 ? (uint64_t)c.token_stride : D;
    const uint64_t page = c.pages > 1 ? (uint64_t)c.page_stride : D;
    const uint64_t heads = (uint64_t)c.heads, rows = (uint64_t)c.page_size;
    const cuuint64_t dims[4] = {D, heads_inner ? heads : rows, heads_inner ? rows : heads, (uint64_t)c.pages};
    const cuuint64_t strides[3] = {2 * (heads_inner ? head : token), 2 * (heads_inner ? token : head), 2 * page};
    const cuuint32_t boxes[4] = {64, heads_inner ? 1 : box, heads_inner ? box : 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, boxes, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? BI_OK : BI_ERR_CUDA;
}

// Launch `kernel` on `s` and report the launch's own result.  cudaLaunchKernelEx returns the
// error of this launch, so a failure left behind by some other library's launch on this thread
// is neither reported as ours nor cleared.
template <typename... KArgs, typename... Args>
bi_status launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = nullptr;
    cfg.numAttrs = 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? BI_OK : BI_ERR_CUDA;
}

// Launch `kernel` with programmatic stream serialization: it may start while the previous kernel
// in the stream finishes, and waits (griddep_wait) for it before touching global memory.
template <typename... KArgs, typename... Args>
bi_status launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? BI_OK : BI_ERR_CUDA;
}

// launch_pdl with clusters of `cluster` blocks.
template <typename... KArgs, typename... Args>
bi_status launch_pdl_clusters(void (*kernel)(KArgs...), unsigned grid, unsigned block, unsigned cluster, size_t smem,
                              cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(block, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attrs[2]{};
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = cluster;
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? BI_OK : BI_ERR_CUDA;
}

// Launch `kernel` with one cluster of bi::kRowCluster CTAs per row, rows on grid.y in slices of
// at most 65535; the kernel takes the slice's first row as its `row0` argument.
template <typename... KArgs, typename... Args>
bi_status launch_row_clusters(void (*kernel)(KArgs...), int64_t M, size_t smem, cudaStream_t s, Args... args)
{
    for (int64_t row0 = 0; row0 < M; row0 += 65535) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(bi::kRowCluster, (unsigned)(M - row0 < 65535 ? M - row0 : 65535), 1);
        cfg.blockDim = dim3(bi::kClThreads, 1, 1);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = bi::kRowCluster;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, kernel, args..., row0) != cudaSuccess) return BI_ERR_CUDA;
    }
    return BI_OK;
}

// N is the number of output columns.  With fuse_silu, B holds 2N rows ([gate; up]) and
// the output is silu(A . gate^T) * (A . up^T).
// Launch 1 (group size G chosen at run time, head size D) and launch 2 of the decode attention.
template <int D>
bi_status launch_attention(int64_t group, dim3 grid, size_t smem, cudaStream_t s, const CUtensorMap &tm_k,
                           const CUtensorMap &tm_v, const bi::AttnParams &p, const int32_t *seq_lens, void *out,
                           int64_t B)
{
    bi_status st;
    switch (group) {
    case 1: st = launch_pdl(bi::decode_attention_split_kernel<1, D>, grid, dim3(bi::kAttnThreads), smem, s, tm_k, tm_v, p); break;
    case 2: st = launch_pdl(bi::decode_attention_split_kernel<2, D>, grid, dim3(bi::kAttnThreads), smem, s, tm_k, tm_v, p); break;
    case 4: st = launch_pdl(bi::decode_attention_split_kernel<4, D>, grid, dim3(bi::kAttnThreads), smem, s, tm_k, tm_v, p); break;
    case 8: st = launch_pdl(bi::decode_attention_split_kernel<8, D>, grid, dim3(bi::kAttnThreads), smem, s, tm_k, tm_v, p); break;
    default: return BI_ERR_UNSUPPORTED;
    }
    if (st != BI_OK || p.out != nullptr) return st;  // one split per sequence: launch 1 wrote out
    return launch_pdl(bi::decode_attention_combine_kernel<D>, dim3((unsigned)p.Hq, (unsigned)B), dim3(D), 0, s,
                      static_cast<const float2 *>(p.part_ms), static_cast<const float *>(p.part_acc), seq_lens,
                      static_cast<__nv_bfloat16 *>(out), (int)p.Hq, p.Lmax);
}

// Tile counts, tensor maps and the launch of the pair GEMM in configuration T.
template <typename T>
bi_status launch_pair(bi::GemmParams p, const void *A, int64_t lda, const void *B, int64_t ldb, int b_layout,
                      int64_t b_rows, int pairs, cudaStream_t s)
{
    // [K, N] weights are staged in 64-column groups per CTA; pair_config never sends them to a
    // tile whose half-width is not a multiple of 64.
    if (b_layout == BI_B_KN && !T::kKNOk) return BI_ERR_UNSUPPORTED;
    const int64_t M = p.M, N = p.N, K = p.K;
    p.m_blocks = (int32_t)((M + bi::kPairBM - 1) / bi::kPairBM);
    p.n_blocks = (int32_t)(p.fuse_silu ? (N + T::kHalf - 1) / T::kHalf : (N + T::kBN - 1) / T::kBN);
    p.k_blocks = (int32_t)((K + T::kStageK - 1) / T::kStageK);
    const int64_t tiles = (int64_t)p.m_blocks * p.n_blocks;
    if (tiles > kI32Max) return BI_ERR_UNSUPPORTED;

    CUtensorMap tm_a, tm_b;
    // The A box copies the rows that exist: M rounded up to 8, at most the CTA's 128.  The tile,
    // the MMA shape and every element's K order are the same for every M.
    p.a_box_rows = (int32_t)(M >= bi::kBM ? bi::kBM : (M + 7) / 8 * 8);
    bi_status st = encode_map(&tm_a, A, (uint64_t)K, (uint64_t)M, (uint64_t)lda, bi::kBK, (uint32_t)p.a_box_rows);
    if (st != BI_OK) return st;
    if (b_layout == BI_B_NK)
        st = encode_map(&tm_b, B, (uint64_t)K, (uint64_t)b_rows, (uint64_t)ldb, bi::kBK, (uint32_t)T::kHalf);
    else
        st = encode_map(&tm_b, B, (uint64_t)b_rows, (uint64_t)K, (uint64_t)ldb, 64, (uint32_t)T::kStageK);
    if (st != BI_OK) return st;

    const int grid = 2 * (int)(tiles < pairs ? tiles : pairs);
    return launch_pdl(bi::gemm_bf16_pair_kernel<T::kBN, T::kStageK>, dim3(grid), dim3(bi::kGemmThreads),
                      (size_t)T::kSmem, s, tm_a, tm_b, p);
}

bi_status gemm_common(const void *input, int64_t ld_input, int addend_mode, const void *A, int64_t lda,
                      const void *B, int64_t ldb, int b_layout, void *C, int64_t ldc, int c_dtype,
                      int64_t M, int64_t N, int64_t K, void *stream, int fuse_silu = 0)
{
    if (M < 0 || N < 0 || K < 0) return BI_ERR_INVALID_ARG;
    if (b_layout != BI_B_KN && b_layout != BI_B_NK) return BI_ERR_INVALID_ARG;
    if (c_dtype != BI_BF16 && c_dtype != BI_F32) return BI_ERR_INVALID_ARG;
    if (M > kI32Max || (fuse_silu ? 2 * N : N) > kI32Max || K > kI32Max) return BI_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return BI_OK;
    const int64_t b_rows = fuse_silu ? 2 * N : N;  // extent of B along the output dimension
    if (!C || ldc < N) return BI_ERR_INVALID_ARG;
    if (addend_mode != bi::kAddNone) {
        if (!input || ld_input < 0 || (ld_input != 0 && ld_input < N)) return BI_ERR_INVALID_ARG;
        if (!aligned16(input) || ld_input % 8 != 0) return BI_ERR_ALIGNMENT;
    }
    const bool c_f32 = c_dtype == BI_F32;
    if (!aligned16(C) || ldc % (c_f32 ? 4 : 8) != 0) return BI_ERR_ALIGNMENT;
    if (K > 0) {
        if (!A || !B) return BI_ERR_INVALID_ARG;
        if (lda < K || ldb < (b_layout == BI_B_KN ? b_rows : K)) return BI_ERR_INVALID_ARG;
        if (!aligned16(A) || !aligned16(B) || lda % 8 != 0 || ldb % 8 != 0) return BI_ERR_ALIGNMENT;
        // [K, 2F] gate/up weights: the up half starts at column F, the innermost coordinate of its
        // tile loads, which a TMA copy needs at a multiple of 16 bytes (8 bf16 elements).
        if (fuse_silu && b_layout == BI_B_KN && N % 8 != 0) return BI_ERR_ALIGNMENT;
    }

    DeviceState *dev = nullptr;
    bi_status st = device_state(&dev);
    if (st != BI_OK) return st;

    bi::GemmParams p{};
    p.M = (int32_t)M;
    p.N = (int32_t)N;
    p.K = (int32_t)K;
    p.fuse_silu = fuse_silu;
    p.b_mn_major = b_layout == BI_B_KN ? 1 : 0;
    p.c_f32 = c_f32 ? 1 : 0;
    p.addend_mode = addend_mode;
    p.ldc = ldc;
    p.ld_addend = ld_input;
    p.C = C;
    p.addend = static_cast<const __nv_bfloat16 *>(input);
    p.status = dev->status;
    p.wait_limit_ns = kWaitLimitNs;
    cudaStream_t s = static_cast<cudaStream_t>(stream);

    if (K == 0 && !fuse_silu) {
        const int64_t total = M * N;
        int64_t blocks = (total + 255) / 256;
        if (blocks > (int64_t)dev->sms * 16) blocks = (int64_t)dev->sms * 16;
        return launch(bi::gemm_k0_fill_kernel, dim3((unsigned)blocks), dim3(256), 0, s, p);
    }

    // The tile configuration is a function of the weight alone (its rows and storage); every M of
    // a given weight runs the same one.
    switch (bi::pair_config(b_rows, b_layout == BI_B_NK)) {
    case bi::kPairNarrow:
        return launch_pair<bi::NarrowTile>(p, A, lda, B, ldb, b_layout, b_rows, dev->gemm_clusters_narrow, s);
    case bi::kPairMid:
        return launch_pair<bi::MidTile>(p, A, lda, B, ldb, b_layout, b_rows, dev->gemm_clusters_mid, s);
    default:
        break;
    }
    return launch_pair<bi::WideTile>(p, A, lda, B, ldb, b_layout, b_rows, dev->gemm_clusters_wide, s);
}

__global__ void selftest_wait_kernel(int32_t *status, uint64_t limit_ns)
{
    __shared__ uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        bi::mbar_init(&bar, 1);
        abort_flag = 0;
        bi::fence_mbar_init();
    }
    __syncthreads();
    // Phase 0 of `bar` never completes: nothing arrives on it.
    if (threadIdx.x == 0) bi::wait_bounded(&bar, 0, &abort_flag, status, limit_ns);
    __syncthreads();
}

// The two launches of the split log_softmax: per-(row, chunk) partials, then the merge and write.
bi_status split_launches(bool bf16, dim3 grid, cudaStream_t s, const uint8_t *xb, float2 *part, float *y, int64_t V)
{
    bi_status st = bf16 ? launch(bi::log_softmax_split_stats_kernel<true>, grid, dim3(bi::kSplitThreads), 0, s, xb,
                                 part, V)
                        : launch(bi::log_softmax_split_stats_kernel<false>, grid, dim3(bi::kSplitThreads), 0, s, xb,
                                 part, V);
    if (st != BI_OK) return st;
    return bf16 ? launch(bi::log_softmax_split_write_kernel<true>, grid, dim3(bi::kSplitThreads), 0, s, xb,
                         static_cast<const float2 *>(part), y, V)
                : launch(bi::log_softmax_split_write_kernel<false>, grid, dim3(bi::kSplitThreads), 0, s, xb,
                         static_cast<const float2 *>(part), y, V);
}

// Whether the heads of a strided [.., heads, D] tensor can be moved in pieces of W entries of `entry` bytes.
inline bool strided_pieces(int64_t W, int64_t entry, const void *p, int64_t s0, int64_t s1)
{
    return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(W * entry - 1)) == 0 && s0 % W == 0 && s1 % W == 0;
}

// The widest piece (in bytes) that entries first .. first + n - 1 of every head can be copied in, between tensors
// that `fits` (pieces of W entries) accepts; 0 for no entries.
template <typename Fits>
int copy_piece(int64_t first, int64_t n, int64_t entry, Fits fits)
{
    if (n == 0) return 0;
    for (int64_t W = 16 / entry; W > 1; W /= 2)
        if (first % W == 0 && n % W == 0 && fits(W)) return (int)(W * entry);
    return (int)entry;
}

// Warps that share a token's heads in the rotation kernels: one where the tokens alone fill the GPU (the
// angles are then worked out once per token), more for fewer tokens, as long as each has heads to take
// (`steps`: head groups of a token).  Every head's arithmetic is the same.
inline int rope_shares(int64_t T, int64_t steps, int sms)
{
    const int64_t want = ((int64_t)sms * 16 + T - 1) / T;  // 16 warps an SM
    return (int)(want < 1 ? 1 : want > steps ? steps : want);
}
inline int64_t rope_steps(int64_t H, int64_t D, int64_t R, int64_t W)
{
    const int64_t units = R / (2 * W), heads = units > 0 && units < 32 ? 32 / units : 1;
    const int64_t turned = units > 0 ? (H + heads - 1) / heads : 0, copied = H * (D - R) / (32 * bi::kRopeCopies);
    return turned > copied ? turned : copied > 0 ? copied : 1;
}

// The launch: warps that share a token, and how many of its steps a warp has in shared memory at once (0 where
// the walk is not streamed).
struct RopeLaunch {
    int shares, stages;
    dim3 grid;
    size_t smem;
    RopeLaunch(int64_t T, int64_t steps, bool streamed, int R, int sms, int resident = bi::kRopeBlocks)
    {
        steps = std::max<int64_t>(steps, 1);
        shares = rope_shares(T, steps, sms);
        const int64_t mine = (steps + shares - 1) / shares;
        stages = !streamed ? 0 : (int)(mine < bi::kRopeStages ? mine : bi::kRopeStages);
        grid = dim3((unsigned)((T * shares + bi::kRopeWarps - 1) / bi::kRopeWarps));
        smem = (size_t)bi::kRopeWarps * (stages * 1024 + R * sizeof(float));
        // Launched while the kernel before it still holds places, a grid that fits the GPU at once would sit unevenly, up to
        // `resident` blocks on one SM and few on another.  A request for more shared memory than an SM has for one block
        // above its share keeps the blocks apart (512 tokens appended 6.6 us without, 5.5 with; 3001 tokens of 13 heads
        // of 96 fp32 turned 7.6 and 7.1; staged, with up to kRopeStagedBlocks: 2048 tokens of 32 heads of 80, 20 turned,
        // 6.8 and 5.6, 4000 of 19 of 192, 74 turned in place, 11.4 and 9.1).  Fewer than four a SM would ask for more than
        // 48 KB a block.
        const int64_t per_sm = ((int64_t)grid.x + sms - 1) / sms;
        if (per_sm >= 4 && per_sm < resident)
            smem = std::max<size_t>(smem, (size_t)(228 * 1024 / (per_sm + 1) - 1024 + 512));  // 1 KB a block is the system's
    }
};

template <typename E, int W, bool STREAM>
bi_status launch_rope(const bi::RopeParams &p, bool half, const RopeLaunch &l, cudaStream_t s)
{
    const dim3 block(bi::kRopeThreads);
    return half ? launch_pdl(bi::rope_kernel<E, W, true, STREAM>, l.grid, block, l.smem, s, p, l.shares, l.stages)
                : launch_pdl(bi::rope_kernel<E, W, false, STREAM>, l.grid, block, l.smem, s, p, l.shares, l.stages);
}

template <typename E>
bi_status launch_rope_staged(const bi::RopeParams &p, bool half, const RopeLaunch &l, cudaStream_t s)
{
    const dim3 block(bi::kRopeThreads);
    return half ? launch_pdl(bi::rope_staged_kernel<E, true>, l.grid, block, l.smem, s, p, l.shares, l.stages)
                : launch_pdl(bi::rope_staged_kernel<E, false>, l.grid, block, l.smem, s, p, l.shares, l.stages);
}

template <typename E, int W>
bi_status launch_rope(const bi::RopeParams &p, bool half, int sms, cudaStream_t s)
{
    if constexpr (sizeof(bi::Piece<E, W>) == 16) {
        // A streamed walk costs 0.3 us more to begin and pays for it where warps have many steps to take (streamed and
        // through registers: one token 2.4 and 2.1, 1024 tokens of 40 heads 6.0 and 5.2, 1200 of 8 heads 3.5 and 3.1;
        // 1500 of 40 heads 7.3 and 7.5, 2048 10.2 and 11.1, 4096 of 16 heads 7.8 and 10.2) or where it takes copied
        // entries along (64 tokens, half of each head turned: 2.6 and 3.1).
        const int rest = p.copy_piece == 16 ? p.D - p.R : 0;
        const RopeLaunch l(p.T, bi::RopeSteps<W>(p.R, rest).steps(p.H), true, p.R, sms);
        if (rest > 0 || p.T >= 12 * sms) return launch_rope<E, W, true>(p, half, l, s);
    }
    return launch_rope<E, W, false>(p, half, RopeLaunch(p.T, rope_steps(p.H, p.D, p.R, W), false, p.R, sms), s);
}

template <int W>
bi_status launch_append(const bi::AppendParams &p, bool half, int sms, cudaStream_t s)
{
    const bi::RopeSteps<W> shape(p.R, bi::append_rest<W>(p));
    const int64_t Hq = p.q ? p.Hq : 0;
    const bool streamed = W == 8 && shape.units > 0;
    const int64_t steps =
        streamed ? (int64_t)shape.steps((int)Hq) + shape.steps(p.Hkv) + (bi::append_values<W>(p) ? shape.steps(p.Hkv) : 0)
                 : rope_steps(Hq + p.Hkv, p.D, p.R, W);
    const RopeLaunch l(p.T, steps, streamed, p.R, sms);
    const dim3 block(bi::kRopeThreads);
    return half ? launch_pdl(bi::paged_append_kernel<W, true>, l.grid, block, l.smem, s, p, l.shares, l.stages)
                : launch_pdl(bi::paged_append_kernel<W, false>, l.grid, block, l.smem, s, p, l.shares, l.stages);
}

bi_status launch_append_staged(const bi::AppendParams &p, bool half, int sms, cudaStream_t s)
{
    const int64_t heads = 64 / p.pieces, Hq = p.q ? p.Hq : 0;
    const RopeLaunch l(p.T, (Hq + heads - 1) / heads + 2 * ((p.Hkv + heads - 1) / heads), true, p.R, sms,
                       bi::kRopeStagedBlocks);
    const dim3 block(bi::kRopeThreads);
    return half ? launch_pdl(bi::paged_append_kernel<8, true, true>, l.grid, block, l.smem, s, p, l.shares, l.stages)
                : launch_pdl(bi::paged_append_kernel<8, false, true>, l.grid, block, l.smem, s, p, l.shares, l.stages);
}

// A cache description that the paged entry points take.
bi_status check_cache(const bi_paged_cache *c)
{
    if (!c || !c->k || !c->v) return BI_ERR_INVALID_ARG;
    if (c->pages <= 0 || c->page_size <= 0 || c->heads <= 0 || c->head_dim <= 0) return BI_ERR_INVALID_ARG;
    if (c->pages > kI32Max || c->page_size > kI32Max || c->heads > 65535 || c->head_dim > bi::kRopeMaxDim)
        return BI_ERR_UNSUPPORTED;
    const int64_t D = c->head_dim, limit = int64_t(1) << 39;  // 2^40 bytes: a tensor map's largest stride
    if (c->page_stride < 0 || c->token_stride < 0 || c->head_stride < 0) return BI_ERR_INVALID_ARG;
    if ((c->pages > 1 && c->page_stride < D) || (c->page_size > 1 && c->token_stride < D) ||
        (c->heads > 1 && c->head_stride < D))
        return BI_ERR_INVALID_ARG;
    if (c->page_stride >= limit || c->token_stride >= limit || c->head_stride >= limit) return BI_ERR_UNSUPPORTED;
    if (!aligned16(c->k) || !aligned16(c->v) || (c->pages > 1 && c->page_stride % 8) ||
        (c->page_size > 1 && c->token_stride % 8) || (c->heads > 1 && c->head_stride % 8))
        return BI_ERR_ALIGNMENT;
    return BI_OK;
}

template <int D, int NT>
bi_status launch_paged(dim3 grid, cudaStream_t s, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                       const bi::PgParams &p)
{
    const bi_status st = launch_pdl(bi::paged_attention_split_kernel<D, NT>, grid, dim3(bi::kPgThreads),
                                    (size_t)bi::PgShape<D>::kSmem, s, tm_k, tm_v, p);
    if (st != BI_OK || p.S == 1) return st;  // one split per sequence: launch 1 wrote out
    const float2 *ml = p.part_ml;
    const float *o = p.part_o;
    if (p.S > bi::kPgSerial)
        return launch_pdl(bi::paged_attention_combine_long_kernel<D>, dim3(D / 32, (unsigned)p.Hq, (unsigned)p.B),
                          dim3(bi::kPgCombineThreads), 0, s, ml, o, p.lens, p.out, (int)p.Hq, (int)p.S, (int)p.max_len);
    const int rows = p.B * p.Hq, per_block = bi::kPgCombineThreads / (D / 4);
    return launch_pdl(bi::paged_attention_combine_kernel<D>, dim3((unsigned)((rows + per_block - 1) / per_block)),
                      dim3(bi::kPgCombineThreads), 0, s, ml, o, p.lens, p.out, (int)p.Hq, (int)p.S, (int)p.max_len, rows);
}

inline unsigned elementwise_blocks(int64_t work, int sms)
{
    int64_t blocks = (work + 255) / 256;
    const int64_t cap = (int64_t)sms * 8;
    return (unsigned)(blocks < 1 ? 1 : (blocks > cap ? cap : blocks));
}

}  // namespace

extern "C" {

bi_status bi_matmul(const void *A, int64_t lda, const void *B, int64_t ldb, bi_b_layout b_layout,
                    void *C, int64_t ldc, bi_dtype c_dtype, int64_t M, int64_t N, int64_t K,
                    void *stream)
{
    return gemm_common(nullptr, 0, bi::kAddNone, A, lda, B, ldb, b_layout, C, ldc, c_dtype, M, N, K,
                       stream);
}

bi_status bi_addmm(const void *input, int64_t ld_input, const void *A, int64_t lda, const void *B,
                   int64_t ldb, bi_b_layout b_layout, void *C, int64_t ldc, bi_dtype c_dtype,
                   int64_t M, int64_t N, int64_t K, void *stream)
{
    return gemm_common(input, ld_input, ld_input == 0 ? bi::kAddBias : bi::kAddMatrix, A, lda, B, ldb,
                       b_layout, C, ldc, c_dtype, M, N, K, stream);
}

bi_status bi_matmul_silu_mul(const void *A, int64_t lda, const void *B, int64_t ldb,
                             bi_b_layout b_layout, void *H, int64_t ldh, int64_t M, int64_t F, int64_t K,
                             void *stream)
{
    if (K == 0)  // empty products: silu(0) * 0 = 0
        return gemm_common(nullptr, 0, bi::kAddNone, A, lda, B, ldb, b_layout, H, ldh, BI_BF16, M, F, 0,
                           stream, 0);
    return gemm_common(nullptr, 0, bi::kAddNone, A, lda, B, ldb, b_layout, H, ldh, BI_BF16, M, F, K, stream,
                       1);
}

bi_status bi_rmsnorm(const void *x, const void *w, void *y, int64_t M, int64_t H, float eps,
                     void *stream)
{
    if (M < 0 || H < 0 || !(eps >= 0.0f)) return BI_ERR_INVALID_ARG;
    if (M > kI32Max || H > kI32Max) return BI_ERR_UNSUPPORTED;
    if (M == 0) return BI_OK;
    if (H == 0 || !x || !w || !y) return BI_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int T = bi::rmsnorm_threads(H);
    bi_status st = BI_OK;
    if (H % 8 == 0) {
        if (!aligned16(x) || !aligned16(w) || !aligned16(y)) return BI_ERR_ALIGNMENT;
        const int64_t cpt = (H / 8 + T - 1) / T;
        const uint4 *xv = static_cast<const uint4 *>(x);
        const uint4 *wv = static_cast<const uint4 *>(w);
        uint4 *yv = static_cast<uint4 *>(y);
        switch (cpt) {
        case 1: st = launch_pdl(bi::rmsnorm_vec_kernel<1>, dim3((unsigned)M), dim3(T), 0, s, xv, wv, yv, H, eps); break;
        case 2: st = launch_pdl(bi::rmsnorm_vec_kernel<2>, dim3((unsigned)M), dim3(T), 0, s, xv, wv, yv, H, eps); break;
        case 3: st = launch_pdl(bi::rmsnorm_vec_kernel<3>, dim3((unsigned)M), dim3(T), 0, s, xv, wv, yv, H, eps); break;
        case 4: st = launch_pdl(bi::rmsnorm_vec_kernel<4>, dim3((unsigned)M), dim3(T), 0, s, xv, wv, yv, H, eps); break;
        default:
            st = launch(bi::rmsnorm_scalar_kernel, dim3((unsigned)M), dim3(T), 0, s,
                        static_cast<const __nv_bfloat16 *>(x), static_cast<const __nv_bfloat16 *>(w),
                        static_cast<__nv_bfloat16 *>(y), H, eps);
        }
        return st;
    }
    return launch(bi::rmsnorm_scalar_kernel, dim3((unsigned)M), dim3(T), 0, s,
                  static_cast<const __nv_bfloat16 *>(x), static_cast<const __nv_bfloat16 *>(w),
                  static_cast<__nv_bfloat16 *>(y), H, eps);
}

bi_status bi_mean(const float *x, float *y, int64_t M, int64_t H, void *stream)
{
    if (M < 0 || H < 0) return BI_ERR_INVALID_ARG;
    if (M > kI32Max || H > kI32Max) return BI_ERR_UNSUPPORTED;
    if (M == 0) return BI_OK;
    if (H == 0 || !x || !y) return BI_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int T = bi::mean_threads(H);
    bi_status st = BI_OK;
    if (H % 4 == 0) {
        if (!aligned16(x)) return BI_ERR_ALIGNMENT;
        if (H / 4 >= 8 * (int64_t)T && T == bi::kMeanRowsThreads) {
            DeviceState *dev = nullptr;
            st = device_state(&dev);
            if (st != BI_OK) return st;
            const int64_t fit = (int64_t)dev->sms * dev->mean_rows_blocks_per_sm;
            st = launch_pdl(bi::mean_rows_kernel, dim3((unsigned)(M < fit ? M : fit)), dim3(T), 0, s,
                            reinterpret_cast<const float4 *>(x), y, H, M);
        } else
            st = launch_pdl(bi::mean_vec_kernel, dim3((unsigned)M), dim3(T), 0, s,
                            reinterpret_cast<const float4 *>(x), y, H);
        return st;
    }
    return launch(bi::mean_scalar_kernel, dim3((unsigned)M), dim3(T), 0, s, x, y, H);
}

bi_status bi_log_softmax(const void *x, bi_dtype x_dtype, float *y, int64_t M, int64_t V, void *stream)
{
    if (M < 0 || V < 0) return BI_ERR_INVALID_ARG;
    if (x_dtype != BI_BF16 && x_dtype != BI_F32) return BI_ERR_INVALID_ARG;
    if (M > kI32Max || V > kI32Max) return BI_ERR_UNSUPPORTED;
    if (M == 0) return BI_OK;
    if (V == 0 || !x || !y) return BI_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int T = bi::log_softmax_threads(V);
    const bool bf16 = x_dtype == BI_BF16;
    const int per = bf16 ? 8 : 4;
    if (V % per == 0) {
        if (!aligned16(x) || !aligned16(y)) return BI_ERR_ALIGNMENT;
        DeviceState *dev = nullptr;
        bi_status st = device_state(&dev);
        if (st != BI_OK) return st;
        const uint8_t *xb = static_cast<const uint8_t *>(x);
        st = bf16 ? launch_pdl(bi::log_softmax_stream_kernel<true>, dim3((unsigned)M), dim3(bi::kLsmThreads),
                               (size_t)bi::kLsmSmem, s, xb, y, V, dev->status, kWaitLimitNs)
                  : launch_pdl(bi::log_softmax_stream_kernel<false>, dim3((unsigned)M), dim3(bi::kLsmThreads),
                               (size_t)bi::kLsmSmem, s, xb, y, V, dev->status, kWaitLimitNs);
        return st;
    }
    return bf16 ? launch(bi::log_softmax_scalar_kernel<true>, dim3((unsigned)M), dim3(T), 0, s, x, y, V)
                : launch(bi::log_softmax_scalar_kernel<false>, dim3((unsigned)M), dim3(T), 0, s, x, y, V);
}

bi_status bi_log_softmax_cluster(const void *x, bi_dtype x_dtype, float *y, int64_t M, int64_t V, void *stream)
{
    if (M < 0 || V < 0) return BI_ERR_INVALID_ARG;
    if (x_dtype != BI_BF16 && x_dtype != BI_F32) return BI_ERR_INVALID_ARG;
    if (M > kI32Max || V > kI32Max) return BI_ERR_UNSUPPORTED;
    if (M == 0) return BI_OK;
    if (V == 0 || !x || !y) return BI_ERR_INVALID_ARG;
    const bool bf16 = x_dtype == BI_BF16;
    const int elem = bf16 ? 2 : 4;
    const int64_t slice_bytes = bi::cluster_slice(V) * elem;
    if (V % (bf16 ? 8 : 4) != 0 || V * elem < bi::kClusterRowBytes || slice_bytes > bi::kClSliceBytesMax)
        return BI_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(y)) return BI_ERR_ALIGNMENT;
    DeviceState *dev = nullptr;
    bi_status st = device_state(&dev);
    if (st != BI_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const uint8_t *xb = static_cast<const uint8_t *>(x);
    st = bf16 ? launch_row_clusters(bi::log_softmax_cluster_kernel<true>, M, (size_t)slice_bytes, s, xb, y, V,
                                    dev->status, kWaitLimitNs)
              : launch_row_clusters(bi::log_softmax_cluster_kernel<false>, M, (size_t)slice_bytes, s, xb, y, V,
                                    dev->status, kWaitLimitNs);
    return st;
}

size_t bi_log_softmax_split_scratch_bytes(int64_t M, int64_t V)
{
    if (M <= 0 || V <= 0) return 0;
    return (size_t)M * (size_t)bi::split_chunks(V) * sizeof(float2);
}

bi_status bi_log_softmax_split(const void *x, bi_dtype x_dtype, float *y, int64_t M, int64_t V, void *scratch,
                               size_t scratch_bytes, void *stream)
{
    if (M < 0 || V < 0) return BI_ERR_INVALID_ARG;
    if (x_dtype != BI_BF16 && x_dtype != BI_F32) return BI_ERR_INVALID_ARG;
    if (M > 65535 || V > kI32Max) return BI_ERR_UNSUPPORTED;  // rows on grid.y
    if (M == 0) return BI_OK;
    if (V == 0 || !x || !y || !scratch) return BI_ERR_INVALID_ARG;
    if (V % 8 != 0) return BI_ERR_UNSUPPORTED;
    if (scratch_bytes < bi_log_softmax_split_scratch_bytes(M, V)) return BI_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(y) || !aligned16(scratch)) return BI_ERR_ALIGNMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)bi::split_chunks(V), (unsigned)M);
    const uint8_t *xb = static_cast<const uint8_t *>(x);
    float2 *part = static_cast<float2 *>(scratch);
    return split_launches(x_dtype == BI_BF16, grid, s, xb, part, y, V);
}

}  // extern "C"

// ---------------------------------------------------------------------------------------------
// Allocation-free split log_softmax.
//
// Some callers cannot hand the library a scratch buffer because they cannot allocate device
// memory when they call it: code that runs under a memory budget fixed at start-up (every
// byte already reserved by a pool it does not own), plugins living inside a host framework
// that controls all device allocation, or callers on a hot path where a cudaMalloc's
// implicit synchronisation is not acceptable.  For them the partials of the split path live
// in this file-scope device array.  It has a fixed size and is part of the module image, so
// every GPU that loads libbi.so holds it until the process exits, and no call allocates.
namespace {

constexpr int64_t kNoAllocPartials = 65536;  // (row, chunk) partials: 512 KiB per device
static __device__ __align__(256) float2 g_noalloc_partials[kNoAllocPartials];

std::mutex g_noalloc_mu;
float2 *g_noalloc_ptr[kMaxDevices] = {};

// Device address of g_noalloc_partials on the current device.  In host code the array's name
// only stands in for the symbol, so its address is looked up once per device, with that device
// current, and cached.
bi_status noalloc_partials(float2 **out)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return BI_ERR_CUDA;
    if (dev < 0 || dev >= kMaxDevices) return BI_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(g_noalloc_mu);
    if (!g_noalloc_ptr[dev]) {
        void *p = nullptr;
        if (cudaGetSymbolAddress(&p, g_noalloc_partials) != cudaSuccess || !p) return BI_ERR_CUDA;
        g_noalloc_ptr[dev] = static_cast<float2 *>(p);
    }
    *out = g_noalloc_ptr[dev];
    return BI_OK;
}

}  // namespace

extern "C" {

bi_status bi_log_softmax_split_noalloc(const void *x, bi_dtype x_dtype, float *y, int64_t M, int64_t V,
                                       void *stream)
{
    if (M < 0 || V < 0) return BI_ERR_INVALID_ARG;
    if (x_dtype != BI_BF16 && x_dtype != BI_F32) return BI_ERR_INVALID_ARG;
    if (M > 65535 || V > kI32Max) return BI_ERR_UNSUPPORTED;
    if (M == 0) return BI_OK;
    if (V == 0 || !x || !y) return BI_ERR_INVALID_ARG;
    if (V % 8 != 0) return BI_ERR_UNSUPPORTED;
    if (M * bi::split_chunks(V) > kNoAllocPartials) return BI_ERR_UNSUPPORTED;  // beyond the fixed array
    if (!aligned16(x) || !aligned16(y)) return BI_ERR_ALIGNMENT;
    float2 *part = nullptr;
    bi_status st = noalloc_partials(&part);
    if (st != BI_OK) return st;
    // Launch 1 overwrites every partial that launch 2 reads, so nothing needs clearing.
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)bi::split_chunks(V), (unsigned)M);
    const uint8_t *xb = static_cast<const uint8_t *>(x);
    return split_launches(x_dtype == BI_BF16, grid, s, xb, part, y, V);
}

size_t bi_decode_attention_scratch_bytes(int64_t B, int64_t Hq, int64_t D, int64_t Lmax)
{
    if (B <= 0 || Hq <= 0 || D <= 0 || Lmax <= 0) return 0;
    const size_t parts = (size_t)B * (size_t)Hq * (size_t)bi::attn_splits(Lmax);
    return parts * ((size_t)D * sizeof(float) + sizeof(float2));
}

bi_status bi_decode_attention(const void *q, const void *k_cache, const void *v_cache, const int32_t *seq_lens,
                              void *out, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t Lmax, float scale,
                              void *scratch, size_t scratch_bytes, void *stream)
{
    if (B < 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || Lmax <= 0) return B == 0 ? BI_OK : BI_ERR_INVALID_ARG;
    if (Hq % Hkv != 0) return BI_ERR_INVALID_ARG;
    const int64_t group = Hq / Hkv;
    if ((D != 64 && D != 128) || (group != 1 && group != 2 && group != 4 && group != 8)) return BI_ERR_UNSUPPORTED;
    if (B > 65535 || Hkv > 65535 || Hq > 65535 || bi::attn_splits(Lmax) > kI32Max) return BI_ERR_UNSUPPORTED;
    if (B * Hkv * bi::attn_splits(Lmax) > kI32Max) return BI_ERR_UNSUPPORTED;  // work items are 32-bit indices
    if (B == 0) return BI_OK;
    if (!q || !k_cache || !v_cache || !seq_lens || !out || !scratch) return BI_ERR_INVALID_ARG;
    if (scratch_bytes < bi_decode_attention_scratch_bytes(B, Hq, D, Lmax)) return BI_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(scratch) ||
        (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
        return BI_ERR_ALIGNMENT;
    DeviceState *dev = nullptr;
    bi_status st = device_state(&dev);
    if (st != BI_OK) return st;
    const int64_t S = bi::attn_splits(Lmax);
    CUtensorMap tm_k, tm_v;
    st = encode_kv_map(&tm_k, k_cache, (uint64_t)D, (uint64_t)Hkv, (uint64_t)Lmax, (uint64_t)B);
    if (st != BI_OK) return st;
    st = encode_kv_map(&tm_v, v_cache, (uint64_t)D, (uint64_t)Hkv, (uint64_t)Lmax, (uint64_t)B);
    if (st != BI_OK) return st;
    bi::AttnParams p{};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.lens = seq_lens;
    p.part_acc = static_cast<float *>(scratch);
    p.part_ms = reinterpret_cast<float2 *>(p.part_acc + (size_t)B * Hq * S * D);
    // With Lmax <= 512 every sequence is one split, whose fold launch 1 does itself.
    p.out = S == 1 ? static_cast<__nv_bfloat16 *>(out) : nullptr;
    p.Hq = (int32_t)Hq;
    p.Hkv = (int32_t)Hkv;
    p.B = (int32_t)B;
    p.Lmax = Lmax;
    p.S = S;
    p.scale = scale;
    p.status = dev->status;
    p.wait_limit_ns = kWaitLimitNs;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // Persistent: one CTA per SM walks the (split, kv head, sequence) items; the grid size only
    // decides which CTA computes an item, never an item's arithmetic.
    const int64_t items = B * Hkv * S;
    const dim3 grid((unsigned)(items < dev->sms ? items : dev->sms));
    const size_t smem = (size_t)bi::kAttnSmem;
    // The group size and the head size are properties of the model, not of the batch.
    return D == 64 ? launch_attention<64>(Hq / Hkv, grid, smem, s, tm_k, tm_v, p, seq_lens, out, B)
                   : launch_attention<128>(Hq / Hkv, grid, smem, s, tm_k, tm_v, p, seq_lens, out, B);
}

bi_status bi_silu_mul(const void *gu, void *h, int64_t M, int64_t F, void *stream)
{
    if (M < 0 || F < 0) return BI_ERR_INVALID_ARG;
    if (M > kI32Max || F > kI32Max) return BI_ERR_UNSUPPORTED;
    if (M == 0 || F == 0) return BI_OK;
    if (!gu || !h) return BI_ERR_INVALID_ARG;
    DeviceState *dev = nullptr;
    bi_status st = device_state(&dev);
    if (st != BI_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (F % 8 == 0) {
        if (!aligned16(gu) || !aligned16(h)) return BI_ERR_ALIGNMENT;
        const int64_t work = M * (F / 8);
        return launch(bi::silu_mul_vec_kernel, dim3(elementwise_blocks(work, dev->sms)), dim3(256), 0, s,
                      static_cast<const uint4 *>(gu), static_cast<uint4 *>(h), M, F);
    }
    return launch(bi::silu_mul_scalar_kernel, dim3(elementwise_blocks(M * F, dev->sms)), dim3(256), 0, s,
                  static_cast<const __nv_bfloat16 *>(gu), static_cast<__nv_bfloat16 *>(h), M, F);
}

bi_status bi_rope(const void *x, int64_t x_token_stride, int64_t x_head_stride, void *y, int64_t y_token_stride,
                  int64_t y_head_stride, bi_dtype x_dtype, const int32_t *positions, const double *inv_freq,
                  int64_t T, int64_t H, int64_t D, int64_t R, bi_rope_layout layout, float scale, int inverse,
                  void *stream)
{
    if (T < 0 || H < 0 || D <= 0 || R < 0 || R > D || R % 2 != 0) return BI_ERR_INVALID_ARG;
    if (x_dtype != BI_BF16 && x_dtype != BI_F32) return BI_ERR_INVALID_ARG;
    if (layout != BI_ROPE_HALF && layout != BI_ROPE_INTERLEAVED) return BI_ERR_INVALID_ARG;
    if (T > kI32Max || H > 65535 || D > bi::kRopeMaxDim) return BI_ERR_UNSUPPORTED;
    if (T == 0 || H == 0) return BI_OK;
    if (!x || !y || (R > 0 && (!positions || !inv_freq))) return BI_ERR_INVALID_ARG;
    if (x_token_stride < 0 || x_head_stride < 0 || (T > 1 && y_token_stride < D) || (H > 1 && y_head_stride < D) ||
        y_token_stride < 0 || y_head_stride < 0)
        return BI_ERR_INVALID_ARG;
    if (x == y && ((T > 1 && x_token_stride != y_token_stride) || (H > 1 && x_head_stride != y_head_stride)))
        return BI_ERR_INVALID_ARG;
    const bool bf16 = x_dtype == BI_BF16;
    const uintptr_t type_mask = bf16 ? 1 : 3;
    if ((reinterpret_cast<uintptr_t>(x) & type_mask) || (reinterpret_cast<uintptr_t>(y) & type_mask) ||
        (reinterpret_cast<uintptr_t>(positions) & 3u) || (reinterpret_cast<uintptr_t>(inv_freq) & 7u))
        return BI_ERR_ALIGNMENT;
    DeviceState *dev = nullptr;
    bi_status st = device_state(&dev);
    if (st != BI_OK) return st;
    // Strides of dimensions of one entry are never used.
    const int64_t xt = T > 1 ? x_token_stride : 0, xh = H > 1 ? x_head_stride : 0;
    const int64_t yt = T > 1 ? y_token_stride : 0, yh = H > 1 ? y_head_stride : 0;
    bi::RopeParams p{};
    p.x = x;
    p.y = y;
    p.x_token = xt;
    p.x_head = xh;
    p.y_token = yt;
    p.y_head = yh;
    p.pos = positions;
    p.inv_freq = inv_freq;
    p.T = T;
    p.H = (int32_t)H;
    p.D = (int32_t)D;
    p.R = (int32_t)R;
    p.scale = scale;
    p.inverse = inverse ? 1 : 0;
    // Pieces of 16 bytes, two entries or one, as sizes, strides and addresses allow.
    const int64_t entry = bf16 ? 2 : 4;
    auto strided = [&](int64_t W) { return strided_pieces(W, entry, x, xt, xh) && strided_pieces(W, entry, y, yt, yh); };
    auto fits = [&](int64_t W) { return R / 2 % W == 0 && strided(W); };
    p.copy_piece = x == y ? 0 : copy_piece(R, D - R, entry, strided);
    const bool half = layout == BI_ROPE_HALF;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t W = 16 / entry, pieces = ((x == y ? R : D) + W - 1) / W, narrow = fits(2) ? 2 : 1;
    // Pairs that fill no 16-byte pieces are turned in shared memory, or walked through registers in narrower pieces.  The walk is
    // the faster in place, where it moves the turned entries only, if the lanes take a head's pairs at once and the pieces
    // are fp32 or the tokens few (us, staged and walked, in place: fp32, 2600 tokens of 16 heads, 60 turned 6.2 and 5.0, 132
    // turned 14.8 and 14.2; bf16, 20 of 80 entries of 32 heads, 1 token 2.6 and 2.3, 8284 13.4 and 14.5).  Between two tensors
    // staging is (the latter 8284: 18.2 and 24.0; fp32 29.3 and 35.8; 16 sizes of fp32 pairs 0.8 to 1.06 of the walk).
    const bool walk = x == y && R / 2 <= 32 * narrow && (!bf16 || T < dev->sms);
    if (R > 0 && !fits(W) && !walk && D % W == 0 && pieces <= 64 && strided(W)) {
        p.pieces = (int32_t)pieces;
        const int64_t heads = 64 / pieces;
        const RopeLaunch l(T, (H + heads - 1) / heads, true, p.R, dev->sms, bi::kRopeStagedBlocks);
        return bf16 ? launch_rope_staged<__nv_bfloat16>(p, half, l, s) : launch_rope_staged<float>(p, half, l, s);
    }
    if (bf16)
        return fits(8)   ? launch_rope<__nv_bfloat16, 8>(p, half, dev->sms, s)
               : fits(2) ? launch_rope<__nv_bfloat16, 2>(p, half, dev->sms, s)
                         : launch_rope<__nv_bfloat16, 1>(p, half, dev->sms, s);
    return fits(4)   ? launch_rope<float, 4>(p, half, dev->sms, s)
           : fits(2) ? launch_rope<float, 2>(p, half, dev->sms, s)
                     : launch_rope<float, 1>(p, half, dev->sms, s);
}

bi_status bi_rope_freqs(int64_t R, double theta, bi_rope_kind kind, const double *params, int64_t n_params,
                        double *inv_freq, double *scale)
{
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    if (R < 0 || R % 2 != 0 || R > bi::kRopeMaxDim || !(theta > 1.0) || !std::isfinite(theta)) return BI_ERR_INVALID_ARG;
    const int need = kind == BI_ROPE_PLAIN ? 0 : kind == BI_ROPE_LINEAR || kind == BI_ROPE_NTK ? 1 : 4;
    if (kind < BI_ROPE_PLAIN || kind > BI_ROPE_BANDED || n_params != need || (need > 0 && !params)) return BI_ERR_INVALID_ARG;
    if (R > 0 && !inv_freq) return BI_ERR_INVALID_ARG;
    for (int i = 0; i < need; ++i)
        if (!std::isfinite(params[i]) || !(params[i] > 0.0)) return BI_ERR_INVALID_ARG;
    const double factor = need > 0 ? params[0] : 1.0;
    if (factor < 1.0) return BI_ERR_INVALID_ARG;
    if (kind == BI_ROPE_NTK && R == 2) return BI_ERR_INVALID_ARG;
    if (need == 4 && !(kind == BI_ROPE_YARN ? params[2] > params[3] : params[3] > params[2])) return BI_ERR_INVALID_ARG;
    if (kind == BI_ROPE_NTK) theta *= std::pow(factor, (double)R / (double)(R - 2));
    double low = 0.0, high = 0.0;
    if (kind == BI_ROPE_YARN) {
        // The pair that makes `turns` turns within the original length.
        auto pair_of = [&](double turns) { return R * std::log(params[1] / (turns * kTwoPi)) / (2.0 * std::log(theta)); };
        low = std::fmax(std::floor(pair_of(params[2])), 0.0);
        high = std::fmin(std::ceil(pair_of(params[3])), (double)(R - 1));
        if (high < 0.0) {  // every pair makes fewer than beta_slow turns
            low = -2.0;
            high = -1.0;
        } else if (low >= high) {  // a step, or every pair makes more than beta_fast turns
            high = low + 0.001;
        }
    }
    for (int64_t i = 0; i < R / 2; ++i) {
        const double f = std::pow(theta, -2.0 * (double)i / (double)R);
        double g = f;
        if (kind == BI_ROPE_LINEAR) {
            g = f / factor;
        } else if (kind == BI_ROPE_YARN) {
            const double ramp = std::fmin(std::fmax(((double)i - low) / (high - low), 0.0), 1.0);
            g = f / factor * ramp + f * (1.0 - ramp);
        } else if (kind == BI_ROPE_BANDED) {
            const double turns = params[1] * f / kTwoPi;  // within the original length
            const double keep = std::fmin(std::fmax((turns - params[2]) / (params[3] - params[2]), 0.0), 1.0);
            g = (1.0 - keep) * f / factor + keep * f;
        }
        inv_freq[i] = g;
    }
    if (scale) *scale = kind == BI_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
    return BI_OK;
}

bi_status bi_paged_append(const void *k, int64_t k_token_stride, int64_t k_head_stride, const void *v,
                          int64_t v_token_stride, int64_t v_head_stride, const void *q, int64_t q_token_stride,
                          int64_t q_head_stride, void *q_out, int64_t q_out_token_stride,
                          int64_t q_out_head_stride, int64_t Hq, const bi_paged_cache *cache,
                          const int32_t *block_table, int64_t table_stride, int64_t max_pages,
                          const int32_t *seq_lens, const int32_t *cu_new, const int32_t *positions,
                          const double *inv_freq, int64_t R, bi_rope_layout layout, float scale, int64_t T,
                          int64_t B, void *stream)
{
    bi_status st = check_cache(cache);
    if (st != BI_OK) return st;
    const int64_t D = cache->head_dim, Hkv = cache->heads;
    if (T < 0 || B < 0 || max_pages < 0 || R < 0 || R > D || R % 2 != 0) return BI_ERR_INVALID_ARG;
    if (layout != BI_ROPE_HALF && layout != BI_ROPE_INTERLEAVED) return BI_ERR_INVALID_ARG;
    if ((q == nullptr) != (q_out == nullptr) || (q && Hq <= 0)) return BI_ERR_INVALID_ARG;
    if (T > kI32Max || B >= kI32Max || max_pages > kI32Max || Hq > 65535) return BI_ERR_UNSUPPORTED;
    if (T == 0 || B == 0) return BI_OK;
    if (!cu_new && T != B) return BI_ERR_INVALID_ARG;
    if (!k || !v || !seq_lens || (max_pages > 0 && !block_table) || (R > 0 && !inv_freq)) return BI_ERR_INVALID_ARG;
    if (B > 1 && table_stride < max_pages) return BI_ERR_INVALID_ARG;
    if (k_token_stride < 0 || k_head_stride < 0 || v_token_stride < 0 || v_head_stride < 0) return BI_ERR_INVALID_ARG;
    const int64_t qt = T > 1 && q ? q_token_stride : 0, qh = Hq > 1 && q ? q_head_stride : 0;
    const int64_t qot = T > 1 && q ? q_out_token_stride : 0, qoh = Hq > 1 && q ? q_out_head_stride : 0;
    if (q) {
        if (qt < 0 || qh < 0 || (T > 1 && qot < D) || (Hq > 1 && qoh < D)) return BI_ERR_INVALID_ARG;
        if (q == q_out && (qt != qot || qh != qoh)) return BI_ERR_INVALID_ARG;
    }
    for (const void *t : {k, v, q, static_cast<const void *>(q_out)})
        if (reinterpret_cast<uintptr_t>(t) & 1u) return BI_ERR_ALIGNMENT;
    for (const void *t : {block_table, seq_lens, cu_new, positions})
        if (reinterpret_cast<uintptr_t>(t) & 3u) return BI_ERR_ALIGNMENT;
    if (reinterpret_cast<uintptr_t>(inv_freq) & 7u) return BI_ERR_ALIGNMENT;
    DeviceState *dev = nullptr;
    st = device_state(&dev);
    if (st != BI_OK) return st;
    bi::AppendParams p{};
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.k_cache = static_cast<__nv_bfloat16 *>(cache->k);
    p.v_cache = static_cast<__nv_bfloat16 *>(cache->v);
    p.k_token = T > 1 ? k_token_stride : 0;
    p.k_head = Hkv > 1 ? k_head_stride : 0;
    p.v_token = T > 1 ? v_token_stride : 0;
    p.v_head = Hkv > 1 ? v_head_stride : 0;
    p.q_token = qt;
    p.q_head = qh;
    p.qo_token = qot;
    p.qo_head = qoh;
    p.c_page = cache->pages > 1 ? cache->page_stride : 0;
    p.c_token = cache->page_size > 1 ? cache->token_stride : 0;
    p.c_head = Hkv > 1 ? cache->head_stride : 0;
    p.table = block_table;
    p.table_row = table_stride;
    p.lens = seq_lens;
    p.cu = cu_new;
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.T = T;
    p.pages = cache->pages;
    p.B = (int32_t)B;
    p.Hq = (int32_t)Hq;
    p.Hkv = (int32_t)Hkv;
    p.D = (int32_t)D;
    p.R = (int32_t)R;
    p.page_size = (int32_t)cache->page_size;
    p.max_pages = (int32_t)max_pages;
    p.scale = scale;
    p.status = dev->status;
    auto turned = [&](int64_t W) {  // the cache's strides and addresses fit any piece
        return strided_pieces(W, 2, k, p.k_token, p.k_head) && strided_pieces(W, 2, q, qt, qh) &&
               strided_pieces(W, 2, q_out, qot, qoh);
    };
    auto fits = [&](int64_t W) { return R / 2 % W == 0 && turned(W); };
    p.rest_piece = copy_piece(R, D - R, 2, turned);
    p.v_piece = copy_piece(0, D, 2, [&](int64_t W) { return strided_pieces(W, 2, v, p.v_token, p.v_head); });
    const bool half = layout == BI_ROPE_HALF;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (R > 0 && !fits(8) && D % 8 == 0 && D <= 512 && turned(8) && p.v_piece == 16) {
        p.pieces = (int32_t)(D / 8);
        return launch_append_staged(p, half, dev->sms, s);
    }
    return fits(8)   ? launch_append<8>(p, half, dev->sms, s)
           : fits(2) ? launch_append<2>(p, half, dev->sms, s)
                     : launch_append<1>(p, half, dev->sms, s);
}

size_t bi_paged_decode_attention_scratch_bytes(int64_t B, int64_t Hq, int64_t D, int64_t max_len)
{
    if (B <= 0 || Hq <= 0 || D <= 0 || bi::pg_splits(max_len) <= 1) return 0;
    const size_t parts = (size_t)(B < bi::kPgSeqs ? B : bi::kPgSeqs) * (size_t)Hq * (size_t)bi::pg_splits(max_len);
    return parts * ((size_t)D * sizeof(float) + sizeof(float2));
}

bi_status bi_paged_decode_attention(const void *q, int64_t q_stride, const bi_paged_cache *cache,
                                    const int32_t *block_table, int64_t table_stride, int64_t max_pages,
                                    const int32_t *seq_lens, void *out, int64_t B, int64_t Hq, int64_t max_len,
                                    float scale, void *scratch, size_t scratch_bytes, void *stream)
{
    bi_status st = check_cache(cache);
    if (st != BI_OK) return st;
    const int64_t D = cache->head_dim, Hkv = cache->heads;
    if (B == 0) return BI_OK;
    if (B < 0 || Hq <= 0 || max_len <= 0 || max_pages <= 0 || Hq % Hkv != 0) return BI_ERR_INVALID_ARG;
    const int64_t G = Hq / Hkv;
    if ((D != 64 && D != 128) || G > 16) return BI_ERR_UNSUPPORTED;
    if (B > 65535 || Hq > 65535 || max_len > kI32Max - bi::kPgSplit || max_pages > kI32Max) return BI_ERR_UNSUPPORTED;
    if (max_len > max_pages * cache->page_size) return BI_ERR_INVALID_ARG;
    const int64_t S = bi::pg_splits(max_len), Bl = B < bi::kPgSeqs ? B : bi::kPgSeqs;
    if (Bl * S > kI32Max || Bl * S * Hkv > kI32Max) return BI_ERR_UNSUPPORTED;  // item numbers are 32-bit
    if (!q || !block_table || !seq_lens || !out || (S > 1 && !scratch)) return BI_ERR_INVALID_ARG;
    if ((B > 1 && (q_stride < Hq * D || table_stride < max_pages))) return BI_ERR_INVALID_ARG;
    if (scratch_bytes < bi_paged_decode_attention_scratch_bytes(B, Hq, D, max_len)) return BI_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || (S > 1 && !aligned16(scratch)) || (B > 1 && q_stride % 8 != 0) ||
        (reinterpret_cast<uintptr_t>(seq_lens) & 3u) || (reinterpret_cast<uintptr_t>(block_table) & 3u))
        return BI_ERR_ALIGNMENT;
    DeviceState *dev = nullptr;
    st = device_state(&dev);
    if (st != BI_OK) return st;

    bi::PgParams p{};
    // A box is the largest run of a tile's tokens that never leaves a page.
    int64_t box = cache->page_size, rest = bi::kPgTile;
    while (rest != 0) {
        const int64_t t = box % rest;
        box = rest;
        rest = t;
    }
    p.box = (int32_t)box;
    while ((1 << p.box_log2) < box) ++p.box_log2;
    p.boxes = bi::kPgTile / (int32_t)box;
    p.chunk = 32 / p.boxes;
    p.by_page = bi::PgDivisor::of((uint32_t)cache->page_size);
    p.by_heads = bi::PgDivisor::of((uint32_t)Hkv);
    p.heads_inner = cache->heads > 1 && (cache->page_size == 1 || cache->head_stride <= cache->token_stride) ? 1 : 0;
    CUtensorMap tm_k, tm_v;
    st = encode_page_map(&tm_k, cache->k, *cache, p.heads_inner != 0, (uint32_t)box);
    if (st != BI_OK) return st;
    st = encode_page_map(&tm_v, cache->v, *cache, p.heads_inner != 0, (uint32_t)box);
    if (st != BI_OK) return st;
    p.q_row = B > 1 ? q_stride : 0;
    p.table_row = B > 1 ? table_stride : 0;
    p.part_o = static_cast<float *>(scratch);
    p.part_ml = reinterpret_cast<float2 *>(p.part_o + (size_t)(S > 1 ? Bl * Hq * S * D : 0));
    p.Hq = (int32_t)Hq;
    p.Hkv = (int32_t)Hkv;
    p.G = (int32_t)G;
    p.S = (int32_t)S;
    p.pages = (int32_t)cache->pages;
    p.max_len = (int32_t)max_len;
    p.scale_log2 = (float)((double)scale * 1.4426950408889634074);
    p.status = dev->status;
    p.wait_limit_ns = kWaitLimitNs;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    for (int64_t b0 = 0; b0 < B; b0 += bi::kPgSeqs) {
        p.B = (int32_t)(B - b0 < bi::kPgSeqs ? B - b0 : bi::kPgSeqs);
        p.q = static_cast<const __nv_bfloat16 *>(q) + b0 * p.q_row;
        p.out = static_cast<__nv_bfloat16 *>(out) + b0 * Hq * D;
        p.lens = seq_lens + b0;
        p.table = block_table + b0 * p.table_row;
        // At most this many items; their true number is known on the device.
        const int64_t items = (int64_t)p.B * Hkv * S;
        const dim3 grid((unsigned)(items < dev->sms ? items : dev->sms));
        if (D == 64)
            st = G <= 8 ? launch_paged<64, 1>(grid, s, tm_k, tm_v, p) : launch_paged<64, 2>(grid, s, tm_k, tm_v, p);
        else
            st = G <= 8 ? launch_paged<128, 1>(grid, s, tm_k, tm_v, p) : launch_paged<128, 2>(grid, s, tm_k, tm_v, p);
        if (st != BI_OK) return st;
    }
    return BI_OK;
}

bi_status bi_token_logprobs(const void *x, int64_t ldx, bi_dtype x_dtype, const int32_t *tokens, float scale,
                            int64_t top_k, float *logprobs, float *entropy, float *logsumexp, float *top_logprobs,
                            int32_t *top_tokens, int64_t M, int64_t V, void *stream)
{
    if (M < 0 || V < 0 || top_k < 0) return BI_ERR_INVALID_ARG;
    if (x_dtype != BI_BF16 && x_dtype != BI_F32) return BI_ERR_INVALID_ARG;
    const double scale_log2 = (double)scale * 1.4426950408889634074;
    if (!(scale > 0.0f) || !std::isfinite((float)scale_log2)) return BI_ERR_INVALID_ARG;
    if (V > bi::kTlMaxV || top_k > bi::kTlMaxTop || M > kI32Max / bi::kTlMaxCluster) return BI_ERR_UNSUPPORTED;
    if (M == 0) return BI_OK;
    if (V == 0 || !x || ldx < V || top_k > V) return BI_ERR_INVALID_ARG;
    if ((logprobs && !tokens) || (top_k > 0 && (!top_logprobs || !top_tokens))) return BI_ERR_INVALID_ARG;
    const bool bf16 = x_dtype == BI_BF16;
    if (reinterpret_cast<uintptr_t>(x) & (bf16 ? 1u : 3u)) return BI_ERR_ALIGNMENT;
    for (const void *t : {static_cast<const void *>(tokens), static_cast<const void *>(logprobs),
                          static_cast<const void *>(entropy), static_cast<const void *>(logsumexp),
                          static_cast<const void *>(top_logprobs), static_cast<const void *>(top_tokens)})
        if (reinterpret_cast<uintptr_t>(t) & 3u) return BI_ERR_ALIGNMENT;
    DeviceState *dev = nullptr;
    bi_status st = device_state(&dev);
    if (st != BI_OK) return st;
    bi::TlParams p{};
    p.x = x;
    p.ldx = ldx;
    p.tokens = tokens;
    p.scale = scale;
    p.scale_log2 = (float)scale_log2;
    p.V = (int32_t)V;
    p.top = (int32_t)top_k;
    p.pieces = (int32_t)((V + bi::tl_piece(bf16) - 1) / bi::tl_piece(bf16));
    p.logprobs = logprobs;
    p.entropy = entropy;
    p.logsumexp = logsumexp;
    p.top_logprobs = top_logprobs;
    p.top_tokens = top_tokens;
    p.status = dev->status;
    // Blocks that share a row: as many as fit the GPU at once with room to spare.  Clusters of 8 up to 2 blocks an SM
    // (top 8 of 64 rows of 151936 bf16: 10.9 us with clusters of 4, 13.2 with 8); of 4 up to 2.8 and of 2 up to 3, if
    // each block has two pieces to take (top 5, with one block a row less and so: 100 rows 14.9 and 13.2 us, 200 rows 22.1
    // and 19.0; clusters of 4 do not pack closer, and the last run after the rest: 108 rows 14.9 and 18.3), else 2; any
    // up to 3.5 where rows are longer than 384 KB and each block's share counts for more (160 rows of 151936 fp32: 26.0
    // us with clusters of 2, 32.8 alone).
    const int64_t sms = dev->sms, row_bytes = V * (bf16 ? 2 : 4);
    auto fit = [&](int64_t blocks, int cluster) {
        if (row_bytes > 384 * 1024) return 2 * blocks <= 7 * sms;
        if (cluster == 8 || p.pieces < 2 * cluster) return blocks <= 2 * sms;
        return cluster == 4 ? 5 * blocks <= 14 * sms : blocks <= 3 * sms;
    };
    p.cluster = bi::kTlMaxCluster;
    while (p.cluster > 1 && (p.cluster > p.pieces || !fit(M * p.cluster, p.cluster))) p.cluster /= 2;
    size_t smem = token_logprobs_smem((p.pieces + p.cluster - 1) / p.cluster, top_k);
    // With more than 2 blocks an SM and at most 3, ask for so much shared memory that no SM takes a fourth while the
    // launch before leaves others short (300 rows of 151936 bf16, top 5: 33.3 us without, 29.0 with).
    const int64_t blocks = M * p.cluster;
    if (blocks > 2 * sms && blocks <= 3 * sms && (p.cluster <= 2 || (p.cluster == 4 && 5 * blocks <= 14 * sms)))
        smem = std::max<size_t>(smem, kTlThirdOfSm);
    const bool vec = aligned16(x) && (M == 1 || ldx % (bf16 ? 8 : 4) == 0);
    void (*kernel)(bi::TlParams) = bf16 ? (vec ? bi::token_logprobs_kernel<true, true> : bi::token_logprobs_kernel<true, false>)
                                        : (vec ? bi::token_logprobs_kernel<false, true> : bi::token_logprobs_kernel<false, false>);
    return launch_pdl_clusters(kernel, (unsigned)(M * p.cluster), bi::kTlThreads, (unsigned)p.cluster, smem,
                               static_cast<cudaStream_t>(stream), p);
}

bi_status bi_get_device_status(void *stream, int32_t *out)
{
    if (!out) return BI_ERR_INVALID_ARG;
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return BI_ERR_CUDA;
    int32_t v = 0;
    if (cudaMemcpyFromSymbol(&v, g_bi_status, sizeof v) != cudaSuccess) return BI_ERR_CUDA;
    const int32_t zero = 0;
    if (cudaMemcpyToSymbol(g_bi_status, &zero, sizeof zero) != cudaSuccess) return BI_ERR_CUDA;
    *out = v;
    return BI_OK;
}

bi_status bi_selftest_wait_timeout(int64_t limit_ns, void *stream)
{
    if (limit_ns < 1000 || limit_ns > 10000000000ll) return BI_ERR_INVALID_ARG;
    DeviceState *dev = nullptr;
    bi_status st = device_state(&dev);
    if (st != BI_OK) return st;
    return launch(selftest_wait_kernel, dim3(1), dim3(32), 0, static_cast<cudaStream_t>(stream), dev->status,
                  (uint64_t)limit_ns);
}

const char *bi_status_string(bi_status status)
{
    switch (status) {
    case BI_OK: return "BI_OK";
    case BI_ERR_INVALID_ARG: return "BI_ERR_INVALID_ARG";
    case BI_ERR_UNSUPPORTED: return "BI_ERR_UNSUPPORTED";
    case BI_ERR_ALIGNMENT: return "BI_ERR_ALIGNMENT";
    case BI_ERR_CUDA: return "BI_ERR_CUDA";
    case BI_ERR_TIMEOUT: return "BI_ERR_TIMEOUT";
    }
    return "BI_ERR_UNKNOWN";
}

void bi_gemm_config(int64_t weight_rows, int32_t *bm, int32_t *bn, int32_t *bk, int32_t *stages, int32_t *mma_k)
{
    const bi::PairConfig c = weight_rows > 0 ? bi::pair_config(weight_rows, true) : bi::kPairWide;
    if (bm) *bm = bi::kPairBM;
    if (bn) *bn = c == bi::kPairNarrow ? bi::NarrowTile::kBN : c == bi::kPairMid ? bi::MidTile::kBN : bi::WideTile::kBN;
    if (stages)
        *stages = c == bi::kPairNarrow ? bi::NarrowTile::kStages : c == bi::kPairMid ? bi::MidTile::kStages
                                                                                      : bi::WideTile::kStages;
    if (bk)
        *bk = c == bi::kPairNarrow ? bi::NarrowTile::kStageK : c == bi::kPairMid ? bi::MidTile::kStageK
                                                                                  : bi::WideTile::kStageK;
    if (mma_k) *mma_k = bi::kMmaK;
}

void bi_tensor_map_cache_stats(int64_t *hits, int64_t *misses)
{
    std::lock_guard<std::mutex> lock(g_map_mu);
    if (hits) *hits = (int64_t)g_map_hits;
    if (misses) *misses = (int64_t)g_map_misses;
}

int32_t bi_version(void) { return 300; }

}  // extern "C"
