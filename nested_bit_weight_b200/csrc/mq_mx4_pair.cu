// Products of MXFP4 matrices with many rows: two CTAs of a cluster share each
// MMA (tcgen05 cta_group::2, 256 rows of A by BN rows of B).
//     D[i, j] = sum_k A[i, k] B[j, k]
// One operand's 256 rows are split over the pair, so each SM loads only half
// of B as well: the bytes that feed one MMA halve against single CTAs, and the
// 4-bit rate is so high (16384 products a clock and SM) that those bytes, from
// L2 through shared memory, are what bounds a large product.
//   rows form     A = X, B = w: a lane holds a row of Y, BN consecutive features;
//                 32 x 64 pieces go through shared memory to TMA stores.
//   slices form   A = w, B = X (bf16 activations as sums of eight MXFP4 rows): a
//                 lane holds a feature; eight columns of D add to one output.
//
// Persistent clusters, tiles dealt in turn (rows of A fastest, so that the
// clusters at work share B tiles in L2).  Tensor memory: two accumulators and
// the scales of every stage of the shared-memory ring (a stage's scales are
// overwritten only once its MMAs are done, with no wait of their own).  That is
// more than 512 columns, so the accumulators overlap by half (0..255, 128..383);
// the epilogue reads the shared half first and lets the next tile's MMAs start.
//
// Roles: a loading warp (both CTAs' loads complete on the even CTA's barrier), a
// warp of the even CTA that issues the MMAs, four epilogue warps.  Waits are
// bounded as in the other kernels, and a cluster barrier at the end keeps a
// CTA until its peer is through.
#include <cuda.h>

#include <atomic>

#include "mq_mx4.cuh"
#include "mq_sm100.cuh"

namespace mq {
namespace {

using namespace sm100;

constexpr int kThreads = 192;
constexpr int kEpiW0 = 2;
constexpr int kTileK = 256;

__device__ unsigned int g_pair_timeout;

#ifdef MQ_TEST_HOOKS
__device__ int g_test_drop_pair;             // as in the single-CTA kernel
#endif

template <int BN>
struct PairCfg {
    static constexpr int kBands = BN / 128;
    static constexpr uint32_t kA = 128 * 128, kB = BN / 2 * 128;     // codes of a stage and CTA
    static constexpr uint32_t kSfA = 1024, kSfB = 1024 * kBands;
    static constexpr uint32_t kStage = kA + kB + kSfA + kSfB;
    static constexpr int kStages = BN == 256 ? 5 : 7;
    static constexpr uint32_t kStg = 4096;                           // one 32-row piece of Y
    static constexpr int kLag = BN == 256 ? 1 : 2;                   // tiles until the accumulator is needed again
    static constexpr uint32_t kD1 = 128;                             // second accumulator
    static constexpr uint32_t kSf = kD1 + BN, kSfCols = 8 + 8 * kBands;
    static_assert(kSf + kStages * kSfCols <= 512, "TMEM columns");
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + 8 * kStg + 512;
    static_assert(kSmem <= 227 * 1024 && kStage % 1024 == 0, "shared memory");
};

struct PairArgs {
    CUtensorMap amap, bmap, ymap;  // codes in boxes of 128 and BN / 2 rows; Y
    CUtensorMap asmap, bsmap;      // scales in boxes of 1 and BN / 128 row bands
    void *Y;
    int64_t ldy;
    int M, N;                      // rows of Y, columns of Y
    int64_t K;
    int Ta, Tb, KT;                // tiles along A and B, K tiles
    int out;
    int tma_y;                     // Y's rows allow TMA stores
};

template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// This lane's row of a 32-row piece (128 bytes, as 32 words) to shared memory
// in the 128-byte swizzle.
__device__ __forceinline__ void stage_row(uint8_t *stg, int lane, const uint32_t (&w)[32]) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4 *>(stg + lane * 128 + ((c ^ (lane & 7)) << 4)) =
            make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
}

// The staged piece (rows m0.., 128 bytes from byte x0 of a row) to Y.
template <int SIZE>
__device__ __forceinline__ void store_piece(const PairArgs &a, const uint8_t *stg, int lane, int m0, int n0) {
    constexpr int kCols = 128 / SIZE;
    if (m0 >= a.M || n0 >= a.N) {                                    // uniform over the warp
        if (lane == 0) bulk_commit();                                // an empty group: bulk_wait_read counts pieces
        return;
    }
    if (a.tma_y) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_2d(&a.ymap, n0, m0, stg);
            bulk_commit();
        }
    } else {
        __syncwarp();
        const int rows = a.M - m0 < 32 ? a.M - m0 : 32;
        for (int r = 0; r < rows; ++r)
#pragma unroll
            for (int h = 0; h < kCols / 32; ++h) {
                const int col = 32 * h + lane, byte = col * SIZE;
                const uint8_t *p = stg + r * 128 + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 15);
                if (n0 + col < a.N) {
                    const int64_t at = (int64_t)(m0 + r) * a.ldy + n0 + col;
                    if constexpr (SIZE == 2) static_cast<uint16_t *>(a.Y)[at] = *reinterpret_cast<const uint16_t *>(p);
                    else static_cast<uint32_t *>(a.Y)[at] = *reinterpret_cast<const uint32_t *>(p);
                }
            }
        __syncwarp();
    }
}

template <int BN, bool SLICES>
__global__ void __launch_bounds__(kThreads, 1)
mx4_pair_kernel(const __grid_constant__ PairArgs a) {
    using C = PairCfg<BN>;
    constexpr int kS = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *stg = smem + kS * C::kStage;                            // [warp][2][4096]
    uint64_t *full = reinterpret_cast<uint64_t *>(stg + 8 * C::kStg);
    uint64_t *empty = full + kS, *dfull = empty + kS, *dfree = dfull + 2;
    volatile int *flags = reinterpret_cast<volatile int *>(dfree + 2);   // [0] abort [2] MMA stages
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(dfree + 2) + 4;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)(blockIdx.x & 1), cluster = (int)(blockIdx.x >> 1), nclusters = (int)(gridDim.x >> 1);
    const int tiles = a.Ta * a.Tb;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kS; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(dfull + i, 1);
            mbar_init(dfree + i, 8);                                 // four epilogue warps of each CTA
        }
        flags[0] = flags[2] = 0;
        fence_mbar_init();
    }
    pdl_wait();
    if (warp == 1) {
        tmem_alloc2(tmem_slot, 512);
        tmem_relinquish2();
    }
    tc_fence_before();
    __syncthreads();
    cluster_arrive();                                                // barriers of both CTAs ready
    cluster_wait();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(tmem_slot);

    if (warp == 0) {
        // -------------------------------------------------------------- loads
        int i = 0;                                                   // stages over all tiles
        bool ok = true;
        const uint32_t full0 = cluster_map(smem_u32(full), 0);       // the even CTA's barriers
        for (int tile = cluster; tile < tiles && ok; tile += nclusters) {
            const int ta = tile % a.Ta, tb = tile / a.Ta;
            for (int kt = 0; kt < a.KT; ++kt, ++i) {
                const int st = i % kS;
#ifdef MQ_TEST_HOOKS
                if (i == 0) {
                    const int drop = lane == 0 ? atomicSub(&g_test_drop_pair, 1) : 0;
                    if (__any_sync(0xFFFFFFFFu, drop > 0)) { ok = false; break; }
                }
#endif
                ok = i < kS || mbar_wait_backoff(empty + st, (uint32_t)(i / kS - 1) & 1u, flags);
                if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
                if (elect_one()) {
                    uint8_t *sA = smem + st * C::kStage, *sB = sA + C::kA, *sfA = sB + C::kB, *sfB = sfA + C::kSfA;
                    const uint32_t bar = full0 + 8u * (uint32_t)st;
                    if (rank == 0) mbar_expect_tx(full + st, 2 * C::kStage);
                    tma_load_2d_pair(sA, &a.amap, kt * 128, ta * 256 + rank * 128, bar);
                    tma_load_2d_pair(sB, &a.bmap, kt * 128, tb * BN + rank * (BN / 2), bar);
                    tma_load_2d_pair(sfA, &a.asmap, kt * 256, ta * 2 + rank, bar);
                    tma_load_2d_pair(sfB, &a.bsmap, kt * 256, tb * C::kBands, bar);
                }
                __syncwarp();
            }
        }
    } else if (warp == 1 && rank == 0) {
        // --------------------------------------------------------------- MMAs
        int i = 0, it = 0;
        bool ok = true;
        for (int tile = cluster; tile < tiles && ok; tile += nclusters, ++it) {
            if (it >= C::kLag) {
                const int w = it - C::kLag;
                ok = mbar_wait_abortable(dfree + (w & 1), (uint32_t)(w >> 1) & 1u, flags);
                if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
            }
            const uint32_t d = tmem + (it & 1 ? C::kD1 : 0u);
            for (int kt = 0; kt < a.KT; ++kt, ++i) {
                const int st = i % kS;
                ok = mbar_wait_abortable(full + st, (uint32_t)(i / kS) & 1u, flags);   // in both CTAs
                if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
                tc_fence_after();
                const int64_t left = a.K - (int64_t)kt * kTileK;
                if (elect_one()) {
                    const uint32_t sA = smem_u32(smem + st * C::kStage), sB = sA + C::kA, sfA = sB + C::kB,
                                   sfB = sfA + C::kSfA;
                    const uint32_t tA = tmem + C::kSf + (uint32_t)st * C::kSfCols, tB = tA + 8;
                    const uint64_t ad = smem_desc_sw128(sA), bd = smem_desc_sw128(sB);
                    const int steps = left >= kTileK ? 4 : (int)((left + 63) / 64);
                    // scales: four columns per 128 rows and group
#pragma unroll
                    for (int g = 0; g < 2; ++g)
                        if (2 * g < steps) {
                            tmem_cp_sf_pair(tA + 4 * g, smem_desc_sf(sfA + 512 * g));
#pragma unroll
                            for (int b = 0; b < C::kBands; ++b)
                                tmem_cp_sf_pair(tB + 4 * (C::kBands * g + b), smem_desc_sf(sfB + 1024 * b + 512 * g));
                        }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < steps)
                            mma_mxf4_pair(d, ad + 2 * j, bd + 2 * j, idesc_mxf4(256, BN, (j & 1) * 2),
                                          tA + 4 * (j >> 1), tB + 4 * C::kBands * (j >> 1), kt + j > 0 ? 1u : 0u);
                    mma_commit_pair(empty + st);
                    if (kt == a.KT - 1) mma_commit_pair(dfull + (it & 1));
                    flags[2] = i + 1;
                }
                __syncwarp();
            }
        }
    } else if (warp >= kEpiW0) {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3;                                      // TMEM lane quarter
        uint8_t *mystg = stg + (warp - kEpiW0) * 2 * C::kStg;
        const uint32_t free0 = cluster_map(smem_u32(dfree), 0);
        int it = 0, piece = 0;
        for (int tile = cluster; tile < tiles; tile += nclusters, ++it) {
            const int ta = tile % a.Ta, tb = tile / a.Ta;
            bool ok = mbar_wait_backoff(dfull + (it & 1), (uint32_t)(it >> 1) & 1u, flags);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            tc_fence_after();
            const uint32_t d = tmem + (it & 1 ? C::kD1 : 0u) + ((uint32_t)(32 * q) << 16);
            const int arow = ta * 256 + rank * 128 + 32 * q;         // first row of A of this warp
            // the columns shared with the other accumulator first
            constexpr int kChunks = BN / 128;
            const int first = C::kLag == 1 && (it & 1) == 0 ? kChunks - 1 : 0;
#pragma unroll 1
            for (int p = 0; p < kChunks; ++p) {
                const int c128 = 128 * ((p + first) % kChunks);
                uint32_t v128[128];
#pragma unroll
                for (int e = 0; e < 4; ++e) tmem_ld32(d + c128 + 32 * e, v128 + 32 * e);
                tmem_ld_wait();
                if (p == (C::kLag == 1 ? 0 : kChunks - 1)) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote_weak(free0 + 8u * (uint32_t)(it & 1));
                }
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                const uint32_t *v = v128 + 64 * hf;
                const int c = c128 + 64 * hf;
                if constexpr (SLICES) {
                    const int64_t n = arow + lane;
                    const int m0 = (tb * BN + c) / kMxSlices;
#pragma unroll
                    for (int e = 0; e < 64 / kMxSlices; ++e) {
                        float y = __uint_as_float(v[kMxSlices * e + kMxSlices - 1]);   // small slices first
#pragma unroll
                        for (int j = kMxSlices - 2; j >= 0; --j) y += __uint_as_float(v[kMxSlices * e + j]);
                        if (n < a.N && m0 + e < a.M) {
                            const int64_t at = (int64_t)(m0 + e) * a.ldy + n;
                            if (a.out == MQ_BF16) static_cast<__nv_bfloat16 *>(a.Y)[at] = __float2bfloat16_rn(y);
                            else if (a.out == MQ_F16) static_cast<__half *>(a.Y)[at] = __float2half_rn(y);
                            else static_cast<float *>(a.Y)[at] = y;
                        }
                    }
                } else {
                    const int n0 = tb * BN + c;
                    if (a.out == MQ_F32) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t w[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) w[e] = v[32 * h + e];
                            uint8_t *s = mystg + (piece & 1) * C::kStg;
                            if (lane == 0) bulk_wait_read<1>();      // the piece before the last has left
                            __syncwarp();
                            stage_row(s, lane, w);
                            store_piece<4>(a, s, lane, arow, n0 + 32 * h);
                            ++piece;
                        }
                    } else {
                        uint32_t w[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float x = __uint_as_float(v[2 * e]), y = __uint_as_float(v[2 * e + 1]);
                            w[e] = a.out == MQ_BF16 ? pack2<__nv_bfloat16>(x, y) : pack2<__half>(x, y);
                        }
                        uint8_t *s = mystg + (piece & 1) * C::kStg;
                        if (lane == 0) bulk_wait_read<1>();
                        __syncwarp();
                        stage_row(s, lane, w);
                        store_piece<2>(a, s, lane, arow, n0);
                        ++piece;
                    }
                }
                }
            }
        }
        if (lane == 0) bulk_wait_all();                              // Y is written before the CTA ends
    }

    // ---- end: copies and MMAs in flight land (already so unless a wait gave up)
    __syncwarp();
    __syncthreads();
    if (threadIdx.x == 0 && flags[0]) {
        atomicOr(&g_pair_timeout, 1u);
        // a pair's stage may stay incomplete once one of its CTAs gave up, so
        // loads are given a millisecond (a load takes microseconds) to land
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < 1000000ull) __nanosleep(1000);
        for (int s = 0; s < kS && s < flags[2]; ++s)
            mbar_wait_bounded(empty + s, (uint32_t)((flags[2] - 1 - s) / kS) & 1u);
    }
    tc_fence_before();
    __syncthreads();
    cluster_arrive();                                                // the peer reads this CTA's memory until here
    cluster_wait();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc2(tmem, 512);
    }
}

using PairFn = void (*)(PairArgs);

template <int BN, bool SLICES>
cudaError_t pick(PairFn *fn, size_t *smem) {
    static std::atomic<uint64_t> done{0};
    *fn = mx4_pair_kernel<BN, SLICES>;
    *smem = PairCfg<BN>::kSmem;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(*fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)PairCfg<BN>::kSmem);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

}  // namespace

bool mx_pair_takes(const MxProduct &p) { return p.M * p.slices > 128; }

mq_status launch_mx_pair(const MxProduct &p, cudaStream_t st) {
    const mq_mx4 *w = p.w;
    const bool slices = p.slices > 1;
    const int64_t cols = p.M * p.slices;
    const int64_t ra = slices ? w->rows : cols, rb = slices ? cols : w->rows;
    constexpr int BN = 256;
    PairFn fn;
    size_t smem;
    cudaError_t e = slices ? pick<BN, true>(&fn, &smem) : pick<BN, false>(&fn, &smem);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
    PairArgs a{};
    a.Y = p.Y;
    a.ldy = p.ldy;
    a.M = (int)p.M;
    a.N = (int)w->rows;
    a.K = w->K;
    a.KT = (int)((w->K + kTileK - 1) / kTileK);
    a.out = p.out;
    const int64_t Ta = (ra + 255) / 256, Tb = (rb + BN - 1) / BN;
    if (Ta * Tb > 0x3FFFFFFF) return fail(MQ_ERR_UNSUPPORTED, "too many output tiles");
    a.Ta = (int)Ta;
    a.Tb = (int)Tb;
    // TMA stores want row strides in 16 bytes, and cut a box off at the tensor's
    // edge in steps of 16 bytes only (columns behind an odd N were overwritten)
    const int size = p.out == MQ_F32 ? 4 : 2;
    a.tma_y = !slices && p.ldy * size % 16 == 0 && w->rows * size % 16 == 0;
    if (!mx_encode_codes(&a.amap, slices ? w->codes : p.xcodes, ra, w->K, 128) ||
        !mx_encode_codes(&a.bmap, slices ? p.xcodes : w->codes, rb, w->K, BN / 2) ||
        !mx_encode_scales(&a.asmap, slices ? w->scales : p.xscales, ra, w->K, 1) ||
        !mx_encode_scales(&a.bsmap, slices ? p.xscales : w->scales, rb, w->K, BN / 128) ||
        (a.tma_y && !mx_encode_y(&a.ymap, p.Y, p.M, w->rows, p.ldy, p.out)))
        return fail(MQ_ERR_CUDA, "cuTensorMapEncodeTiled (MXFP4 product)");
    int64_t clusters = Ta * Tb < 74 ? Ta * Tb : 74;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * clusters));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, fn, a);
    return e == cudaSuccess ? MQ_OK : cuda_fail(e, "mx4_pair_kernel");
}

bool mx_pair_take_timeout(bool *set) {
    unsigned v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_pair_timeout, sizeof(v)) != cudaSuccess) return false;
    if (v && cudaMemcpyToSymbol(g_pair_timeout, &z, sizeof(z)) != cudaSuccess) return false;
    *set = v != 0;
    return true;
}

#ifdef MQ_TEST_HOOKS
int pair_test_drop(int n) { return (int)cudaMemcpyToSymbol(g_test_drop_pair, &n, sizeof(n)); }
#endif

}  // namespace mq
