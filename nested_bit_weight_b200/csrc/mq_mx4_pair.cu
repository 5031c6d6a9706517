// Products of MXFP4 matrices with many rows: two CTAs of a cluster share each
// MMA (tcgen05 cta_group::2, 256 rows of A by BN rows of B).
//     D[i, j] = sum_k A[i, k] B[j, k]
// One operand's 256 rows are split over the pair, so each SM loads only half
// of B as well.  The 4-bit rate is so high (16384 products a clock and SM) that a
// tile of 256 x 256 already takes 70 bytes a clock and SM from L2 at full rate,
// and single CTAs would take twice that (470 us where a pair takes 86).
// Measured: 4096 x 14336 x 4096 in 86 us (5.6 PFLOP/s), 8192^3 in 179 us (6.1);
// the power cap bounds these: the SM clock falls from 1965 to 1450-1650 MHz, and
// two thirds to three quarters of the cycles carry MMAs.  100 bf16 rows through
// 4096 x 14336: 24 us with the slices' own kernel (5), bound by L2 to shared memory
// (MMAs in 47 % of the cycles); 256 rows through 14336 x 4096 43 us, where MMAs take
// 66 %.
//   rows form     (S = 0) A = X, B = w: a lane holds a row of Y, BN consecutive
//                 features; 32-row pieces go through shared memory to TMA stores.
//   columns form  (S >= 1) A = w, B = X: a lane holds a feature, so that a warp
//                 stores 32 neighbours of a row of Y whatever Y's alignment.  S = 1
//                 where Y does not allow TMA stores, S = 8 for bf16 activations:
//                 eight columns of D add to one output.
//
// Persistent clusters, tiles dealt in turn (rows of A fastest, so that the
// clusters at work share B tiles in L2).  Tensor memory: two accumulators and
// the scales of every stage of the shared-memory ring (a stage's scales are
// overwritten only once its MMAs are done, with no wait of their own).  With 256
// columns that is more than 512, so the accumulators overlap by half (0..255,
// 128..383); the epilogue reads the shared half first and lets the next tile's
// MMAs start.
//
// Roles: a loading warp (both CTAs' loads complete on the even CTA's barrier), a
// warp of the even CTA that issues the MMAs, four epilogue warps.  Waits are
// bounded as in the other kernels, and a cluster barrier at the end keeps a
// CTA until its peer is through.
#include <cuda.h>

#include <atomic>
#include <type_traits>

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
__device__ int g_test_drop_pair;             // as in the kernel for few rows
#endif

template <int BN>
struct PairCfg {
    static constexpr int kBands = BN > 128 ? 2 : 1;                  // scale bands loaded for B
    static constexpr uint32_t kA = 128 * 128, kB = BN / 2 * 128;     // codes of a stage and CTA
    static constexpr uint32_t kSfA = 1024, kSfB = 1024 * kBands;
    static constexpr uint32_t kStage = kA + kB + kSfA + kSfB;
    static constexpr int kStages = BN > 128 ? 5 : 7;
    static constexpr uint32_t kStg = 4096;                           // one 32-row piece of Y
    static constexpr int kLag = BN == 256 ? 1 : 2;                   // tiles until the accumulator is needed again
    static constexpr uint32_t kD1 = BN == 256 ? 128 : 192;           // second accumulator
    static constexpr uint32_t kSf = 384, kSfCols = 8 + 8 * kBands;   // scales of the stages
    static_assert(kD1 + BN <= kSf && kSf + kStages * kSfCols <= 512, "TMEM columns");
    // A pair holds tensor memory while its second half may still wait for some, as
    // the clusters of the nested GEMV do; CTAs of both side by side on two SMs could
    // each hold what the other wants.  So no pair leaves the 20 KB that the smallest
    // of those needs beside it (the converters, which need none, still fit).
    static constexpr size_t kNeed = 1024 + (size_t)kStages * kStage + 8 * kStg + 512,
                            kSmem = kNeed < 207 * 1024 ? 207 * 1024 : kNeed;
    static_assert(kSmem <= 227 * 1024 && kStage % 1024 == 0, "shared memory");
};

struct PairArgs {
    CUtensorMap amap, bmap, ymap;  // codes in boxes of 128 and bn / 2 rows; Y
    CUtensorMap asmap, bsmap;      // scales in boxes of 1 and kBands row bands
    void *Y;
    int64_t ldy;
    int M, N;                      // rows of Y, columns of Y
    int64_t K;
    int Ta, Tb, KT;                // tiles along A and B, K tiles
    int bn;                        // rows of B a tile, a multiple of 16, at most BN
    int tpt;                       // S > 1: rows of X a tile
    int out;
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

// The staged piece (32 rows from m0, 128 bytes of columns from n0) to Y.
__device__ __forceinline__ void store_piece(const PairArgs &a, const uint8_t *stg, int lane, int m0, int n0) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        if (m0 < a.M && n0 < a.N) tma_store_2d(&a.ymap, n0, m0, stg);
        bulk_commit();                                               // empty or not: bulk_wait_read counts pieces
    }
}

// COUNT values of feature n, rows m0.. below mend of Y.
template <class T, int COUNT>
__device__ __forceinline__ void store_column(const PairArgs &a, int m0, int mend, int64_t n, const float (&y)[COUNT]) {
    if (n >= a.N) return;
    T *dst = static_cast<T *>(a.Y) + (int64_t)m0 * a.ldy + n;
#pragma unroll
    for (int e = 0; e < COUNT; ++e) {
        if (m0 + e < mend) {
            if constexpr (sizeof(T) == 4) *dst = y[e];
            else if constexpr (std::is_same<T, __half>::value) *dst = __float2half_rn(y[e]);
            else *dst = __float2bfloat16_rn(y[e]);
        }
        dst += a.ldy;
    }
}

template <int BN, int S>
__global__ void __launch_bounds__(kThreads, 1)
mx4_pair_kernel(const __grid_constant__ PairArgs a) {
    using C = PairCfg<BN>;
    constexpr int kS = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *stg = smem + kS * C::kStage;                            // [warp][2][4096]
    uint64_t *full = reinterpret_cast<uint64_t *>(stg + 8 * C::kStg);
    uint64_t *empty = full + kS, *dfull = empty + kS, *dfree = dfull + 2, *ready = dfree + 2;
    volatile int *flags = reinterpret_cast<volatile int *>(ready + 1);   // [0] abort
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(ready + 1) + 4;

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
        mbar_init(ready, 1);
        flags[0] = 0;
        fence_mbar_init();
    }
    if (threadIdx.x == 0) {
        // nothing is read before the wait; the weights only come into L2
        const CUtensorMap *wmap = S ? &a.amap : &a.bmap;
        const int y = S ? (cluster % a.Ta) * 256 + rank * 128 : (cluster / a.Ta) * a.bn + rank * (a.bn / 2);
        for (int kt = 0; kt < kS && kt < a.KT; ++kt) tma_prefetch_2d(wmap, kt * 128, y);
        prefetch_tensormap(S ? &a.bmap : &a.amap);
        prefetch_tensormap(&a.asmap);
        prefetch_tensormap(&a.bsmap);
    }
    __syncthreads();
    cluster_arrive();                                                // barriers of both CTAs ready
    cluster_wait();
    pdl_wait();

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
                    if (rank == 0) mbar_expect_tx(full + st, 2 * (C::kA + (uint32_t)a.bn * 64u + C::kSfA + C::kSfB));
                    tma_load_2d_pair(sA, &a.amap, kt * 128, ta * 256 + rank * 128, bar);
                    tma_load_2d_pair(sB, &a.bmap, kt * 128, tb * a.bn + rank * (a.bn / 2), bar);
                    tma_load_2d_pair(sfA, &a.asmap, kt * 256, ta * 2 + rank, bar);
                    tma_load_2d_pair(sfB, &a.bsmap, kt * 256, S > 1 ? tb * C::kBands : tb * a.bn / 128, bar);
                }
                __syncwarp();
            }
        }
    } else if (warp == 1) {
        // --------------------------------------------------------------- MMAs
        // tensor memory is taken after the previous kernel, so that it never waits
        // for columns held here, and only with it in hand does this kernel let the
        // next one start
        tmem_alloc2(tmem_slot, 512);
        tmem_relinquish2();
        pdl_launch_dependents();
        named_arrive(1, 160);                                        // the epilogue may read the address
        if (rank == 1) {
            if (lane == 0) mbar_arrive_remote_weak(cluster_map(smem_u32(ready), 0));
        }
        __syncwarp();
        const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(tmem_slot);
        // everything that does not change is worked out before the loop, and the
        // ring's slot and phase are counted, not divided for: what this warp does
        // between a stage's MMAs and the next is time the tensor core idles
        int it = 0, last = -1;                                       // last slot committed
        uint32_t st = 0, phase = 0, lastphase = 0;
        bool ok = rank == 0 && mbar_wait_abortable(ready, 0, flags); // the odd CTA has its columns too
        ok = __all_sync(0xFFFFFFFFu, ok);                            // its warp has nothing more to do
        const uint32_t s0 = smem_u32(smem);
        const uint64_t ad0 = smem_desc_sw128(s0), bd0 = smem_desc_sw128(s0 + C::kA),
                       sa0 = smem_desc_sf(s0 + C::kA + C::kB), sb0 = smem_desc_sf(s0 + C::kA + C::kB + C::kSfA);
        const uint32_t idesc = idesc_mxf4(256, S ? a.bn : BN, 0);
        const int tail = (int)((a.K - (int64_t)(a.KT - 1) * kTileK + 63) / 64);   // MMAs of the last stage of a tile
        for (int tile = cluster; tile < tiles && ok; tile += nclusters, ++it) {
            if (it >= C::kLag) {
                const int w = it - C::kLag;
                ok = mbar_wait_abortable(dfree + (w & 1), (uint32_t)(w >> 1) & 1u, flags);
                if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
            }
            const uint32_t d = tmem + (it & 1 ? C::kD1 : 0u);
            // first scale column of the tile's rows of B in its bands (rows form and
            // S = 1: tiles start at multiples of 64; S > 1: each tile has its own bands)
            const uint32_t b0 = S > 1 ? 0u : (uint32_t)((tile / a.Ta) * a.bn % 128) / 32u;
            for (int kt = 0; kt < a.KT; ++kt) {
                ok = mbar_wait_abortable(full + st, phase, flags);   // in both CTAs
                if (!(ok = __all_sync(0xFFFFFFFFu, ok))) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t step = (uint64_t)st * (C::kStage >> 4);
                    const uint32_t tA = tmem + C::kSf + st * C::kSfCols, tB = tA + 8;
                    const int steps = kt + 1 < a.KT ? 4 : tail;
                    // scales: four columns per 128 rows and group
#pragma unroll
                    for (int g = 0; g < 2; ++g)
                        if (2 * g < steps) {
                            tmem_cp_sf_pair(tA + 4 * g, sa0 + step + 32 * g);
#pragma unroll
                            for (int b = 0; b < C::kBands; ++b)
                                tmem_cp_sf_pair(tB + 4 * (C::kBands * g + b), sb0 + step + 64 * b + 32 * g);
                        }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < steps)
                            mma_mxf4_pair(d, ad0 + step + 2 * j, bd0 + step + 2 * j, idesc + ((j & 1) ? kIdescSf2 : 0u),
                                          tA + 4 * (j >> 1), tB + b0 + 4 * C::kBands * (j >> 1), kt + j > 0 ? 1u : 0u);
                    mma_commit_pair(empty + st);
                    if (kt == a.KT - 1) mma_commit_pair(dfull + (it & 1));
                }
                __syncwarp();
                last = (int)st;
                lastphase = phase;
                if (++st == kS) {
                    st = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!ok && last >= 0) mbar_wait_bounded(empty + last, lastphase);   // MMAs in flight land
    } else if (warp >= kEpiW0) {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3;                                      // TMEM lane quarter
        named_sync(1, 160);
        tc_fence_after();
        const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(tmem_slot);
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
            auto drained = [&] {                                     // the accumulator (its shared half) is read
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote_weak(free0 + 8u * (uint32_t)(it & 1));
            };
            if constexpr (S == 0) {
                // 128 columns at a time (64 where 128 do not divide them), with
                // overlapping accumulators the shared half first
                constexpr int kCols = BN % 128 ? 64 : 128, kChunks = BN / kCols;
                const int first = C::kLag == 1 && (it & 1) == 0 ? kChunks - 1 : 0;
#pragma unroll 1
                for (int p = 0; p < kChunks; ++p) {
                    const int c0 = kCols * ((p + first) % kChunks);
                    __syncwarp();                                    // one lane issued the last piece
                    uint32_t v[kCols];
#pragma unroll
                    for (int e = 0; e < kCols / 32; ++e) tmem_ld32(d + c0 + 32 * e, v + 32 * e);
                    tmem_ld_wait();
                    if (p == (C::kLag == 1 ? 0 : kChunks - 1)) drained();
                    const int n0 = tb * BN + c0;
                    if (a.out == MQ_F32) {
#pragma unroll
                        for (int h = 0; h < kCols / 32; ++h, ++piece) {
                            uint32_t w[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) w[e] = v[32 * h + e];
                            uint8_t *s = mystg + (piece & 1) * C::kStg;
                            if (lane == 0) bulk_wait_read<1>();      // the piece before the last has left
                            __syncwarp();
                            stage_row(s, lane, w);
                            store_piece(a, s, lane, arow, n0 + 32 * h);
                        }
                    } else {
#pragma unroll
                        for (int h = 0; h < kCols / 64; ++h, ++piece) {
                            uint32_t w[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const float x = __uint_as_float(v[64 * h + 2 * e]),
                                            y = __uint_as_float(v[64 * h + 2 * e + 1]);
                                w[e] = a.out == MQ_BF16 ? pack2<__nv_bfloat16>(x, y) : pack2<__half>(x, y);
                            }
                            uint8_t *s = mystg + (piece & 1) * C::kStg;
                            if (lane == 0) bulk_wait_read<1>();
                            __syncwarp();
                            stage_row(s, lane, w);
                            store_piece(a, s, lane, arow, n0 + 64 * h);
                        }
                    }
                }
            } else {
                // eight rows of Y (32 with S = 1) at a time
                constexpr int kRows = S == 1 ? 32 : 8, kCols = kRows * S;
                const int64_t n = arow + lane;
                const int rows = S == 1 ? a.bn : a.tpt, m0 = tb * rows, mend = a.M - m0 < rows ? a.M : m0 + rows;
#pragma unroll 1
                for (int c = 0; c * S < a.bn && m0 + c < mend; c += kRows) {
                    __syncwarp();                                    // lanes beyond N left the last stores early
                    uint32_t v[kCols];
                    float y[kRows];
#pragma unroll
                    for (int e = 0; e < kCols / 32; ++e) tmem_ld32(d + c * S + 32 * e, v + 32 * e);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < kRows; ++e) {
                        y[e] = __uint_as_float(v[S * e + S - 1]);    // small slices first
#pragma unroll
                        for (int j = S - 2; j >= 0; --j) y[e] += __uint_as_float(v[S * e + j]);
                    }
                    if (a.out == MQ_BF16) store_column<__nv_bfloat16>(a, m0 + c, mend, n, y);
                    else if (a.out == MQ_F16) store_column<__half>(a, m0 + c, mend, n, y);
                    else store_column<float>(a, m0 + c, mend, n, y);
                }
                drained();
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
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_arrive();                                                // the peer reads this CTA's memory until here
    cluster_wait();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc2(*reinterpret_cast<volatile uint32_t *>(tmem_slot), 512);
    }
}

using PairFn = void (*)(PairArgs);

template <int BN, int S>
cudaError_t pick(PairFn *fn, size_t *smem) {
    static std::atomic<uint64_t> done{0};
    *fn = mx4_pair_kernel<BN, S>;
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

constexpr int kClusters = 74;                // two CTAs each, one an SM

// Clocks of a product of Ta x Tb tiles with bn rows of B: rounds of tiles, each
// about 1500 at its ends and KT stages of four MMAs (bn / 2 clocks each, at least
// 75) or of 19 KiB + 64 bn bytes from L2 (58 a clock).
int64_t clocks(int64_t Ta, int64_t Tb, int bn, int64_t KT) {
    const int mma = 4 * (bn / 2 < 75 ? 75 : bn / 2), load = (19456 + 64 * bn) / 58;
    return (Ta * Tb + kClusters - 1) / kClusters * (KT * (mma > load ? mma : load) + 1500);
}

}  // namespace

bool mx_pair_takes(const MxProduct &p) { return p.slices != 1 ? p.slice.Tb > 0 : p.M > 128; }

MxSlicing mx_slicing(int64_t M, int64_t N) {
    MxSlicing s{};
    if (M * kMxSlices <= 128) {                  // one tile of the kernel for few rows
        s.tpt = (int)M;
        s.rows = M * kMxSlices;
        s.bands = 1;
        s.bn = (int)s.rows;
        return s;
    }
    // 24 rows of X a tile; 32 where only that lets the clusters take all tiles at
    // once (100 x 4096 x 14336: 24.4 us, with 24 rows and a second round for six of
    // 80 tiles 32.3).  Elsewhere the narrower tile is ahead, with its two whole
    // accumulators and fewer columns that wait for L2 (128 x 14336 x 4096: 26.5
    // against 29.2, 32 x 4096 x 4096: 9.1 against 10.4).
    const int64_t Ta = (N + 255) / 256;
    const int most = Ta * ((M + 23) / 24) > kClusters && Ta * ((M + 31) / 32) <= kClusters ? 32 : 24;
    s.Tb = (int)((M + most - 1) / most);
    s.tpt = (int)((M + s.Tb - 1) / s.Tb);        // rows of X dealt evenly
    s.bn = (s.tpt * kMxSlices + 15) / 16 * 16;
    s.rows = (int64_t)s.Tb * s.bn;
    s.bands = (int64_t)s.Tb * 2;
    return s;
}

namespace {

// Form and tiles of a product.
struct PairPlan {
    int S, bn;                     // as the kernel's template argument and PairArgs::bn
    int64_t Ta, Tb;
};
PairPlan pair_plan(const MxProduct &p) {
    const int64_t N = p.w->rows, KT = (p.w->K + kTileK - 1) / kTileK;
    const int size = p.out == MQ_F32 ? 4 : 2;
    if (p.slices != 1) return {kMxSlices, p.slice.bn, (N + 255) / 256, p.slice.Tb};
    // the cheapest of the widths, the widest first
    auto cheapest = [KT](int64_t Ta, int64_t B, int bn, int bn1, int bn2) {
        for (int b : {bn1, bn2})
            if (clocks(Ta, (B + b - 1) / b, b, KT) < clocks(Ta, (B + bn - 1) / bn, bn, KT)) bn = b;
        return bn;
    };
    // TMA stores want row strides in 16 bytes (below 2^40), and cut a box off at
    // the tensor's edge in steps of 16 bytes only
    if (p.ldy * size % 16 == 0 && N * size % 16 == 0 && p.ldy < ((int64_t)1 << 36)) {
        const int64_t Ta = (p.M + 255) / 256;
        const int bn = cheapest(Ta, N, 256, 192, 128);
        return {0, bn, Ta, (N + bn - 1) / bn};
    }
    const int64_t Ta = (N + 255) / 256;
    const int bn = cheapest(Ta, p.M, 192, 128, 64);
    return {1, bn, Ta, (p.M + bn - 1) / bn};
}

}  // namespace

mq_status launch_mx_pair(const MxProduct &p, cudaStream_t st) {
    const mq_mx4 *w = p.w;
    const PairPlan plan = pair_plan(p);
    const int64_t Ta = plan.Ta, Tb = plan.Tb;
    PairArgs a{};
    a.Y = p.Y;
    a.ldy = p.ldy;
    a.M = (int)p.M;
    a.N = (int)w->rows;
    a.K = w->K;
    a.KT = (int)((w->K + kTileK - 1) / kTileK);
    a.out = p.out;
    a.bn = plan.bn;
    PairFn fn;
    size_t smem;
    cudaError_t e;
    bool maps;
    if (plan.S == 0) {
        e = a.bn == 256 ? pick<256, 0>(&fn, &smem) : a.bn == 192 ? pick<192, 0>(&fn, &smem) : pick<128, 0>(&fn, &smem);
        maps = mx_encode_codes(&a.amap, p.xcodes, p.M, w->K, 128) && mx_encode_scales(&a.asmap, p.xscales, p.M, w->K, 1) &&
               mx_encode_codes(&a.bmap, w->codes, w->rows, w->K, a.bn / 2) &&
               mx_encode_scales(&a.bsmap, w->scales, w->rows, w->K, a.bn > 128 ? 2 : 1) &&
               mx_encode_y(&a.ymap, p.Y, p.M, w->rows, p.ldy, p.out);
    } else {
        int64_t xrows = p.M, sfrows = p.M;
        if (plan.S == 1) {
            e = pick<192, 1>(&fn, &smem);
        } else {
            a.tpt = p.slice.tpt;
            xrows = p.slice.rows;
            sfrows = p.slice.bands * 128;
            e = a.bn > 192 ? pick<256, kMxSlices>(&fn, &smem) : pick<192, kMxSlices>(&fn, &smem);
        }
        maps = mx_encode_codes(&a.amap, w->codes, w->rows, w->K, 128) &&
               mx_encode_scales(&a.asmap, w->scales, w->rows, w->K, 1) &&
               mx_encode_codes(&a.bmap, p.xcodes, xrows, w->K, a.bn / 2) &&
               mx_encode_scales(&a.bsmap, p.xscales, sfrows, w->K, 2);
    }
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
    if (!maps) return fail(MQ_ERR_CUDA, "cuTensorMapEncodeTiled (MXFP4 product)");
    if (Ta * Tb > 0x3FFFFFFF) return fail(MQ_ERR_UNSUPPORTED, "too many output tiles");
    a.Ta = (int)Ta;
    a.Tb = (int)Tb;
    const int64_t clusters = Ta * Tb < kClusters ? Ta * Tb : kClusters;
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

#ifdef MQ_TEST_HOOKS
// Test-hook builds only: how a product is tiled (host arithmetic alone).  Returns 0
// (rows form), 1 or 8 (columns form, plain and sliced bf16 rows) with plan =
// {rows of B a tile, tiles along A, tiles along B}, or -1 for the kernel for few rows.
extern "C" __attribute__((visibility("default"))) int mq_test_mx4_plan(int64_t M, int64_t N, int64_t K, int out,
                                                                       int64_t ldy, int bf16_rows, int64_t *plan) {
    using namespace mq;
    const mq_mx4 w{nullptr, nullptr, N, K};
    MxProduct p{nullptr, nullptr, M, bf16_rows ? kMxSlices : 1, &w, nullptr, out, ldy, nullptr, 0, {}};
    if (bf16_rows) p.slice = mx_slicing(M, N);
    if (!mx_pair_takes(p)) return -1;
    const PairPlan t = pair_plan(p);
    plan[0] = t.bn;
    plan[1] = t.Ta;
    plan[2] = t.Tb;
    return t.S;
}
// The least shared memory of a pair's CTA.
extern "C" __attribute__((visibility("default"))) size_t mq_test_mx4_pair_smem() {
    using namespace mq;
    size_t s = PairCfg<256>::kSmem;
    for (size_t b : {PairCfg<192>::kSmem, PairCfg<128>::kSmem}) s = b < s ? b : s;
    return s;
}
#endif
