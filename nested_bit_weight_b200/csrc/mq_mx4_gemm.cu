// Products of MXFP4 matrices on the block-scaled 4-bit tensor cores:
//     D[n, m] = sum_k W[n, k] X[m, k]        (tcgen05 kind::mxf4, fp32 in TMEM)
// The tensor core takes the elements as they are stored (two per byte, K-major)
// and applies both operands' power-of-two scales itself, so nothing is
// decoded: a CTA streams codes and scales to shared memory and issues MMAs.
// With bf16 activations every row of X is eight MXFP4 rows whose sum it is
// (mq_mx4.cuh), and the epilogue adds their eight columns of D.
//
// Weights are the MMA's M operand (128 rows a tile), rows of X its N operand
// (BN of them), so that a few tokens still fill the tensor core.
//
// Work: one cluster of CS CTAs per output tile, each CTA a contiguous share of
// K; the parts are summed through distributed shared memory, in CTA order
// (deterministic, no workspace).
//
// Roles: a warp whose one thread loads (TMA for the codes, one bulk copy per
// row band for the scales), a warp whose one thread copies the scales to TMEM
// and issues the MMAs, four warps for the epilogue.  Scales have their own
// TMEM columns for each stage of the shared-memory ring, so a stage's scales
// are overwritten only once its MMAs are done.
//
// Every wait is bounded (about a second); one that gives up sets a CTA abort
// flag and the device flag read by mq_device_status.  Copies and MMAs in
// flight land before the CTA exits.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "mq_mx4.cuh"
#include "mq_sm100.cuh"

namespace mq {
mq_status launch_mx_slices(const uint16_t *X, int64_t M, int64_t K, int64_t ldx, uint8_t *codes,
                           uint8_t *scales, cudaStream_t st);
namespace {

using namespace sm100;

constexpr int kTileN = 128;                  // weight rows per tile (MMA M)
constexpr int kTileK = 256;                  // columns per stage (128 bytes of codes a row)
constexpr int kThreads = 192;
constexpr int kEpiW0 = 2;                    // first epilogue warp

__device__ unsigned int g_mx_timeout;        // set when a bounded wait gave up

#ifdef MQ_TEST_HOOKS
// Test-hook builds only: while positive, a CTA drops its loads, so that the
// waits for them run out (the timeout path, with no fault and no trap).
__device__ int g_test_drop_mx4;
#endif

template <int BN>
struct MxCfg {
    static constexpr int kBands = BN > 128 ? 2 : 1;                 // 128-row bands of the N operand
    static constexpr uint32_t kA = kTileN * 128, kB = BN * 128;     // codes of a stage
    static constexpr uint32_t kSfA = 1024, kSfB = 1024 * kBands;    // scales of a stage
    static constexpr uint32_t kStage = kA + kB + kSfA + kSfB;       // a multiple of 1024
    // two CTAs an SM up to 64 columns, one above
    static constexpr int kStages = (int)(((BN <= 64 ? 113 : 226) * 1024 - 2048) / kStage) < 8
                                       ? (int)(((BN <= 64 ? 113 : 226) * 1024 - 2048) / kStage) : 8;
    static constexpr uint32_t kSfCols = 8 + 8 * kBands;             // TMEM columns of a stage's scales
    static constexpr uint32_t kD = 0, kSf = BN < 32 ? 32 : BN;      // TMEM: accumulator, then scales
    static constexpr uint32_t kCols = kSf + kStages * kSfCols <= 256 ? 256 : 512;
    static_assert(kSf + kStages * kSfCols <= kCols, "TMEM columns");
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + 1024;
    // the parts of a split tile lie in the ring: 128 x BN fp32
    static_assert((size_t)kStages * kStage >= (size_t)BN * kTileN * 4, "parts fit the ring");
};

struct MxArgs {
    CUtensorMap wmap, xmap;        // codes as (K / 2 bytes, rows), boxes 128 x 128 and 128 x BN
    const uint8_t *ws, *xs;        // scales
    void *Y;
    int64_t ldy;
    int M, N;                      // rows of X before slicing, output features
    int64_t K, G;                  // columns, 128-column groups
    int MB, KT, CS;                // X tiles, K tiles, CTAs per output tile
    int slices;                    // 1, or kMxSlices columns of D per row of X
    int out;                       // type of Y
};

__device__ __forceinline__ void store_y(const MxArgs &a, int64_t m, int64_t n, float v) {
    const int64_t at = m * a.ldy + n;
    if (a.out == MQ_BF16) static_cast<__nv_bfloat16 *>(a.Y)[at] = __float2bfloat16_rn(v);
    else if (a.out == MQ_F16) static_cast<__half *>(a.Y)[at] = __float2half_rn(v);
    else static_cast<float *>(a.Y)[at] = v;
}

template <int BN>
__global__ void __launch_bounds__(kThreads)
mx4_gemm_kernel(const __grid_constant__ MxArgs a) {
    using C = MxCfg<BN>;
    constexpr int kS = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kS * C::kStage), *empty = full + kS, *done = empty + kS;
    volatile int *flags = reinterpret_cast<volatile int *>(done + 1);   // [0] abort [1] loads [2] MMA stages
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1) + 4;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = a.CS > 1 ? (int)(blockIdx.x % a.CS) : 0;
    const int tile = (int)(blockIdx.x / a.CS), t = tile / a.MB, mb = tile % a.MB;
    const int k0 = (int)((int64_t)rank * a.KT / a.CS), k1 = (int)((int64_t)(rank + 1) * a.KT / a.CS);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kS; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        mbar_init(done, 1);
        flags[0] = flags[1] = flags[2] = 0;
        fence_mbar_init();
    }
    // the operands may come from the previous kernel; tensor memory is taken
    // after it too, so that it never waits for columns held here
    pdl_wait();
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(tmem_slot);

    if (warp == 0) {
        // -------------------------------------------------------------- loads
        const int64_t xband = (int64_t)mb * BN / 128, xbands = ((int64_t)a.M * a.slices + 127) / 128;
        const int bands = xbands - xband < C::kBands ? (int)(xbands - xband) : C::kBands;
        for (int i = 0; i < k1 - k0; ++i) {
            const int st = i % kS, kt = k0 + i;
#ifdef MQ_TEST_HOOKS
            if (i == 0) {
                const int drop = lane == 0 ? atomicSub(&g_test_drop_mx4, 1) : 0;
                if (__any_sync(0xFFFFFFFFu, drop > 0)) break;
            }
#endif
            const bool ok = i < kS || mbar_wait_backoff(empty + st, (uint32_t)(i / kS - 1) & 1u, flags);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            if (elect_one()) {
                uint8_t *sA = smem + st * C::kStage, *sB = sA + C::kA, *sfA = sB + C::kB, *sfB = sfA + C::kSfA;
                const uint32_t sfbytes = 512u * (uint32_t)(a.G - 2 * kt < 2 ? a.G - 2 * kt : 2);
                mbar_expect_tx(full + st, C::kA + C::kB + sfbytes * (1 + bands));
                tma_load_2d(sA, &a.wmap, kt * 128, t * kTileN, full + st);
                tma_load_2d(sB, &a.xmap, kt * 128, mb * BN, full + st);
                bulk_g2s(sfA, a.ws + ((int64_t)t * a.G + 2 * kt) * 512, sfbytes, full + st);
                for (int b = 0; b < bands; ++b)
                    bulk_g2s(sfB + b * 1024, a.xs + ((xband + b) * a.G + 2 * kt) * 512, sfbytes, full + st);
                flags[1] = i + 1;
            }
            __syncwarp();
        }
    } else if (warp == 1) {
        // --------------------------------------------------------------- MMAs
        for (int i = 0; i < k1 - k0; ++i) {
            const int st = i % kS;
            const bool ok = mbar_wait_abortable(full + st, (uint32_t)(i / kS) & 1u, flags);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            tc_fence_after();
            const int64_t left = a.K - (int64_t)(k0 + i) * kTileK;
            if (elect_one()) {
                const uint32_t sA = smem_u32(smem + st * C::kStage), sB = sA + C::kA, sfA = sB + C::kB,
                               sfB = sfA + C::kSfA;
                const uint32_t tA = tmem + C::kSf + st * C::kSfCols, tB = tA + 8;
                const uint64_t ad = smem_desc_sw128(sA), bd = smem_desc_sw128(sB);
                const int steps = left >= kTileK ? 4 : (int)((left + 63) / 64);
                // scales: four columns per 128 rows and group
#pragma unroll
                for (int g = 0; g < 2; ++g)
                    if (2 * g < steps) {
                        tmem_cp_sf(tA + 4 * g, smem_desc_sf(sfA + 512 * g));
#pragma unroll
                        for (int b = 0; b < C::kBands; ++b)
                            tmem_cp_sf(tB + 4 * (C::kBands * g + b), smem_desc_sf(sfB + 1024 * b + 512 * g));
                    }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < steps)
                        mma_mxf4(tmem + C::kD, ad + 2 * j, bd + 2 * j, idesc_mxf4(kTileN, BN, (j & 1) * 2),
                                 tA + 4 * (j >> 1), tB + 4 * C::kBands * (j >> 1), i + j > 0 ? 1u : 0u);
                mma_commit(empty + st);
                if (i == k1 - k0 - 1) mma_commit(done);
                flags[2] = i + 1;
            }
            __syncwarp();
        }
    }
    __syncwarp();

    // ------------------------------------------------------------ epilogue
    bool ok = true;
    const int q = warp & 3, row = 32 * q + lane;              // TMEM lane quarter of this warp
    const int64_t n = (int64_t)t * kTileN + row;
    const int cols = BN / a.slices;                           // rows of X of this tile
    const int64_t m0 = (int64_t)mb * cols;
    float *part = reinterpret_cast<float *>(smem);            // [column][128], once the ring is idle
    if (warp >= kEpiW0) {
        ok = mbar_wait_backoff(done, 0, flags);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        if (ok) {
            const uint32_t base = tmem + C::kD + ((uint32_t)(32 * q) << 16);
#pragma unroll 1
            for (int c = 0; c < BN; c += 8) {
                if (m0 + c / a.slices >= a.M) break;
                uint32_t v[8];
                tmem_ld8(base + c, v);
                tmem_ld_wait();
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = __uint_as_float(v[j]);
                int cnt = 8, col = c;
                if (a.slices == kMxSlices) {                  // small slices first
                    float s = y[7];
#pragma unroll
                    for (int j = 6; j >= 0; --j) s += y[j];
                    y[0] = s;
                    cnt = 1;
                    col = c / kMxSlices;
                }
                for (int j = 0; j < cnt; ++j) {
                    if (a.CS > 1) part[(col + j) * kTileN + row] = y[j];
                    else if (n < a.N && m0 + col + j < a.M) store_y(a, m0 + col + j, n, y[j]);
                }
            }
        }
        tc_fence_before();
    }
    if (a.CS > 1) {
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        if (warp >= kEpiW0 && ok) {
            // 32-row pieces of the tile's columns, dealt to the CTAs in turn
            const int live = a.M - m0 < cols ? (int)(a.M - m0) : cols;
            for (int u = rank * 4 + (warp - kEpiW0); u < live * 4; u += a.CS * 4) {
                const int col = u >> 2, r = 32 * (u & 3) + lane;
                const uint32_t at = smem_u32(part + col * kTileN + r);
                float y = 0.f;
                for (int c = 0; c < a.CS; ++c) y += ld_cluster_f32(cluster_map(at, (uint32_t)c));
                const int64_t nn = (int64_t)t * kTileN + r;
                if (nn < a.N) store_y(a, m0 + col, nn, y);
            }
        }
        __syncwarp();
        cluster_arrive();                                     // no CTA leaves while its part is read
        cluster_wait();
    }

    // ---- end: copies and MMAs in flight land (already so unless a wait gave up)
    __syncthreads();
    if (threadIdx.x == 0 && flags[0]) {
        atomicOr(&g_mx_timeout, 1u);
        for (int s = 0; s < kS && s < flags[1]; ++s)
            mbar_wait_bounded(full + s, (uint32_t)((flags[1] - 1 - s) / kS) & 1u);
        for (int s = 0; s < kS && s < flags[2]; ++s)
            mbar_wait_bounded(empty + s, (uint32_t)((flags[2] - 1 - s) / kS) & 1u);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kCols);
    }
}

using MxFn = void (*)(MxArgs);

template <int BN>
cudaError_t pick(MxFn *fn, size_t *smem) {
    static std::atomic<uint64_t> done{0};
    *fn = mx4_gemm_kernel<BN>;
    *smem = MxCfg<BN>::kSmem;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(*fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)MxCfg<BN>::kSmem);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

mq_status launch(const MxProduct &p, cudaStream_t st) {
    if (mx_pair_takes(p)) return launch_mx_pair(p, st);
    const mq_mx4 *w = p.w;
    const int64_t cols = p.M * p.slices;
    const int BN = cols <= 8 ? 8 : cols <= 16 ? 16 : cols <= 32 ? 32 : cols <= 64 ? 64 : cols <= 128 ? 128 : 256;
    MxFn fn;
    size_t smem;
    const cudaError_t pe = BN == 8    ? pick<8>(&fn, &smem)
                           : BN == 16  ? pick<16>(&fn, &smem)
                           : BN == 32  ? pick<32>(&fn, &smem)
                           : BN == 64  ? pick<64>(&fn, &smem)
                           : BN == 128 ? pick<128>(&fn, &smem)
                                       : pick<256>(&fn, &smem);
    if (pe != cudaSuccess) return cuda_fail(pe, "cudaFuncSetAttribute");
    MxArgs a{};
    if (!mx_encode_codes(&a.wmap, w->codes, w->rows, w->K, kTileN) ||
        !mx_encode_codes(&a.xmap, p.xcodes, cols, w->K, BN))
        return fail(MQ_ERR_CUDA, "cuTensorMapEncodeTiled (MXFP4 codes)");
    a.ws = w->scales;
    a.xs = p.xscales;
    a.Y = p.Y;
    a.ldy = p.ldy;
    a.M = (int)p.M;
    a.N = (int)w->rows;
    a.K = w->K;
    a.G = mx_groups(w->K);
    a.MB = (int)((cols + BN - 1) / BN);
    a.KT = (int)((w->K + kTileK - 1) / kTileK);
    a.slices = p.slices;
    a.out = p.out;
    const int64_t tiles = (w->rows + kTileN - 1) / kTileN * a.MB;
    // K is split while the CTAs still fit the GPU once and each keeps two
    // stages of K
    a.CS = 1;
    while (a.CS < 8 && tiles * a.CS * 2 <= 148 && a.KT >= a.CS * 4) a.CS *= 2;
    if (tiles * a.CS > 0x7FFFFFFF) return fail(MQ_ERR_UNSUPPORTED, "mq_mx4_gemm: too many output tiles");
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.CS;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * a.CS));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, a);
    return e == cudaSuccess ? MQ_OK : cuda_fail(e, "mx4_gemm_kernel");
}

mq_status check_y(const char *what, int64_t N, const void *Y, int dtype, int64_t ldy) {
    if (dtype != MQ_BF16 && dtype != MQ_F16 && dtype != MQ_F32)
        return failf(MQ_ERR_INVALID_ARG, "%s: unknown y_dtype", what);
    if (ldy < N || ldy > INT64_MAX / 8) return failf(MQ_ERR_INVALID_ARG, "%s: need ldy >= N", what);
    if (!Y) return failf(MQ_ERR_INVALID_ARG, "%s: Y is NULL", what);
    if (!aligned16(Y)) return failf(MQ_ERR_MISALIGNED, "%s: Y must be 16-byte aligned", what);
    return MQ_OK;
}

// Workspace of mq_mx4_gemm_bf16: the slices' codes, then their scales.
size_t slice_code_bytes(int64_t M, int64_t K) {
    return ((size_t)M * kMxSlices * (size_t)(K / 2) + 15) / 16 * 16;
}

}  // namespace

PFN_cuTensorMapEncodeTiled_v12000 mx_encoder() {
    static std::atomic<void *> cached{nullptr};
    void *f = cached.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        cached.store(f, std::memory_order_release);
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
}

bool mx_encode_codes(CUtensorMap *map, const uint8_t *codes, int64_t rows, int64_t K, int box) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = mx_encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)(K / 2), (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(K / 2)};
    const cuuint32_t boxes[2] = {128, (cuuint32_t)box}, estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(codes), dims, strides, boxes, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool mx_encode_scales(CUtensorMap *map, const uint8_t *scales, int64_t rows, int64_t K, int box) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = mx_encoder();
    if (!enc) return false;
    const int64_t G = mx_groups(K);
    const cuuint64_t dims[2] = {(cuuint64_t)G * 128, (cuuint64_t)((rows + 127) / 128)};
    const cuuint64_t strides[1] = {(cuuint64_t)G * 512};
    const cuuint32_t boxes[2] = {256, (cuuint32_t)box}, estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t *>(scales), dims, strides, boxes, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool mx_encode_y(CUtensorMap *map, void *Y, int64_t M, int64_t N, int64_t ldy, int out) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = mx_encoder();
    if (!enc) return false;
    const int size = out == MQ_F32 ? 4 : 2;
    const cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)M};
    const cuuint64_t strides[1] = {(cuuint64_t)(ldy * size)};
    const cuuint32_t boxes[2] = {(cuuint32_t)(128 / size), 32}, estr[2] = {1, 1};
    const CUtensorMapDataType t = out == MQ_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                  : out == MQ_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                  : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return enc(map, t, 2, Y, dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool mx4_take_timeout(bool *set) {
    unsigned v = 0, z = 0;
    bool pair = false;
    if (!mx_pair_take_timeout(&pair)) return false;
    if (cudaMemcpyFromSymbol(&v, g_mx_timeout, sizeof(v)) != cudaSuccess) return false;
    if (v && cudaMemcpyToSymbol(g_mx_timeout, &z, sizeof(z)) != cudaSuccess) return false;
    *set = v != 0 || pair;
    return true;
}

}  // namespace mq

using namespace mq;

extern "C" mq_status mq_mx4_gemm(const mq_mx4 *X, const mq_mx4 *w, void *Y, int y_dtype, int64_t ldy,
                                 void *stream) {
    mq_status s = check_mx4(X, "mq_mx4_gemm (X)");
    if (s != MQ_OK) return s;
    if ((s = check_mx4(w, "mq_mx4_gemm (w)")) != MQ_OK) return s;
    if (X->K != w->K) return fail(MQ_ERR_INVALID_ARG, "mq_mx4_gemm: X and w differ in K");
    if (w->rows < 1) return fail(MQ_ERR_INVALID_ARG, "mq_mx4_gemm: w has no rows");
    if (X->rows == 0) return MQ_OK;
    if ((s = check_y("mq_mx4_gemm", w->rows, Y, y_dtype, ldy)) != MQ_OK) return s;
    cudaStream_t st = (cudaStream_t)stream;
    if ((s = bind_device(st)) != MQ_OK) return s;
    return launch(MxProduct{X->codes, X->scales, X->rows, 1, w, Y, y_dtype, ldy}, st);
}

extern "C" size_t mq_mx4_gemm_bf16_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (M < 1 || M > kMxMaxDim / kMxSlices || N < 1 || N > kMxMaxDim || K < kMxBlock || K % kMxBlock || K > kMxMaxDim)
        return 0;
    return slice_code_bytes(M, K) + mq_mx4_scale_bytes(M * kMxSlices, K);
}

extern "C" mq_status mq_mx4_gemm_bf16(const uint16_t *X, int64_t M, int64_t ldx, const mq_mx4 *w, void *Y,
                                      int y_dtype, int64_t ldy, void *workspace, size_t workspace_bytes,
                                      void *stream) {
    mq_status s = check_mx4(w, "mq_mx4_gemm_bf16 (w)");
    if (s != MQ_OK) return s;
    if (w->rows < 1) return fail(MQ_ERR_INVALID_ARG, "mq_mx4_gemm_bf16: w has no rows");
    if (M < 0 || M > kMxMaxDim / kMxSlices) return fail(MQ_ERR_INVALID_ARG, "mq_mx4_gemm_bf16: M out of range");
    if (M == 0) return MQ_OK;
    if (!X) return fail(MQ_ERR_INVALID_ARG, "mq_mx4_gemm_bf16: X is NULL");
    if (ldx < w->K || ldx > INT64_MAX / 8) return fail(MQ_ERR_INVALID_ARG, "mq_mx4_gemm_bf16: need ldx >= K");
    if (!aligned16(X) || (M > 1 && ldx % 8) || (workspace && !aligned16(workspace)))
        return fail(MQ_ERR_MISALIGNED, "mq_mx4_gemm_bf16: X, its row stride and the workspace must be 16-byte aligned");
    if ((s = check_y("mq_mx4_gemm_bf16", w->rows, Y, y_dtype, ldy)) != MQ_OK) return s;
    const size_t need = mq_mx4_gemm_bf16_workspace_bytes(M, w->rows, w->K);
    if (need && (!workspace || workspace_bytes < need))
        return fail(MQ_ERR_WORKSPACE, "workspace smaller than mq_mx4_gemm_bf16_workspace_bytes");
    cudaStream_t st = (cudaStream_t)stream;
    if ((s = bind_device(st)) != MQ_OK) return s;
    uint8_t *codes = static_cast<uint8_t *>(workspace), *scales = codes + slice_code_bytes(M, w->K);
    if ((s = launch_mx_slices(X, M, w->K, ldx, codes, scales, st)) != MQ_OK) return s;
    return launch(MxProduct{codes, scales, M, kMxSlices, w, Y, y_dtype, ldy}, st);
}

#ifdef MQ_TEST_HOOKS
// Test-hook builds only: make the next `n` CTAs of an MXFP4 product drop their loads.
namespace mq {
int pair_test_drop(int n);
}
extern "C" __attribute__((visibility("default"))) int mq_test_drop_mx4_loads(int n) {
    const int e = mq::pair_test_drop(n);
    return e ? e : (int)cudaMemcpyToSymbol(mq::g_test_drop_mx4, &n, sizeof(n));
}
#endif
