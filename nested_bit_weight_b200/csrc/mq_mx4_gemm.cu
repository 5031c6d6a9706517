// Products of MXFP4 matrices on the block-scaled 4-bit tensor cores:
//     D[n, m] = sum_k W[n, k] X[m, k]        (tcgen05 kind::mxf4, fp32 in TMEM)
// The tensor core takes the elements as they are stored (two per byte, K-major)
// and applies both operands' power-of-two scales itself, so nothing is
// decoded: a CTA streams codes and scales to shared memory and issues MMAs.
// With bf16 activations every row of X is eight MXFP4 rows whose sum it is
// (mq_mx4.cuh), and the epilogue adds their eight columns of D.  This kernel
// serves up to 128 MXFP4 rows; more go to the pair product (mq_mx4_pair.cu).
//
// Weights are the MMA's M operand (128 rows a tile), rows of X its N operand
// (BN of them), so that a few tokens still fill the tensor core.
//
// Work: one cluster of CS CTAs per output tile, each CTA a contiguous share of
// K; the parts are summed through distributed shared memory, in CTA order
// (deterministic, no workspace): each CTA stores its part of four columns
// straight from registers to the CTA that owns them, and the stores complete
// on that CTA's barrier, so that no CTA waits for another but the owner for what
// it is sent (two cluster barriers and copies out of shared memory took 1.8 of
// 8.8 us for one token through 14336 x 4096).
//
// Roles: a warp that loads (TMA for the codes, bulk copies for the scales), a
// warp that copies the scales to TMEM and issues the MMAs, four warps for the
// epilogue.  With up to four bf16 rows (FUSED) those four make the eight MXFP4
// rows of each row themselves, a stage at a time, straight into the MMA's
// operand; every CTA repeats that small work, and a launch and a pass through
// memory are saved.  Scales have their own TMEM columns for each stage of the
// shared-memory ring, so a stage's scales are overwritten only once its MMAs
// are done.
//
// Programmatic dependent launch: nothing is read or written before
// griddepcontrol.wait; the weights are only brought into L2 before it.
//
// Bound by HBM for large weights (one token through 28672 x 8192: 23 us, 5.5 TB/s),
// by its start and end for small ones (1024 x 4096: 3.6 us, 14336 x 4096: 8.6 us
// of which 4.8 are HBM's), above 64 rows by the parts' way to their owner
// (128 x 4096 x 14336: 14 us).
//
// Every wait is bounded (about a second); one that gives up sets a CTA abort
// flag and the device flag read by mq_device_status.  Copies and MMAs in
// flight land before the CTA exits, and a CTA that gave up stays until the others
// of its cluster have ended or given up too, since they may still send it parts.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "mq_mx4.cuh"
#include "mq_sm100.cuh"

namespace mq {
namespace {

using namespace sm100;

constexpr int kTileN = 128;                  // weight rows per tile (MMA M)
constexpr int kTileK = 256;                  // columns per stage (128 bytes of codes a row)
constexpr int kThreads = 192;
constexpr int kMinStages = 4;                // of K for each CTA of a split
constexpr int kEpiW0 = 2;                    // first epilogue warp

__device__ unsigned int g_mx_timeout;        // set when a bounded wait gave up

#ifdef MQ_TEST_HOOKS
// Test-hook builds only: while positive, a CTA drops its loads, so that the
// waits for them run out (the timeout path, with no fault and no trap); while
// set, the last CTA of each cluster sends its parts only after the others' waits
// for them have run out.
__device__ int g_test_drop_mx4, g_test_late_mx4;
#endif

template <int BN>
struct MxCfg {
    static_assert(BN <= 128, "one row band of scales");
    static constexpr uint32_t kA = kTileN * 128, kB = BN * 128;     // codes of a stage
    static constexpr uint32_t kSfA = 1024, kSfB = 1024;    // scales of a stage
    static constexpr uint32_t kStage = kA + kB + kSfA + kSfB;       // a multiple of 1024
    // parts sent to this CTA: [CTA][owned columns / 4][128][4] fp32, at least four
    // columns for each of eight CTAs
    static constexpr uint32_t kParts = (BN < 32 ? 32 : BN) * kTileN * 4;
    // two CTAs an SM up to 32 columns, one above
    static constexpr int kPerSm = BN <= 32 ? 2 : 1;
    static constexpr int kRoom = (kPerSm == 2 ? 113 : 226) * 1024 - 2048 - (int)kParts;
    static constexpr int kStages = kRoom / (int)kStage < 6 ? kRoom / (int)kStage : 6;
    static constexpr uint32_t kSfCols = 16;           // TMEM columns of a stage's scales
    static constexpr uint32_t kSf = BN < 32 ? 32 : BN;              // TMEM: accumulator, then scales
    static constexpr uint32_t kCols = kSf + kStages * kSfCols <= 256 ? 256 : 512;
    static_assert(kSf + kStages * kSfCols <= kCols, "TMEM columns");
    // With one row of X the four slicing warps are on four stages at once: in a
    // shorter ring one of them would wait two phases ahead of a barrier, which
    // its parity cannot express.
    static_assert(kStages >= 4, "ring");
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + kParts + 1024;
    // no more CTAs on an SM than tensor memory has room for
    static_assert((512 / kCols + 1) * kSmem > 228 * 1024, "CTAs an SM");
};

struct MxArgs {
    CUtensorMap wmap, xmap;        // codes as (K / 2 bytes, rows), boxes 128 x 128 and 128 x BN
    const uint8_t *ws, *xs;        // scales
    const uint8_t *X;              // FUSED: bf16 rows and their stride in bytes
    int64_t ldx_bytes;
    void *Y;
    int64_t ldy;
    int M, N;                      // rows of X before slicing, output features
    int64_t K, G;                  // columns, 128-column groups
    int KT, CS;                    // K tiles, CTAs per output tile
    int lper;                      // log2 of the columns a CTA of a cluster adds up, at least 2
    int slices;                    // 1, or kMxSlices columns of D per row of X
    int out;                       // type of Y
};

// Whether bf16 rows are cut into slices inside the product.  Cutting a row is one
// chain of dependent operations, about 700 clocks a stage, which the four warps run
// side by side: on different stages (one or two rows), on different rows (three or
// four).  That keeps up with one or two rows always.  With three or four the
// weights decide; four rows, against a kernel of their own before: 1024 x 4096 4.8
// us against 6.1, 4096 x 4096 5.0 against 6.4, the same from 14336 x 4096 (11.5) to
// 8192 x 8192 (12.1 against 12.0, 2^26 weights; there it saves the workspace),
// 10240 x 8192 19.0 against 14.6, 28672 x 8192 34 against 26.5.
bool fused_rows(int64_t M, int64_t N, int64_t K) { return M <= 2 || (M <= 4 && N * K <= (int64_t)1 << 26); }

template <class T>
__device__ __forceinline__ T to(float v);
template <>
__device__ __forceinline__ float to<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half to<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 to<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Rows m0 .. m0 + 3 (those below M) of feature n to Y.
template <class T>
__device__ __forceinline__ void store4(const MxArgs &a, int m0, int64_t n, const float (&y)[4]) {
    T *dst = static_cast<T *>(a.Y) + (int64_t)m0 * a.ldy + n;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (m0 + e < a.M) *dst = to<T>(y[e]);
        dst += a.ldy;
    }
}

// The accumulator's `live` columns of this thread's row (with slices, each the
// sum of eight), four at a time, to put(column, values).
template <int BN, class Put>
__device__ __forceinline__ void read_columns(uint32_t base, int slices, int live, Put put) {
    constexpr int kStep = BN < 32 ? BN : 32;
#pragma unroll 1
    for (int c = 0; c < BN; c += kStep) {
        if (c / slices >= live) break;
        __syncwarp();                        // lanes of features beyond N left the last stores early
        uint32_t v[kStep];
        if constexpr (kStep == 8) tmem_ld8(base + c, v);
        else if constexpr (kStep == 16) tmem_ld16(base + c, v);
        else tmem_ld32(base + c, v);
        tmem_ld_wait();
        if (slices == kMxSlices) {
            float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < kStep / kMxSlices; ++e) {             // small slices first
                y[e] = __uint_as_float(v[kMxSlices * e + kMxSlices - 1]);
#pragma unroll
                for (int j = kMxSlices - 2; j >= 0; --j) y[e] += __uint_as_float(v[kMxSlices * e + j]);
            }
            put(c / kMxSlices, y);
        } else {
#pragma unroll
            for (int g = 0; g < kStep / 4; ++g) {
                const float y[4] = {__uint_as_float(v[4 * g]), __uint_as_float(v[4 * g + 1]),
                                    __uint_as_float(v[4 * g + 2]), __uint_as_float(v[4 * g + 3])};
                if (c + 4 * g < live) put(c + 4 * g, y);
            }
        }
    }
}

// The epilogue warps have read tensor memory: the MMA warp may give it back.  It
// does so before any CTA waits for another's parts: a CTA that held columns
// while it waited for one that still wants them could lock up with another
// kernel's cluster that does the same the other way round.
__device__ __forceinline__ void tmem_read() {
    __syncwarp();
    tc_fence_before();
    named_arrive(2, 160);
}

// Epilogue of one thread: its row of the tile, straight to Y or in parts to the
// CTAs that own the columns, which then add what they were sent.
template <int BN, class T>
__device__ __forceinline__ void epilogue(const MxArgs &a, uint32_t base, float *parts, uint64_t *sent, int rank,
                                         int64_t n, int row, bool ok, volatile int *flags) {
    if (a.CS == 1) {
        if (ok)
            read_columns<BN>(base, a.slices, a.M, [&](int col, const float (&y)[4]) {
                if (n < a.N) store4<T>(a, col, n, y);
            });
        tmem_read();
        return;
    }
    const int lper = a.lper, first = rank << lper, left = a.M - first, per = 1 << lper;
    const int groups = ((left < per ? left : per) + 3) / 4;   // of four columns owned; <= 0: none
    float4 *const p4 = reinterpret_cast<float4 *>(parts);     // [CTA][group][row]
#ifdef MQ_TEST_HOOKS
    if (g_test_late_mx4 && rank == a.CS - 1)
        for (const uint64_t t0 = global_ns(); global_ns() - t0 < 4 * kWaitNs;) __nanosleep(1000);
#endif
    if (ok) {
        const uint32_t to0 = smem_u32(p4 + ((size_t)rank << (lper - 2)) * kTileN + row), bar0 = smem_u32(sent);
        read_columns<BN>(base, a.slices, a.M, [&](int col, const float (&y)[4]) {
            const uint32_t owner = (uint32_t)(col >> lper), at = to0 + (uint32_t)((col & (per - 1)) >> 2) * (kTileN * 16);
            st_async_v4(cluster_map(at, owner), y[0], y[1], y[2], y[3], cluster_map(bar0, owner));
        });
    }
    tmem_read();
    if (groups <= 0) return;
    // also when this CTA gave up: until then stores to this CTA's memory may be on
    // their way (after a wait that runs out, see the end of the kernel)
    const bool got = mbar_wait_cluster_bounded(sent, 0);
    if (!got) flags[0] = 1;
    if (!got || !ok) return;
#pragma unroll 2
    for (int g = 0; g < groups; ++g) {
        float y[4] = {0.f, 0.f, 0.f, 0.f};
        for (int c = 0; c < a.CS; ++c) {                      // in CTA order
            const float4 z = p4[(((size_t)c << (lper - 2)) + g) * kTileN + row];
            y[0] += z.x;
            y[1] += z.y;
            y[2] += z.z;
            y[3] += z.w;
        }
        if (n < a.N) store4<T>(a, first + 4 * g, n, y);
    }
}

template <int BN, bool FUSED>
__global__ void __launch_bounds__(kThreads)
mx4_gemm_kernel(const __grid_constant__ MxArgs a) {
    using C = MxCfg<BN>;
    constexpr int kS = C::kStages;
    constexpr int kPrefetch = 16;                // stages brought into L2 ahead
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float *parts = reinterpret_cast<float *>(smem + kS * C::kStage);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kS * C::kStage + C::kParts), *empty = full + kS;
    uint64_t *done = empty + kS, *sent = done + 1;
    volatile int *flags = reinterpret_cast<volatile int *>(sent + 1);   // [0] abort [1] loads
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sent + 1) + 4;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = a.CS > 1 ? (int)(blockIdx.x % a.CS) : 0;
    const int t = (int)(blockIdx.x / a.CS);      // tile: 128 features, all rows of X
    const int k0 = (int)((int64_t)rank * a.KT / a.CS), k1 = (int)((int64_t)(rank + 1) * a.KT / a.CS);

    if (threadIdx.x == 0) {
        if (!FUSED) prefetch_tensormap(&a.xmap);
        for (int i = 0; i < kPrefetch && i < k1 - k0; ++i) tma_prefetch_2d(&a.wmap, (k0 + i) * 128, t * kTileN);
        for (int i = 0; i < kS; ++i) {
            mbar_init(full + i, FUSED ? 1 + a.M : 1);   // the loads and the slicing warps
            mbar_init(empty + i, 1);
        }
        mbar_init(done, 1);
        mbar_init(sent, 1);
        flags[0] = flags[1] = 0;
        fence_mbar_init();
    }
    __syncthreads();
    if (a.CS > 1) cluster_arrive();              // this CTA's barriers are ready (waited for before the parts)
    // the operands may come from the previous kernel; tensor memory is taken
    // after it too, so that it never waits for columns held here
    pdl_wait();

    if (warp == 0) {
        // -------------------------------------------------------------- loads
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
                mbar_expect_tx(full + st, C::kA + sfbytes + (FUSED ? 0u : C::kB + sfbytes));
                tma_load_2d(sA, &a.wmap, kt * 128, t * kTileN, full + st);
                bulk_g2s(sfA, a.ws + ((int64_t)t * a.G + 2 * kt) * 512, sfbytes, full + st);
                if constexpr (!FUSED) {
                    tma_load_2d(sB, &a.xmap, kt * 128, 0, full + st);
                    bulk_g2s(sfB, a.xs + 2 * (int64_t)kt * 512, sfbytes, full + st);   // rows of X: one band
                }
                flags[1] = i + 1;
            }
            __syncwarp();
        }
    } else if (warp == 1) {
        // --------------------------------------------------------------- MMAs
        tmem_alloc(tmem_slot, C::kCols);
        tmem_relinquish();
        // only now may the next kernel start: one that takes tensor memory before
        // its own wait could otherwise hold the columns this one needs
        pdl_launch_dependents();
        named_arrive(1, 160);                    // the epilogue may read the address
        const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(tmem_slot);
        // what does not change is worked out before the loop, and the ring's slot
        // and phase are counted: see the pair product
        uint32_t st = 0, phase = 0;
        const uint32_t s0 = smem_u32(smem);
        const uint64_t ad0 = smem_desc_sw128(s0), bd0 = smem_desc_sw128(s0 + C::kA),
                       sa0 = smem_desc_sf(s0 + C::kA + C::kB), sb0 = smem_desc_sf(s0 + C::kA + C::kB + C::kSfA);
        const uint32_t idesc = idesc_mxf4(kTileN, BN, 0);
        const int64_t left = a.K - (int64_t)(k1 - 1) * kTileK;
        const int tail = left >= kTileK ? 4 : (int)((left + 63) / 64);   // MMAs of the last stage
        int i = 0;
        for (; i < k1 - k0; ++i) {
            const bool ok = mbar_wait_abortable(full + st, phase, flags);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t step = (uint64_t)st * (C::kStage >> 4);
                const uint32_t tA = tmem + C::kSf + st * C::kSfCols, tB = tA + 8;
                const int steps = i + 1 < k1 - k0 ? 4 : tail;
                // scales: four columns per 128 rows and group
                tmem_cp_sf(tA, sa0 + step);
                tmem_cp_sf(tB, sb0 + step);
                if (steps > 2) {
                    tmem_cp_sf(tA + 4, sa0 + step + 32);
                    tmem_cp_sf(tB + 4, sb0 + step + 32);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < steps)
                        mma_mxf4(tmem, ad0 + step + 2 * j, bd0 + step + 2 * j, idesc + ((j & 1) ? kIdescSf2 : 0u),
                                 tA + 4 * (j >> 1), tB + 4 * (j >> 1), i + j > 0 ? 1u : 0u);
                mma_commit(empty + st);
                if (i == k1 - k0 - 1) mma_commit(done);
            }
            __syncwarp();
            if (++st == kS) {
                st = 0;
                phase ^= 1u;
            }
        }
        // MMAs in flight land (after a wait that gave up)
        if (i > 0 && i < k1 - k0) mbar_wait_bounded(empty + (i - 1) % kS, (uint32_t)((i - 1) / kS) & 1u);
    }
    __syncwarp();

    if constexpr (FUSED) {
        if (warp >= kEpiW0) {
            // ------------------------------------------------------- slices of X
            // 256 columns of a row at a time, eight a lane; the next values are
            // loaded while the last are cut
            const int groups = 4 / a.M;                              // stages at a time
            const int m = (warp - kEpiW0) % a.M, grp = (warp - kEpiW0) / a.M;   // grp == groups: three rows, no work
            const uint8_t *xrow = a.X + m * a.ldx_bytes + lane * 16;
            const uint32_t swz = (uint32_t)(lane >> 2), at = (uint32_t)(lane & 3) * 4;
            auto load = [&](int i) {
                const int kt = k0 + i;
                return kt < k1 && (int64_t)kt * kTileK + lane * 8 < a.K
                           ? *reinterpret_cast<const uint4 *>(xrow + (int64_t)kt * kTileK * 2)
                           : make_uint4(0u, 0u, 0u, 0u);
            };
            uint4 next = load(grp);
            for (int i = grp; grp < groups && i < k1 - k0; i += groups) {
                const int st = i % kS;
                const uint32_t x[4] = {next.x, next.y, next.z, next.w};
                next = load(i + groups);
                float f[8];
                uint32_t a2 = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f[2 * j] = __uint_as_float(x[j] << 16);
                    f[2 * j + 1] = __uint_as_float(x[j] & 0xFFFF0000u);
                    a2 = __vmaxu2(a2, x[j] & 0x7FFF7FFFu);
                }
                a2 = __vmaxu2(a2, __shfl_xor_sync(0xFFFFFFFFu, a2, 1));
                a2 = __vmaxu2(a2, __shfl_xor_sync(0xFFFFFFFFu, a2, 2));
                const uint32_t E = mx_slice0_byte(max(a2 & 0xFFFFu, a2 >> 16) << 16);
                __half2 u[4] = {};
                if (E != 255u) mx_slice_start(f, mx_inverse(E), u);
                const bool ok = i < kS || mbar_wait_backoff(empty + st, (uint32_t)(i / kS - 1) & 1u, flags);
                if (!__all_sync(0xFFFFFFFFu, ok)) break;
                // eight rows of B: one swizzle atom; eight rows of its scales
                uint8_t *sB = smem + st * C::kStage + C::kA, *sf = sB + C::kB + C::kSfA + (lane >> 4) * 512 +
                                                                  m * kMxSlices * 16 + ((lane >> 2) & 3);
                sB += m * 1024 + at;
#pragma unroll
                for (int j = 0; j < kMxSlices; ++j) {
                    const uint32_t Ej = mx_slice_byte(E, j);
                    *reinterpret_cast<uint32_t *>(sB + j * 128 + ((swz ^ (uint32_t)j) << 4)) =
                        mx_slice_codes(u, Ej - mx_slice_byte(E, j + 1));
                    if ((lane & 3) == 0) sf[j * 16] = (uint8_t)Ej;
                }
                fence_proxy_async_smem();                            // the tensor core reads what was written
                __syncwarp();
                if (lane == 0) mbar_arrive(full + st);
            }
            __syncwarp();
        }
    }

    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, row = 32 * q + lane;              // TMEM lane quarter of this warp
    if (a.CS > 1) cluster_wait();
    if (warp >= kEpiW0) {
        if (a.CS > 1 && threadIdx.x == 32 * kEpiW0) {
            const int left = a.M - (rank << a.lper), own = left < (1 << a.lper) ? left : 1 << a.lper;
            if (own > 0) mbar_expect_tx(sent, (uint32_t)a.CS * (uint32_t)((own + 3) / 4) * (kTileN * 16));
        }
        bool ok = mbar_wait_backoff(done, 0, flags);
        ok = __all_sync(0xFFFFFFFFu, ok);
        named_sync(1, 160);
        tc_fence_after();
        const uint32_t base = *reinterpret_cast<volatile uint32_t *>(tmem_slot) + ((uint32_t)(32 * q) << 16);
        const int64_t n = (int64_t)t * kTileN + row;
        if (a.out == MQ_BF16) epilogue<BN, __nv_bfloat16>(a, base, parts, sent, rank, n, row, ok, flags);
        else if (a.out == MQ_F16) epilogue<BN, __half>(a, base, parts, sent, rank, n, row, ok, flags);
        else epilogue<BN, float>(a, base, parts, sent, rank, n, row, ok, flags);
    } else if (warp == 1) {
        named_sync(2, 160);
        tc_fence_after();
        tmem_dealloc(*reinterpret_cast<volatile uint32_t *>(tmem_slot), C::kCols);
    }

    // ---- end: copies in flight land (already so unless a wait gave up)
    __syncthreads();
    const bool gave_up = flags[0] != 0;                       // set by nobody from here on
    if (threadIdx.x == 0 && gave_up) {
        atomicOr(&g_mx_timeout, 1u);
        for (int s = 0; s < kS && s < flags[1]; ++s)
            mbar_wait_bounded(full + s, (uint32_t)((flags[1] - 1 - s) / kS) & 1u);
    }
    __syncwarp();
    if (a.CS > 1 && gave_up) {
        // A CTA of the cluster that is only late still sends its parts here.  Every
        // CTA ends (its waits are bounded) or comes to this barrier, and a thread
        // that has ended counts as arrived, so CTAs whose waits held pay nothing;
        // then a millisecond for stores issued just before (they take microseconds)
        cluster_arrive();
        cluster_wait();
        if (threadIdx.x == 0)
            for (const uint64_t t0 = global_ns(); global_ns() - t0 < 1000000ull;) __nanosleep(1000);
    }
    __syncthreads();                                          // shared memory stays until then
}

using MxFn = void (*)(MxArgs);

template <int BN, bool FUSED>
cudaError_t pick(MxFn *fn, size_t *smem) {
    static std::atomic<uint64_t> done{0};
    *fn = mx4_gemm_kernel<BN, FUSED>;
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
    const bool fused = p.X != nullptr;
    const int64_t cols = p.M * p.slices;
    const int BN = cols <= 8 ? 8 : cols <= 16 ? 16 : cols <= 32 ? 32 : cols <= 64 ? 64 : 128;
    MxFn fn;
    size_t smem;
    const cudaError_t pe = BN == 8    ? fused ? pick<8, true>(&fn, &smem) : pick<8, false>(&fn, &smem)
                           : BN == 16  ? fused ? pick<16, true>(&fn, &smem) : pick<16, false>(&fn, &smem)
                           : BN == 32  ? fused ? pick<32, true>(&fn, &smem) : pick<32, false>(&fn, &smem)
                           : BN == 64  ? pick<64, false>(&fn, &smem)
                                       : pick<128, false>(&fn, &smem);
    if (pe != cudaSuccess) return cuda_fail(pe, "cudaFuncSetAttribute");
    MxArgs a{};
    if (!mx_encode_codes(&a.wmap, w->codes, w->rows, w->K, kTileN) ||
        (!fused && !mx_encode_codes(&a.xmap, p.xcodes, cols, w->K, BN)))
        return fail(MQ_ERR_CUDA, "cuTensorMapEncodeTiled (MXFP4 codes)");
    a.ws = w->scales;
    a.xs = p.xscales;
    a.X = reinterpret_cast<const uint8_t *>(p.X);
    a.ldx_bytes = p.ldx * 2;
    a.Y = p.Y;
    a.ldy = p.ldy;
    a.M = (int)p.M;
    a.N = (int)w->rows;
    a.K = w->K;
    a.G = mx_groups(w->K);
    a.KT = (int)((w->K + kTileK - 1) / kTileK);
    a.slices = p.slices;
    a.out = p.out;
    const int64_t tiles = (w->rows + kTileN - 1) / kTileN;
    // K is split while the CTAs still fit the GPU once (kPerSm an SM) and each keeps
    // kMinStages of K (16 x 4096 x 4096 with two stages each took 7.2 us, with four
    // 5.3, with six 6.4)
    a.CS = 1;
    while (a.CS < 8 && tiles * a.CS * 2 <= (BN <= 32 ? 296 : 148) && a.KT >= a.CS * 2 * kMinStages) a.CS *= 2;
    for (a.lper = 2; (a.CS << a.lper) < BN / p.slices;) ++a.lper;
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

// Rows of bf16 X at most: their slices, with the rows that fill up tiles, are
// numbered in 32 bits.
constexpr int64_t kMaxRows = (int64_t)1 << 27;

// Workspace of mq_mx4_gemm_bf16: the slices' codes, then their scales.
size_t slice_code_bytes(const MxSlicing &sl, int64_t K) { return ((size_t)sl.rows * (size_t)(K / 2) + 15) / 16 * 16; }

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
    return launch(MxProduct{X->codes, X->scales, X->rows, 1, w, Y, y_dtype, ldy, nullptr, 0, {}}, st);
}

extern "C" size_t mq_mx4_gemm_bf16_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (M < 1 || M > kMaxRows || N < 1 || N > kMxMaxDim || K < kMxBlock || K % kMxBlock || K > kMxMaxDim)
        return 0;
    if (fused_rows(M, N, K)) return 0;
    const MxSlicing sl = mx_slicing(M, N);
    return slice_code_bytes(sl, K) + (size_t)sl.bands * (size_t)mx_groups(K) * 512;
}

extern "C" mq_status mq_mx4_gemm_bf16(const uint16_t *X, int64_t M, int64_t ldx, const mq_mx4 *w, void *Y,
                                      int y_dtype, int64_t ldy, void *workspace, size_t workspace_bytes,
                                      void *stream) {
    mq_status s = check_mx4(w, "mq_mx4_gemm_bf16 (w)");
    if (s != MQ_OK) return s;
    if (w->rows < 1) return fail(MQ_ERR_INVALID_ARG, "mq_mx4_gemm_bf16: w has no rows");
    if (M < 0 || M > kMaxRows) return fail(MQ_ERR_INVALID_ARG, "mq_mx4_gemm_bf16: M out of range");
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
    MxProduct p{nullptr, nullptr, M, kMxSlices, w, Y, y_dtype, ldy, nullptr, 0, {}};
    if (fused_rows(M, w->rows, w->K)) {
        p.X = X;
        p.ldx = ldx;
        return launch(p, st);
    }
    p.slice = mx_slicing(M, w->rows);
    uint8_t *codes = static_cast<uint8_t *>(workspace), *scales = codes + slice_code_bytes(p.slice, w->K);
    if ((s = launch_mx_slices(X, M, w->K, ldx, p.slice, codes, scales, st)) != MQ_OK) return s;
    p.xcodes = codes;
    p.xscales = scales;
    return launch(p, st);
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
// Make the last CTA of each cluster send its parts late (0: no longer).
extern "C" __attribute__((visibility("default"))) int mq_test_late_mx4_parts(int on) {
    return (int)cudaMemcpyToSymbol(mq::g_test_late_mx4, &on, sizeof(on));
}
#endif
