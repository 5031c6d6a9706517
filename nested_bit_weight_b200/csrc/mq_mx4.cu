// MXFP4 converters (include/mq.h): dense rows and nested parents to MXFP4,
// MXFP4 to dense values, and bf16 rows to sums of MXFP4 rows.  All are bound
// by HBM (a few operations per element), so what counts is that loads and
// stores are wide and that several are in flight per thread.
#include "mq_bits.cuh"
#include "mq_mx4.cuh"
#include "mq_sm100.cuh"

namespace mq {
namespace {

// Two fp32 numbers in one 64-bit register pair (one instruction for both).
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Eight numbers times f to eight codes.
__device__ __forceinline__ uint32_t scaled_codes8(const float (&u)[8], float f) {
    const uint64_t ff = pair(f, f);
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpair(mul2(pair(u[2 * i], u[2 * i + 1]), ff), v[2 * i], v[2 * i + 1]);
    return mx_codes8(v);
}

// The larger magnitude of both halves (or of one number); a NaN wins, the signs
// are left meaningless.
template <int DT>
__device__ __forceinline__ uint32_t max_abs(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (DT == MQ_BF16) asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else if constexpr (DT == MQ_F16) asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// N consecutive elements of one lane as loaded: 16-byte words, or 32-byte ones
// where the rows are aligned to that.
template <int DT, int N>
struct Raw {
    static constexpr int kBytes = DT == MQ_F32 ? 4 : 2, kWords = N * kBytes / 4;
    uint32_t w[kWords];
    template <bool WIDE>
    __device__ void load(const void *p) {
        if constexpr (WIDE) {
#pragma unroll
            for (int i = 0; i < kWords; i += 8)
                asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                             : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]), "=r"(w[i + 4]),
                               "=r"(w[i + 5]), "=r"(w[i + 6]), "=r"(w[i + 7])
                             : "l"(static_cast<const uint8_t *>(p) + 4 * i));
        } else {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const uint4 v = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p) + 4 * i);
                w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
            }
        }
    }
    __device__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    // Largest magnitude of the 32 / N adjacent lanes that hold a block, as fp32 bits.
    __device__ uint32_t amax() const {
        uint32_t m = w[0];
#pragma unroll
        for (int i = 1; i < kWords; ++i) m = max_abs<DT>(m, w[i]);
#pragma unroll
        for (int l = 1; l < 32 / N; l *= 2) m = max_abs<DT>(m, __shfl_xor_sync(0xFFFFFFFFu, m, l));
        if constexpr (DT == MQ_F32) return m & 0x7FFFFFFFu;
        m = max_abs<DT>(m, m >> 16) & 0x7FFFu;
        if constexpr (DT == MQ_BF16) return m << 16;
        return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
    }
    // Eight of the elements as fp32, from element 8 h.
    __device__ void get(int h, float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == MQ_F32) {
                f[2 * i] = __uint_as_float(w[8 * h + 2 * i]);
                f[2 * i + 1] = __uint_as_float(w[8 * h + 2 * i + 1]);
            } else if constexpr (DT == MQ_BF16) {
                f[2 * i] = __uint_as_float(w[4 * h + i] << 16);
                f[2 * i + 1] = __uint_as_float(w[4 * h + i] & 0xFFFF0000u);
            } else {
                const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&w[4 * h + i]));
                f[2 * i] = t.x;
                f[2 * i + 1] = t.y;
            }
        }
    }
};

// Rows per warp and step: so many loads of a thread are in flight.
__host__ __device__ constexpr int quant_rows(int dtype) { return dtype == MQ_F32 ? 2 : 4; }
constexpr int kQuantCols = 512;               // columns of a warp, 16 a lane
constexpr int kDeqRows = 4;

// One warp: 512 columns of a few rows (all in one 128-row band).  Steps beyond
// the matrix (the padding rows and columns of the scale blocks) write zero scale
// bytes only.  8192 x 4096 bf16 in 14.6 us (5.8 TB/s), 14336 x 4096 fp32 in 40 us
// (6.6 TB/s): HBM.  Eight elements a lane with 16-byte loads took 17.9 us.
template <int DT, bool WIDE>
__global__ void __launch_bounds__(256)
mx_quantize_kernel(const uint8_t *__restrict__ X, int64_t rows, int64_t K, int64_t ld_bytes, uint32_t C,
                   uint32_t total, uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
    constexpr int kRows = quant_rows(DT);
    sm100::pdl_wait();
    sm100::pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t G = mx_groups(K);
    const uint32_t nwarps = gridDim.x * 8;
    for (uint32_t i = blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += nwarps) {
        const uint32_t q = i / C;
        const int64_t r0 = (int64_t)q * kRows, c = (int64_t)(i - q * C) * kQuantCols + lane * 16;
        const int live = c < K ? (int)(rows - r0 < kRows ? (rows > r0 ? rows - r0 : 0) : kRows) : 0;
        const uint8_t *src = X + r0 * ld_bytes + c * Raw<DT, 16>::kBytes;
        Raw<DT, 16> raw[kRows];
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            if (j < live) raw[j].template load<WIDE>(src);
            else raw[j].zero();
            src += ld_bytes;
        }
        uint8_t *dst = codes + r0 * (K / 2) + c / 2;
        uint8_t *sc = scales + mx_scale_at(r0, c >> 7, G) + ((lane >> 1) & 3);   // 16 bytes a row
        const bool write_scale = (lane & 1) == 0 && c < G * 128;
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const uint32_t E = mx_scale_byte(raw[j].amax());
            if (write_scale) sc[j * 16] = (uint8_t)E;
            if (j < live) {
                uint2 code = make_uint2(0u, 0u);
                if (E != 255u) {
                    const float inv = mx_inverse(E);
                    float f[8];
                    raw[j].get(0, f);
                    code.x = scaled_codes8(f, inv);
                    raw[j].get(1, f);
                    code.y = scaled_codes8(f, inv);
                }
                *reinterpret_cast<uint2 *>(dst) = code;
            }
            dst += K / 2;
        }
    }
}

// Row m of bf16 X to S = kMxSlices rows of an MXFP4 matrix whose sum it is
// (mq_mx4.cuh), in tiles of `tpt` rows of X: codes in row tile * bn + (m % tpt) * S + j,
// scales in row band_rows * tile + (m % tpt) * S + j.  Rows and columns between are not
// written: their products fall into columns that nothing reads.  One warp: 256
// columns of one row.  100 x 14336 in about 4 us, one chain of eight dependent
// roundings per warp.
__global__ void __launch_bounds__(256)
mx_slices_kernel(const uint8_t *__restrict__ X, int64_t K, int64_t ld_bytes, uint32_t C, uint32_t total,
                 uint32_t tpt, int bn, int band_rows, uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
    constexpr int S = kMxSlices;
    sm100::pdl_wait();                        // X may come from the previous kernel
    sm100::pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t G = mx_groups(K);
    const uint32_t nwarps = gridDim.x * 8;
    for (uint32_t i = blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += nwarps) {
        const uint32_t q = i / C, tl = q / tpt;
        const int64_t m = q, c = (int64_t)(i - q * C) * 256 + lane * 8, tile = tl;
        const int local = (int)(q - tl * tpt) * S;
        Raw<MQ_BF16, 8> raw;
        if (c < K) raw.load<false>(X + m * ld_bytes + c * 2);
        else raw.zero();
        float x[8];
        raw.get(0, x);
        const uint32_t E = mx_slice0_byte(raw.amax());
        __half2 u[4] = {};
        if (E != 255u) mx_slice_start(x, mx_inverse(E), u);
        // scale bytes: a lane writes those of block lane % 8 for slices lane / 8, + 4
        const uint32_t Eb = __shfl_sync(0xFFFFFFFFu, E, (lane & 7) * 4);
        const int64_t cb = c - lane * 8 + (lane & 7) * 32;
#pragma unroll
        for (int h = 0; h < S / 4; ++h) {
            const int j = 4 * h + (lane >> 3);
            if (cb < G * 128)
                scales[mx_scale_at(tile * band_rows + local + j, cb >> 7, G) + ((cb >> 5) & 3)] =
                    (uint8_t)mx_slice_byte(Eb, j);
        }
        if (c >= K) continue;
        uint8_t *dst = codes + (tile * bn + local) * (K / 2) + c / 2;
#pragma unroll
        for (int j = 0; j < S; ++j)
            *reinterpret_cast<uint32_t *>(dst + j * (K / 2)) =
                mx_slice_codes(u, mx_slice_byte(E, j) - mx_slice_byte(E, j + 1));
    }
}

// 32 bytes of results: one store where rows are aligned to that, else two.
template <bool WIDE>
__device__ __forceinline__ void store32(void *p, const uint32_t (&v)[8]) {
    if constexpr (WIDE) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
                     "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        static_cast<uint4 *>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        static_cast<uint4 *>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

// One warp: 512 columns of a few rows, 16 a lane.  8192 x 4096 to bf16 in 14.9 us
// (5.7 TB/s): HBM.
template <bool F32, bool WIDE>
__global__ void __launch_bounds__(256)
mx_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t rows,
                     int64_t K, uint32_t C, uint32_t total, uint8_t *__restrict__ out, int64_t ld_bytes) {
    sm100::pdl_wait();
    sm100::pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t G = mx_groups(K);
    const uint32_t nwarps = gridDim.x * 8;
    for (uint32_t i = blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += nwarps) {
        const uint32_t q = i / C;
        const int64_t r0 = (int64_t)q * kDeqRows, c = (int64_t)(i - q * C) * kQuantCols + lane * 16;
        if (c >= K) continue;
        const int live = rows - r0 < kDeqRows ? (int)(rows - r0) : kDeqRows;
        const uint8_t *src = codes + r0 * (K / 2) + c / 2;
        const uint8_t *sc = scales + mx_scale_at(r0, c >> 7, G) + ((c >> 5) & 3);
        uint8_t *dst = out + r0 * ld_bytes + c * (F32 ? 4 : 2);
        uint2 w[kDeqRows];
        uint32_t E[kDeqRows];
#pragma unroll
        for (int j = 0; j < kDeqRows; ++j) {
            w[j] = make_uint2(0u, 0u);
            E[j] = 0;
            if (j < live) {
                w[j] = *reinterpret_cast<const uint2 *>(src);
                E[j] = sc[j * 16];
            }
            src += K / 2;
        }
#pragma unroll
        for (int j = 0; j < kDeqRows; ++j) {
            if (j >= live) break;
            const uint64_t s2 = pair(mx_value(E[j]), mx_value(E[j]));
            uint32_t v[16];                                         // fp32 bits, or bf16 pairs in the first eight
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float u[8];
                mx_units8(h ? w[j].y : w[j].x, u);
#pragma unroll
                for (int e = 0; e < 4; ++e) {                       // exact (at most 2 significant bits)
                    unpair(mul2(pair(u[2 * e], u[2 * e + 1]), s2), u[2 * e], u[2 * e + 1]);
                    if constexpr (F32) {
                        v[8 * h + 2 * e] = __float_as_uint(u[2 * e]);
                        v[8 * h + 2 * e + 1] = __float_as_uint(u[2 * e + 1]);
                    } else {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(u[2 * e], u[2 * e + 1]);
                        v[4 * h + e] = *reinterpret_cast<const uint32_t *>(&b);
                    }
                }
            }
            store32<WIDE>(dst, {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]});
            if constexpr (F32) store32<WIDE>(dst + 32, {v[8], v[9], v[10], v[11], v[12], v[13], v[14], v[15]});
            dst += ld_bytes;
        }
    }
}

// s (u - z) as an fp32 number that rounds to fewer bits as the exact value
// would: cut toward zero, the last bit set when something was cut off.  The
// 64-bit product is exact (11 bits of s times at most 33 of the difference).
__device__ __forceinline__ float scaled_level_odd(double s, double u, double z) {
    const double w = s * (u - z);
    const float f = __double2float_rz(w);
    return (double)f == w ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// Zero points outside 32 <= z < 4096 (none in practice), out of line: the levels
// in 64 bits, cut with a sticky bit.  Returns the scale byte, codes in c.
template <int R>
__device__ __noinline__ uint32_t nested_block_any(const uint32_t *B, float s, float z, uint32_t *c) {
    constexpr double kHalf = R == 8 ? 0.5 : (double)(1 << (7 - R > 0 ? 7 - R : 0));
    uint32_t m = 0;
    for (int j = 0; j < 32; ++j) {
        const float v = scaled_level_odd(s, (double)((B[j & 7] >> (8 * (j >> 3))) & 0xFFu) + kHalf, z);
        m = max(m, __float_as_uint(v) & 0x7FFFFFFFu);
    }
    const uint32_t E = mx_scale_byte(m);
    const float f = E == 255u ? 0.f : mx_inverse(E);
#pragma unroll 1
    for (int b = 0; b < 4; ++b) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = scaled_level_odd(s, (double)((B[e] >> (8 * b)) & 0xFFu) + kHalf, z);
        c[b] = E == 255u ? 0u : scaled_codes8(v, f);
    }
    return E;
}

// The block (32 columns of a row, one word of each plane) as MXFP4: returns the
// scale byte, codes in c.
template <int R, bool ASYM>
__device__ __forceinline__ uint32_t nested_block(const uint32_t (&P)[8], float s, float z, uint32_t (&c)[4]) {
    constexpr float kHalf = R == 8 ? 0.5f : (float)(1 << (7 - R > 0 ? 7 - R : 0));   // 2^(7-r)
    uint32_t B[8];
    byte_words<R>(P, B);                                             // byte b of B[e]: column 8 b + e
    if constexpr (ASYM) {
        if (!(z >= 32.f && z < 4096.f)) {
            uint32_t Bm[8], cm[4];
#pragma unroll
            for (int e = 0; e < 8; ++e) Bm[e] = B[e];
            const uint32_t E = nested_block_any<R>(Bm, s, z, cm);
#pragma unroll
            for (int b = 0; b < 4; ++b) c[b] = cm[b];
            return E;
        }
    }
    // The level minus z has at most 13 significant bits here, so its product
    // with the 11 bits of s is exact in fp32, and so is every step: a byte is
    // set into 2^15 + byte by one permute, the rest is one addition and, once
    // the block's largest level is known, one multiplication by s times the
    // power of two.
    float v[4][8], m = 0.f;
    const uint64_t off = pair(kHalf - z - 32768.f, kHalf - z - 32768.f);
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const uint32_t sel = 0x7604u | ((uint32_t)b << 4);
            const uint64_t t = add2(pair(__uint_as_float(prmt(B[e], 0x47000000u, sel)),
                                         __uint_as_float(prmt(B[e + 1], 0x47000000u, sel))), off);
            unpair(t, v[b][e], v[b][e + 1]);
            m = fmaxf(m, fmaxf(fabsf(v[b][e]), fabsf(v[b][e + 1])));
        }
    // s may carry a sign (-0.0, or a negative scale of a caller's own view): it
    // belongs to the elements alone
    const float a = fabsf(s) * m;
    const uint32_t E = mx_scale_byte(__float_as_uint(a));
    const float f = a > 0.f ? s * mx_inverse(E) : s;                 // all zeros: keep their signs
#pragma unroll
    for (int b = 0; b < 4; ++b) c[b] = E == 255u ? 0u : scaled_codes8(v[b], f);
    return E;
}

// One thread: four words of each plane (rows 32 apart), each one block of MXFP4;
// four adjacent lanes hold a row's 128 columns, so a warp reads 128 contiguous
// bytes of each plane and writes whole 64-byte runs.  128 threads take one 128 x 128
// block, so that what locates it is worked out once for 128 elements a thread.
// 14336 x 4096 at r = 4 in 16.5 us, with zero points 17.5 (3.7 TB/s): about 245
// instructions for 32 weights, half of them on the half-rate integer pipe, keep 57
// to 70 % of the issue slots busy; HBM would take 9.4 us.
template <int R, bool ASYM>
__global__ void __launch_bounds__(128, R <= 4 ? 7 : 5)
mx_from_nested_kernel(const uint32_t *__restrict__ planes, const uint16_t *__restrict__ s16,
                      const uint16_t *__restrict__ z16, int64_t N, int64_t K, uint32_t G, uint32_t blocks,
                      uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
    sm100::pdl_wait();
    sm100::pdl_launch_dependents();
    constexpr int kWords = 4;
    const int64_t plane_words = (int64_t)blocks * 512;
    const int w = threadIdx.x & 3, n0 = (int)(threadIdx.x >> 2);     // word and first row of this thread
    for (uint32_t block = blockIdx.x; block < blocks; block += gridDim.x) {
        const uint32_t t = block / G, g = block - t * G;
        const uint32_t *src = planes + (int64_t)block * 512 + threadIdx.x;
        uint32_t P[kWords][8];
        float s[kWords], z[kWords];
#pragma unroll
        for (int h = 0; h < kWords; ++h) {
#pragma unroll
            for (int p = 0; p < 8; ++p) P[h][p] = p < R ? __ldcs(src + p * plane_words + h * 128) : 0u;
            s[h] = __half2float(__ushort_as_half(s16[(int64_t)block * 128 + h * 32 + n0]));
            z[h] = ASYM ? __half2float(__ushort_as_half(z16[(int64_t)block * 128 + h * 32 + n0])) : 128.f;
        }
        const int64_t row = (int64_t)t * 128 + n0;
        uint8_t *dst = codes + row * (K / 2) + g * 64 + w * 16, *sc = scales + mx_scale_at(row, g, G) + w;
        const int left = N - row > 128 ? 128 : (int)(N - row);       // rows from this thread's first on
#pragma unroll
        for (int h = 0; h < kWords; ++h) {
            uint32_t c[4];
            const uint32_t E = nested_block<R, ASYM>(P[h], s[h], z[h], c);
            sc[h * 4] = (uint8_t)(h * 32 < left ? E : 0u);           // rows 32 on: the next four bytes
            if (h * 32 < left) *reinterpret_cast<uint4 *>(dst + h * 32 * (K / 2)) = make_uint4(c[0], c[1], c[2], c[3]);
        }
    }
}

// Warp-sized steps of a converter (some columns of some rows; numbered in 32 bits,
// 2^31 or more are refused) and blocks of eight warps for them.
struct Steps {
    uint32_t C, total;
    int grid;
};
bool steps_for(int64_t row_steps, int64_t K, int cols, Steps *s) {
    const int64_t C = (K + cols - 1) / cols;
    if (row_steps > (int64_t)UINT32_MAX / 2 / C) return false;
    s->C = (uint32_t)C;
    s->total = (uint32_t)(row_steps * C);
    s->grid = (int)((s->total + 7) / 8 < 148 * 32 ? (s->total + 7) / 8 : 148 * 32);
    return true;
}

// Blocks of `threads`, allowed to start before the previous kernel has ended
// (every kernel here waits for it before it reads or writes anything).
template <class... P, class... A>
cudaError_t launch_pdl(void (*fn)(P...), int grid, int threads, cudaStream_t st, A... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, static_cast<P>(args)...);
}

bool mx_sizes(int64_t rows, int64_t K) {
    return rows >= 0 && rows <= kMxMaxDim && K >= kMxBlock && K % kMxBlock == 0 && K <= kMxMaxDim;
}

}  // namespace

mq_status check_mx4(const mq_mx4 *m, const char *what) {
    if (!m) return failf(MQ_ERR_INVALID_ARG, "%s: the MXFP4 matrix is NULL", what);
    if (!mx_sizes(m->rows, m->K))
        return failf(MQ_ERR_INVALID_ARG, "%s: need rows >= 0 and K a positive multiple of 32", what);
    if (m->rows > 0 && (!m->codes || !m->scales))
        return failf(MQ_ERR_INVALID_ARG, "%s: the MXFP4 matrix has a NULL buffer", what);
    if (!aligned16(m->codes) || !aligned16(m->scales))
        return failf(MQ_ERR_MISALIGNED, "%s: codes and scales must be 16-byte aligned", what);
    return MQ_OK;
}

mq_status launch_mx_slices(const uint16_t *X, int64_t M, int64_t K, int64_t ldx, const MxSlicing &sl,
                           uint8_t *codes, uint8_t *scales, cudaStream_t st) {
    Steps n;
    if (!steps_for(M, K, 256, &n)) return fail(MQ_ERR_UNSUPPORTED, "mq_mx4_gemm_bf16: X is too large");
    const cudaError_t e =
        launch_pdl(mx_slices_kernel, n.grid, 256, st, reinterpret_cast<const uint8_t *>(X), K, ldx * 2, n.C, n.total,
                   sl.tpt, sl.bn, sl.Tb ? 256 : 128, codes, scales);
    return e == cudaSuccess ? MQ_OK : cuda_fail(e, "mx_slices_kernel");
}

}  // namespace mq

using namespace mq;

extern "C" size_t mq_mx4_code_bytes(int64_t rows, int64_t K) {
    return mx_sizes(rows, K) ? (size_t)rows * (size_t)(K / 2) : 0;
}

extern "C" size_t mq_mx4_scale_bytes(int64_t rows, int64_t K) {
    return mx_sizes(rows, K) ? (size_t)((rows + 127) / 128) * (size_t)mx_groups(K) * 512 : 0;
}

extern "C" mq_status mq_mx4_quantize(const void *X, int dtype, int64_t rows, int64_t K, int64_t ld,
                                     uint8_t *codes_out, uint8_t *scales_out, void *stream) {
    if (dtype != MQ_BF16 && dtype != MQ_F16 && dtype != MQ_F32)
        return fail(MQ_ERR_INVALID_ARG, "mq_mx4_quantize: unknown dtype");
    const int64_t size = dtype == MQ_F32 ? 4 : 2;
    if (!mx_sizes(rows, K))
        return fail(MQ_ERR_INVALID_ARG, "mq_mx4_quantize: need rows >= 0 and K a positive multiple of 32");
    if (ld < K || ld > INT64_MAX / 8) return fail(MQ_ERR_INVALID_ARG, "mq_mx4_quantize: need ld >= K");
    if (rows == 0) return MQ_OK;
    if (!X || !codes_out || !scales_out)
        return fail(MQ_ERR_INVALID_ARG, "NULL pointer passed to mq_mx4_quantize");
    if (!aligned16(X) || !aligned16(codes_out) || !aligned16(scales_out) || (rows > 1 && ld * size % 16))
        return fail(MQ_ERR_MISALIGNED, "mq_mx4_quantize: pointers and the row stride must be 16-byte aligned");
    cudaStream_t st = (cudaStream_t)stream;
    const mq_status bs = bind_device(st);
    if (bs != MQ_OK) return bs;
    Steps n;
    if (!steps_for((rows + 127) / 128 * (128 / quant_rows(dtype)), K, kQuantCols, &n))
        return fail(MQ_ERR_UNSUPPORTED, "mq_mx4_quantize: the matrix is too large");
    const uint8_t *x = static_cast<const uint8_t *>(X);
    // 32-byte loads where every row starts on 32 bytes
    const bool wide = (reinterpret_cast<uintptr_t>(X) | (uintptr_t)(rows > 1 ? ld * size : 0)) % 32 == 0;
    const auto fn = dtype == MQ_BF16  ? wide ? mx_quantize_kernel<MQ_BF16, true> : mx_quantize_kernel<MQ_BF16, false>
                    : dtype == MQ_F16 ? wide ? mx_quantize_kernel<MQ_F16, true> : mx_quantize_kernel<MQ_F16, false>
                    : wide            ? mx_quantize_kernel<MQ_F32, true>
                                      : mx_quantize_kernel<MQ_F32, false>;
    const cudaError_t e = launch_pdl(fn, n.grid, 256, st, x, rows, K, ld * size, n.C, n.total, codes_out, scales_out);
    return e == cudaSuccess ? MQ_OK : cuda_fail(e, "mx_quantize_kernel");
}

extern "C" mq_status mq_mx4_from_nested(const mq_weights *w, uint8_t *codes_out, uint8_t *scales_out,
                                        void *stream) {
    if (!w) return fail(MQ_ERR_INVALID_ARG, "weights view is NULL");
    mq_status s = check_weights(w, w->N, w->K);
    if (s != MQ_OK) return s;
    if (!mx_sizes(w->N, w->K)) return fail(MQ_ERR_INVALID_ARG, "mq_mx4_from_nested: N or K too large");
    if (!codes_out || !scales_out) return fail(MQ_ERR_INVALID_ARG, "NULL pointer passed to mq_mx4_from_nested");
    if (!aligned16(codes_out) || !aligned16(scales_out))
        return fail(MQ_ERR_MISALIGNED, "mq_mx4_from_nested: the outputs must be 16-byte aligned");
    cudaStream_t st = (cudaStream_t)stream;
    if ((s = bind_device(st)) != MQ_OK) return s;
    using Fn = void (*)(const uint32_t *, const uint16_t *, const uint16_t *, int64_t, int64_t, uint32_t, uint32_t,
                        uint8_t *, uint8_t *);
    static const Fn fns[2][8] = {
        {mx_from_nested_kernel<1, false>, mx_from_nested_kernel<2, false>, mx_from_nested_kernel<3, false>,
         mx_from_nested_kernel<4, false>, mx_from_nested_kernel<5, false>, mx_from_nested_kernel<6, false>,
         mx_from_nested_kernel<7, false>, mx_from_nested_kernel<8, false>},
        {mx_from_nested_kernel<1, true>, mx_from_nested_kernel<2, true>, mx_from_nested_kernel<3, true>,
         mx_from_nested_kernel<4, true>, mx_from_nested_kernel<5, true>, mx_from_nested_kernel<6, true>,
         mx_from_nested_kernel<7, true>, mx_from_nested_kernel<8, true>}};
    const int64_t blocks = (w->N + 127) / 128 * (w->K / kGroup);
    if (blocks > (int64_t)UINT32_MAX / 2) return fail(MQ_ERR_UNSUPPORTED, "mq_mx4_from_nested: the matrix is too large");
    const int grid = (int)(blocks < 148 * 32 ? blocks : 148 * 32);
    const cudaError_t e = launch_pdl(fns[w->zeros != nullptr][w->r - 1], grid, 128, st, w->planes, w->scales, w->zeros, w->N, w->K,
                                     w->K / kGroup, blocks, codes_out, scales_out);
    return e == cudaSuccess ? MQ_OK : cuda_fail(e, "mx_from_nested_kernel");
}

extern "C" mq_status mq_mx4_dequantize(const mq_mx4 *m, void *out, int dtype, int64_t ld, void *stream) {
    mq_status s = check_mx4(m, "mq_mx4_dequantize");
    if (s != MQ_OK) return s;
    if (dtype != MQ_BF16 && dtype != MQ_F32)
        return fail(MQ_ERR_INVALID_ARG, "mq_mx4_dequantize: dtype must be MQ_BF16 or MQ_F32");
    const int64_t size = dtype == MQ_F32 ? 4 : 2;
    if (ld < m->K || ld > INT64_MAX / 8) return fail(MQ_ERR_INVALID_ARG, "mq_mx4_dequantize: need ld >= K");
    if (m->rows == 0) return MQ_OK;
    if (!out) return fail(MQ_ERR_INVALID_ARG, "mq_mx4_dequantize: out is NULL");
    if (!aligned16(out) || (m->rows > 1 && ld * size % 16))
        return fail(MQ_ERR_MISALIGNED, "mq_mx4_dequantize: out and its row stride must be 16-byte aligned");
    cudaStream_t st = (cudaStream_t)stream;
    if ((s = bind_device(st)) != MQ_OK) return s;
    Steps n;
    if (!steps_for((m->rows + kDeqRows - 1) / kDeqRows, m->K, kQuantCols, &n))
        return fail(MQ_ERR_UNSUPPORTED, "mq_mx4_dequantize: the matrix is too large");
    uint8_t *o = static_cast<uint8_t *>(out);
    const bool wide = (reinterpret_cast<uintptr_t>(out) | (uintptr_t)(m->rows > 1 ? ld * size : 0)) % 32 == 0;
    const auto fn = dtype == MQ_F32 ? wide ? mx_dequantize_kernel<true, true> : mx_dequantize_kernel<true, false>
                    : wide          ? mx_dequantize_kernel<false, true>
                                    : mx_dequantize_kernel<false, false>;
    const cudaError_t e = launch_pdl(fn, n.grid, 256, st, m->codes, m->scales, m->rows, m->K, n.C, n.total, o, ld * size);
    return e == cudaSuccess ? MQ_OK : cuda_fail(e, "mx_dequantize_kernel");
}
