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

// Eight consecutive elements as loaded: one or two 16-byte words.  amax is the
// largest magnitude of the block of 32 in this and the three adjacent lanes, as
// fp32 bits; magnitudes are compared as integers, so that a NaN wins.
template <int DT>
struct Raw8 {
    uint4 v;
    static constexpr int kBytes = 2;
    __device__ void load(const void *p) { v = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
    __device__ uint32_t amax() const {
        constexpr uint32_t kMag = 0x7FFF7FFFu;
        uint32_t m = __vmaxu2(__vmaxu2(v.x & kMag, v.y & kMag), __vmaxu2(v.z & kMag, v.w & kMag));
        m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        m = max(m & 0xFFFFu, m >> 16);
        if constexpr (DT == MQ_BF16) return m << 16;
        return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m))) & 0x7FFFFFFFu;
    }
    __device__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == MQ_BF16) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            } else {
                const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                f[2 * i] = t.x;
                f[2 * i + 1] = t.y;
            }
        }
    }
};
template <>
struct Raw8<MQ_F32> {
    uint4 a, b;
    static constexpr int kBytes = 4;
    __device__ void load(const void *p) {
        a = __ldcs(reinterpret_cast<const uint4 *>(p));
        b = __ldcs(reinterpret_cast<const uint4 *>(p) + 1);
    }
    __device__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
    __device__ uint32_t amax() const {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        return max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    }
    __device__ void get(float (&f)[8]) const {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    }
};

// Rows per warp and step: so many 16-byte loads of a thread are in flight.
__host__ __device__ constexpr int quant_rows(int dtype) { return dtype == MQ_F32 ? 4 : 8; }
constexpr int kDeqRows = 8;

// One warp: 256 columns of a few rows (all in one 128-row band).  Steps beyond
// the matrix (the padding rows and columns of the scale blocks) write zero scale
// bytes only.
template <int DT>
__global__ void __launch_bounds__(256)
mx_quantize_kernel(const uint8_t *__restrict__ X, int64_t rows, int64_t K, int64_t ld_bytes,
                   uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
    constexpr int kRows = quant_rows(DT);
    sm100::pdl_wait();
    sm100::pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t G = mx_groups(K), C = (K + 255) / 256, steps = (rows + 127) / 128 * (128 / kRows);
    const int64_t total = steps * C, nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    for (int64_t i = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5; i < total; i += nwarps) {
        const int64_t r0 = i / C * kRows, c = (i % C) * 256 + lane * 8;
        const int live = c < K ? (int)(rows - r0 < kRows ? (rows > r0 ? rows - r0 : 0) : kRows) : 0;
        const uint8_t *src = X + r0 * ld_bytes + c * Raw8<DT>::kBytes;
        Raw8<DT> raw[kRows];
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            if (j < live) raw[j].load(src + j * ld_bytes);
            else raw[j].zero();
        }
        uint8_t *dst = codes + r0 * (K / 2) + c / 2;
        uint8_t *sc = scales + mx_scale_at(r0, c >> 7, G) + ((lane >> 2) & 3);   // 16 bytes a row
        const bool write_scale = (lane & 3) == 0 && c < G * 128;
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const uint32_t E = mx_scale_byte(raw[j].amax());
            if (write_scale) sc[j * 16] = (uint8_t)E;
            if (j < live) {
                float f[8];
                raw[j].get(f);
                *reinterpret_cast<uint32_t *>(dst + j * (K / 2)) = E == 255u ? 0u : scaled_codes8(f, mx_inverse(E));
            }
        }
    }
}

// Row m of bf16 X to S rows of an MXFP4 matrix whose sum it is (mq_mx4.cuh), in
// tiles of `tpt` rows of X: codes in row tile * bn + (m % tpt) * S + j, scales in
// row band_rows * tile + (m % tpt) * S + j.  Rows and columns between are not
// written: their products fall into columns that nothing reads.  One warp: 256
// columns of one row.
template <int S>
__global__ void __launch_bounds__(256)
mx_slices_kernel(const uint8_t *__restrict__ X, int64_t M, int64_t K, int64_t ld_bytes, int tpt, int bn,
                 int band_rows, uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
    sm100::pdl_wait();                        // X may come from the previous kernel
    sm100::pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t G = mx_groups(K), C = (K + 255) / 256;
    const int64_t total = M * C, nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    for (int64_t i = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5; i < total; i += nwarps) {
        const int64_t m = i / C, c = (i % C) * 256 + lane * 8, tile = m / tpt;
        const int local = (int)(m - tile * tpt) * S;
        Raw8<MQ_BF16> raw;
        if (c < K) raw.load(X + m * ld_bytes + c * 2);
        else raw.zero();
        float u[8];
        raw.get(u);
        uint32_t E = mx_slice0_byte(raw.amax());
        const bool bad = E == 255u;
        const float inv = bad ? 0.f : mx_inverse(E);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = bad ? 0.f : u[e] * inv;
        uint8_t *dst = codes + (tile * bn + local) * (K / 2) + c / 2;
#pragma unroll
        for (int j = 0; j < S; ++j) {
            if ((lane & 3) == 0 && c < G * 128)
                scales[mx_scale_at(tile * band_rows + local + j, c >> 7, G) + ((lane >> 2) & 3)] = (uint8_t)E;
            const uint32_t En = mx_next_slice(E, j);
            const uint32_t code = mx_slice_codes(u, E - En);
            if (c < K) *reinterpret_cast<uint32_t *>(dst + j * (K / 2)) = code;
            E = En;
        }
    }
}

// One warp: 256 columns of a few rows.
template <bool F32>
__global__ void __launch_bounds__(256)
mx_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t rows,
                     int64_t K, uint8_t *__restrict__ out, int64_t ld_bytes) {
    sm100::pdl_wait();
    sm100::pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t G = mx_groups(K), C = (K + 255) / 256, steps = (rows + kDeqRows - 1) / kDeqRows;
    const int64_t total = steps * C, nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    for (int64_t i = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5; i < total; i += nwarps) {
        const int64_t r0 = i / C * kDeqRows, c = (i % C) * 256 + lane * 8;
        if (c >= K) continue;
        const int live = rows - r0 < kDeqRows ? (int)(rows - r0) : kDeqRows;
        const uint8_t *src = codes + r0 * (K / 2) + c / 2;
        const uint8_t *sc = scales + mx_scale_at(r0, c >> 7, G) + ((c >> 5) & 3);
        uint8_t *dst = out + r0 * ld_bytes + c * (F32 ? 4 : 2);
        uint32_t w[kDeqRows], E[kDeqRows];
#pragma unroll
        for (int j = 0; j < kDeqRows; ++j) {
            w[j] = E[j] = 0;
            if (j < live) {
                w[j] = __ldcs(reinterpret_cast<const uint32_t *>(src + j * (K / 2)));
                E[j] = sc[j * 16];
            }
        }
#pragma unroll
        for (int j = 0; j < kDeqRows; ++j) {
            if (j >= live) break;
            float u[8];
            mx_units8(w[j], u);
            const uint64_t s2 = pair(mx_value(E[j]), mx_value(E[j]));
#pragma unroll
            for (int e = 0; e < 4; ++e)                             // exact (at most 2 significant bits)
                unpair(mul2(pair(u[2 * e], u[2 * e + 1]), s2), u[2 * e], u[2 * e + 1]);
            if constexpr (F32) {
                float4 *q = reinterpret_cast<float4 *>(dst + j * ld_bytes);
                q[0] = make_float4(u[0], u[1], u[2], u[3]);
                q[1] = make_float4(u[4], u[5], u[6], u[7]);
            } else {
                uint32_t h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(u[2 * e], u[2 * e + 1]);
                    h[e] = *reinterpret_cast<const uint32_t *>(&b);
                }
                *reinterpret_cast<uint4 *>(dst + j * ld_bytes) = make_uint4(h[0], h[1], h[2], h[3]);
            }
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

// The block (32 columns of a row, one word of each plane) as MXFP4: returns the
// scale byte, codes in c.
template <int R>
__device__ __forceinline__ uint32_t nested_block(const uint32_t (&P)[8], float s, float z, uint32_t (&c)[4]) {
    constexpr float kHalf = R == 8 ? 0.5f : (float)(1 << (7 - R > 0 ? 7 - R : 0));   // 2^(7-r)
    uint32_t B[8];
    byte_words<R>(P, B);                                             // byte b of B[e]: column 8 b + e
    float v[4][8];
    uint32_t E;
    float f;
    if (z >= 32.f && z < 4096.f) {
        // The level minus z has at most 13 significant bits here, so its product
        // with the 11 bits of s is exact in fp32, and so is every step: a byte
        // is set into 2^15 + byte by one permute, the rest is one addition and,
        // once the block's largest level is known, one multiplication by s
        // times the power of two.
        const uint64_t off = pair(kHalf - z - 32768.f, kHalf - z - 32768.f);
        float m = 0.f;
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
        const float a = s * m;
        E = mx_scale_byte(__float_as_uint(a));
        f = a > 0.f ? s * mx_inverse(E) : s;                         // all zeros: keep their signs
    } else {
        // other zero points (none in practice): 64 bits, cut with a sticky bit
        uint32_t m = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[b][e] = scaled_level_odd(s, (double)((B[e] >> (8 * b)) & 0xFFu) + (double)kHalf, z);
                m = max(m, __float_as_uint(v[b][e]) & 0x7FFFFFFFu);
            }
        E = mx_scale_byte(m);
        f = E == 255u ? 0.f : mx_inverse(E);
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) c[b] = E == 255u ? 0u : scaled_codes8(v[b], f);
    return E;
}

// One thread: one word of each plane, which is one block of MXFP4; four adjacent
// lanes hold a row's 128 columns, so a warp reads 128 contiguous bytes of each
// plane and writes whole 64-byte runs.  A block of threads takes whole 128 x 128
// blocks, so nothing is divided per thread.
template <int R>
__global__ void __launch_bounds__(256)
mx_from_nested_kernel(const uint32_t *__restrict__ planes, const uint16_t *__restrict__ s16,
                      const uint16_t *__restrict__ z16, int64_t N, int64_t K,
                      uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
    sm100::pdl_wait();
    sm100::pdl_launch_dependents();
    const int64_t G = K / kGroup, blocks = (N + 127) / 128 * G, plane_words = blocks * 512;
    const int w = threadIdx.x & 3, n0 = (int)(threadIdx.x >> 2);     // word and first row of this thread
    for (int64_t block = blockIdx.x; block < blocks; block += gridDim.x) {
        const int64_t t = block / G, g = block - t * G;
        uint32_t P[2][8];
        float s[2], z[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int p = 0; p < 8; ++p)
                P[h][p] = p < R ? __ldcs(planes + p * plane_words + block * 512 + h * 256 + threadIdx.x) : 0u;
            s[h] = __half2float(__ushort_as_half(s16[block * 128 + h * 64 + n0]));
            z[h] = z16 ? __half2float(__ushort_as_half(z16[block * 128 + h * 64 + n0])) : 128.f;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t row = t * 128 + h * 64 + n0;
            uint32_t c[4];
            const uint32_t E = nested_block<R>(P[h], s[h], z[h], c);
            scales[mx_scale_at(row, g, G) + w] = (uint8_t)(row < N ? E : 0u);
            if (row < N)
                *reinterpret_cast<uint4 *>(codes + row * (K / 2) + g * 64 + w * 16) = make_uint4(c[0], c[1], c[2], c[3]);
        }
    }
}

int grid_for(int64_t work, int per_block) {
    int64_t g = (work + per_block - 1) / per_block;
    if (g > 148 * 32) g = 148 * 32;
    return (int)(g < 1 ? 1 : g);
}

// 256 threads a block, allowed to start before the previous kernel has ended
// (every kernel here waits for it before it reads or writes anything).
template <class... P, class... A>
cudaError_t launch_pdl(void (*fn)(P...), int grid, cudaStream_t st, A... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(256);
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
    const cudaError_t e =
        launch_pdl(sl.S == 6 ? mx_slices_kernel<6> : mx_slices_kernel<8>, grid_for(M * ((K + 255) / 256) * 32, 256), st,
                   reinterpret_cast<const uint8_t *>(X), M, K, ldx * 2, sl.tpt, sl.bn, sl.Tb ? 256 : 128, codes, scales);
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
    const int grid = grid_for((rows + 127) / 128 * (128 / quant_rows(dtype)) * ((K + 255) / 256) * 32, 256);
    const uint8_t *x = static_cast<const uint8_t *>(X);
    const auto fn = dtype == MQ_BF16  ? mx_quantize_kernel<MQ_BF16>
                    : dtype == MQ_F16 ? mx_quantize_kernel<MQ_F16>
                                      : mx_quantize_kernel<MQ_F32>;
    const cudaError_t e = launch_pdl(fn, grid, st, x, rows, K, ld * size, codes_out, scales_out);
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
    using Fn = void (*)(const uint32_t *, const uint16_t *, const uint16_t *, int64_t, int64_t, uint8_t *, uint8_t *);
    static const Fn fns[8] = {mx_from_nested_kernel<1>, mx_from_nested_kernel<2>, mx_from_nested_kernel<3>,
                              mx_from_nested_kernel<4>, mx_from_nested_kernel<5>, mx_from_nested_kernel<6>,
                              mx_from_nested_kernel<7>, mx_from_nested_kernel<8>};
    const int grid = grid_for((w->N + 127) / 128 * (w->K / kGroup), 1);
    const cudaError_t e = launch_pdl(fns[w->r - 1], grid, st, w->planes, w->scales, w->zeros, w->N, w->K, codes_out, scales_out);
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
    const int grid = grid_for((m->rows + kDeqRows - 1) / kDeqRows * ((m->K + 255) / 256) * 32, 256);
    uint8_t *o = static_cast<uint8_t *>(out);
    const cudaError_t e = launch_pdl(dtype == MQ_F32 ? mx_dequantize_kernel<true> : mx_dequantize_kernel<false>, grid, st,
                                     m->codes, m->scales, m->rows, m->K, o, ld * size);
    return e == cudaSuccess ? MQ_OK : cuda_fail(e, "mx_dequantize_kernel");
}
