// MXFP4 converters (include/mq.h): dense rows and nested parents to MXFP4,
// MXFP4 to dense values, and bf16 rows to sums of MXFP4 rows.  All are bound
// by HBM (a few operations per element), so what counts is that loads and
// stores are wide and that several are in flight per thread.
#include "mq_bits.cuh"
#include "mq_mx4.cuh"
#include "mq_sm100.cuh"

namespace mq {
namespace {

// Eight consecutive elements as fp32.
template <int DT>
struct Raw8;                                  // as loaded: one or two 16-byte words
template <>
struct Raw8<MQ_BF16> {
    uint4 v;
    __device__ void load(const void *p) { v = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
    __device__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static constexpr int kBytes = 2;
};
template <>
struct Raw8<MQ_F16> {
    uint4 v;
    __device__ void load(const void *p) { v = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
    __device__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        }
    }
    static constexpr int kBytes = 2;
};
template <>
struct Raw8<MQ_F32> {
    uint4 a, b;
    __device__ void load(const void *p) {
        a = __ldcs(reinterpret_cast<const uint4 *>(p));
        b = __ldcs(reinterpret_cast<const uint4 *>(p) + 1);
    }
    __device__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
    __device__ void get(float (&f)[8]) const {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    }
    static constexpr int kBytes = 4;
};

// Largest magnitude (as bits, so that a NaN wins) of a block of 32: eight
// numbers in each of four adjacent lanes.
__device__ __forceinline__ uint32_t block_amax(const float (&f)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    return max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
}

// The four scale bytes of 128 columns (16 lanes), gathered in each lane.
__device__ __forceinline__ uint32_t gather_scales(uint32_t E, int lane) {
    uint32_t w = E << (8 * ((lane >> 2) & 3));
    w |= __shfl_xor_sync(0xFFFFFFFFu, w, 4);
    return w | __shfl_xor_sync(0xFFFFFFFFu, w, 8);
}

constexpr int kQRows = 4;                     // rows per warp and step (loads in flight)

// One warp: 256 columns of four rows.  Steps beyond the matrix (the padding
// rows and columns of the scale blocks) write zero scale bytes only.
template <int DT>
__global__ void __launch_bounds__(256)
mx_quantize_kernel(const uint8_t *__restrict__ X, int64_t rows, int64_t K, int64_t ld_bytes,
                   uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
    const int lane = threadIdx.x & 31;
    const int64_t G = mx_groups(K), C = (K + 255) / 256, quads = (rows + 127) / 128 * (128 / kQRows);
    const int64_t total = quads * C, nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    for (int64_t i = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5; i < total; i += nwarps) {
        const int64_t r0 = i / C * kQRows, c = (i % C) * 256 + lane * 8;
        Raw8<DT> raw[kQRows];
#pragma unroll
        for (int j = 0; j < kQRows; ++j) {
            if (r0 + j < rows && c < K) raw[j].load(X + (r0 + j) * ld_bytes + c * Raw8<DT>::kBytes);
            else raw[j].zero();
        }
#pragma unroll
        for (int j = 0; j < kQRows; ++j) {
            const int64_t row = r0 + j;
            float f[8];
            raw[j].get(f);
            const uint32_t E = mx_scale_byte(block_amax(f));
            const uint32_t sw = gather_scales(E, lane);
            if ((lane & 15) == 0 && c < G * 128)
                *reinterpret_cast<uint32_t *>(scales + mx_scale_at(row, c >> 7, G)) = sw;
            if (row < rows && c < K) {
                uint32_t code = 0;
                if (E != 255u) {
                    const float inv = mx_inverse(E);
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] *= inv;
                    code = mx_codes8(f);
                }
                *reinterpret_cast<uint32_t *>(codes + row * (K / 2) + c / 2) = code;
            }
        }
    }
}

// Row m of bf16 X to the rows 8 m .. 8 m + 7 of an MXFP4 matrix whose sum it
// is (mq_mx4.cuh).  One warp: 256 columns of one row.
__global__ void __launch_bounds__(256)
mx_slices_kernel(const uint8_t *__restrict__ X, int64_t M, int64_t K, int64_t ld_bytes,
                 uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
    sm100::pdl_wait();                        // X may come from the previous kernel
    const int lane = threadIdx.x & 31;
    const int64_t G = mx_groups(K), C = (K + 255) / 256, Mp = (M + 15) / 16 * 16;
    const int64_t total = Mp * C, nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    for (int64_t i = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5; i < total; i += nwarps) {
        const int64_t m = i / C, c = (i % C) * 256 + lane * 8;
        Raw8<MQ_BF16> raw;
        if (m < M && c < K) raw.load(X + m * ld_bytes + c * 2);
        else raw.zero();
        float u[8];
        raw.get(u);
        uint32_t E = mx_slice0_byte(block_amax(u));
        const bool bad = E == 255u;
        const float inv = bad ? 0.f : mx_inverse(E);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = bad ? 0.f : u[e] * inv;
#pragma unroll
        for (int j = 0; j < kMxSlices; ++j) {
            const int64_t row = m * kMxSlices + j;
            const uint32_t sw = gather_scales(E, lane);
            if ((lane & 15) == 0 && c < G * 128)
                *reinterpret_cast<uint32_t *>(scales + mx_scale_at(row, c >> 7, G)) = sw;
            const uint32_t En = mx_next_slice(E, j);
            const uint32_t code = mx_slice_codes(u, E - En);
            if (m < M && c < K) *reinterpret_cast<uint32_t *>(codes + row * (K / 2) + c / 2) = code;
            E = En;
        }
    }
}

// One warp: 256 columns of four rows.
template <bool F32>
__global__ void __launch_bounds__(256)
mx_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t rows,
                     int64_t K, uint8_t *__restrict__ out, int64_t ld_bytes) {
    const int lane = threadIdx.x & 31;
    const int64_t G = mx_groups(K), C = (K + 255) / 256, quads = (rows + kQRows - 1) / kQRows;
    const int64_t total = quads * C, nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    for (int64_t i = (blockIdx.x * (int64_t)blockDim.x + threadIdx.x) >> 5; i < total; i += nwarps) {
        const int64_t r0 = i / C * kQRows, c = (i % C) * 256 + lane * 8;
        if (c >= K) continue;
        uint32_t w[kQRows], E[kQRows];
#pragma unroll
        for (int j = 0; j < kQRows; ++j) {
            w[j] = E[j] = 0;
            if (r0 + j < rows) {
                w[j] = __ldcs(reinterpret_cast<const uint32_t *>(codes + (r0 + j) * (K / 2) + c / 2));
                E[j] = scales[mx_scale_at(r0 + j, c >> 7, G) + ((c >> 5) & 3)];
            }
        }
#pragma unroll
        for (int j = 0; j < kQRows; ++j) {
            if (r0 + j >= rows) break;
            float u[8];
            mx_units8(w[j], u);
            const float s = mx_value(E[j]);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] *= s;              // exact (at most 2 significant bits)
            uint8_t *p = out + (r0 + j) * ld_bytes;
            if constexpr (F32) {
                float4 *q = reinterpret_cast<float4 *>(p + c * 4);
                q[0] = make_float4(u[0], u[1], u[2], u[3]);
                q[1] = make_float4(u[4], u[5], u[6], u[7]);
            } else {
                uint32_t h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(u[2 * e], u[2 * e + 1]);
                    h[e] = *reinterpret_cast<const uint32_t *>(&b);
                }
                *reinterpret_cast<uint4 *>(p + c * 2) = make_uint4(h[0], h[1], h[2], h[3]);
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

// One thread: 32 columns of a row (one word of each plane), which are one
// block of MXFP4; four adjacent lanes hold a row's 128 columns, so a warp
// reads 128 contiguous bytes of each plane and writes whole 64-byte runs.
template <int R>
__global__ void __launch_bounds__(256)
mx_from_nested_kernel(const uint32_t *__restrict__ planes, const uint16_t *__restrict__ s16,
                      const uint16_t *__restrict__ z16, int64_t N, int64_t K,
                      uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
    const int64_t G = K / kGroup, N128 = (N + 127) / 128 * 128;
    const int64_t plane_words = N128 * (K / 32);
    const int lane = threadIdx.x & 31;
    constexpr float kHalf = R == 8 ? 0.5f : (float)(1 << (7 - R > 0 ? 7 - R : 0));   // 2^(7-r)
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < plane_words;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t block = i >> 9;                            // (row tile, group)
        const int w = (int)(i & 3), n = (int)(i >> 2) & 127;     // word and row of the block
        const int64_t t = block / G, g = block - t * G, row = t * 128 + n;
        uint32_t P[8], B[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) P[p] = p < R ? __ldcs(planes + p * plane_words + i) : 0u;
        const float s = __half2float(__ushort_as_half(s16[block * 128 + n]));
        const float z = z16 ? __half2float(__ushort_as_half(z16[block * 128 + n])) : 128.f;
        byte_words<R>(P, B);                                     // byte b of B[e]: column 8 b + e
        float v[4][8];
        // For 32 <= z < 4096 the level minus z has at most 13 significant
        // bits, so its product with the 11 bits of s is exact in fp32; other
        // zero points (none in practice) take the 64-bit form.
        if (z >= 32.f && z < 4096.f) {
            const float off = kHalf - z;
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[b][e] = s * ((float)((B[e] >> (8 * b)) & 0xFFu) + off);
        } else {
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[b][e] = scaled_level_odd(s, (double)((B[e] >> (8 * b)) & 0xFFu) + (double)kHalf, z);
        }
        uint32_t m = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[b][e]) & 0x7FFFFFFFu);
        const uint32_t E = row < N ? mx_scale_byte(m) : 0u;
        uint32_t sw = E << (8 * w);
        sw |= __shfl_xor_sync(0xFFFFFFFFu, sw, 1);
        sw |= __shfl_xor_sync(0xFFFFFFFFu, sw, 2);
        if ((lane & 3) == 0) *reinterpret_cast<uint32_t *>(scales + mx_scale_at(row, g, G)) = sw;
        if (row < N) {
            uint32_t c[4] = {0, 0, 0, 0};
            if (E != 255u) {
                const float inv = mx_inverse(E);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[b][e] *= inv;
                    c[b] = mx_codes8(v[b]);
                }
            }
            *reinterpret_cast<uint4 *>(codes + row * (K / 2) + g * 64 + w * 16) = make_uint4(c[0], c[1], c[2], c[3]);
        }
    }
}

int grid_for(int64_t work, int per_block) {
    int64_t g = (work + per_block - 1) / per_block;
    if (g > 148 * 32) g = 148 * 32;
    return (int)(g < 1 ? 1 : g);
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

mq_status launch_mx_slices(const uint16_t *X, int64_t M, int64_t K, int64_t ldx, uint8_t *codes,
                           uint8_t *scales, cudaStream_t st) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid_for((M + 15) / 16 * 16 * ((K + 255) / 256) * 32, 256));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, mx_slices_kernel, reinterpret_cast<const uint8_t *>(X), M, K,
                                             ldx * 2, codes, scales);
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
    const int grid = grid_for((rows + 127) / 128 * (128 / kQRows) * ((K + 255) / 256) * 32, 256);
    const uint8_t *x = static_cast<const uint8_t *>(X);
    if (dtype == MQ_BF16)
        mx_quantize_kernel<MQ_BF16><<<grid, 256, 0, st>>>(x, rows, K, ld * size, codes_out, scales_out);
    else if (dtype == MQ_F16)
        mx_quantize_kernel<MQ_F16><<<grid, 256, 0, st>>>(x, rows, K, ld * size, codes_out, scales_out);
    else
        mx_quantize_kernel<MQ_F32><<<grid, 256, 0, st>>>(x, rows, K, ld * size, codes_out, scales_out);
    const cudaError_t e = cudaGetLastError();
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
    const int grid = grid_for((w->N + 127) / 128 * 128 * (w->K / 32), 256);
    fns[w->r - 1]<<<grid, 256, 0, st>>>(w->planes, w->scales, w->zeros, w->N, w->K, codes_out, scales_out);
    const cudaError_t e = cudaGetLastError();
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
    const int grid = grid_for((m->rows + kQRows - 1) / kQRows * ((m->K + 255) / 256) * 32, 256);
    uint8_t *o = static_cast<uint8_t *>(out);
    if (dtype == MQ_F32)
        mx_dequantize_kernel<true><<<grid, 256, 0, st>>>(m->codes, m->scales, m->rows, m->K, o, ld * size);
    else
        mx_dequantize_kernel<false><<<grid, 256, 0, st>>>(m->codes, m->scales, m->rows, m->K, o, ld * size);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? MQ_OK : cuda_fail(e, "mx_dequantize_kernel");
}
