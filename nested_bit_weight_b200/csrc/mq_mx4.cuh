// MXFP4 (include/mq.h: e2m1 elements, one power-of-two scale per 32 columns):
// the block arithmetic and the storage indices shared by the converters and
// the products.
#pragma once

#include <cuda.h>

#include "mq_common.cuh"

namespace mq {

constexpr int kMxBlock = 32;                 // columns per scale
constexpr int64_t kMxMaxDim = ((int64_t)1 << 31) - 256;   // rows and K (32-bit coordinates)

// Validate an MXFP4 matrix; returns MQ_OK or the failing status.
mq_status check_mx4(const mq_mx4 *m, const char *what);

// Tensor map of codes (rows x K / 2 bytes) in boxes of 128 bytes x `box` rows,
// 128-byte swizzle; bytes and rows beyond the matrix read as zeros.
bool mx_encode_codes(CUtensorMap *map, const uint8_t *codes, int64_t rows, int64_t K, int box);
// Tensor map of scale blocks (`rows` matrix rows) in boxes of two blocks x `box`
// row bands (1024 bytes a band); blocks beyond the buffer read as zeros.
bool mx_encode_scales(CUtensorMap *map, const uint8_t *scales, int64_t rows, int64_t K, int box);
// Tensor map of Y (M x N of type `out`, row stride ldy) in boxes of 128 bytes x 32
// rows, 128-byte swizzle; the row stride must be a multiple of 16 bytes.
bool mx_encode_y(CUtensorMap *map, void *Y, int64_t M, int64_t N, int64_t ldy, int out);

// How M bf16 rows lie as MXFP4 rows (a workspace of the product): kMxSlices a row,
// `tpt` rows of X a tile of `bn` MXFP4 rows; a tile's scales start a row band of
// their own.  Tb = 0: one tile, of the kernel for few rows.
struct MxSlicing {
    int Tb, tpt, bn;
    int64_t rows, bands;           // MXFP4 rows, row bands of scales
};
MxSlicing mx_slicing(int64_t M, int64_t N);   // N: output features
mq_status launch_mx_slices(const uint16_t *X, int64_t M, int64_t K, int64_t ldx, const MxSlicing &sl,
                           uint8_t *codes, uint8_t *scales, cudaStream_t st);

// One product: X of M MXFP4 rows (slices = 1) or as laid out by `slice`, w of N rows.
struct MxProduct {
    const uint8_t *xcodes, *xscales;
    int64_t M;
    int slices;
    const mq_mx4 *w;
    void *Y;
    int out;
    int64_t ldy;
    const uint16_t *X;             // bf16 rows cut within the product (few rows), or NULL
    int64_t ldx;
    MxSlicing slice;
};
bool mx_pair_takes(const MxProduct &p);
mq_status launch_mx_pair(const MxProduct &p, cudaStream_t st);
bool mx_pair_take_timeout(bool *set);

// Column groups of 128 (scale blocks of a row band).
__host__ __device__ __forceinline__ int64_t mx_groups(int64_t K) { return (K + 127) / 128; }

// Byte of the scales buffer that holds row `row`, columns 128 g .. 128 g + 31
// (the three bytes behind it: the next 32 columns each).
__host__ __device__ __forceinline__ int64_t mx_scale_at(int64_t row, int64_t g, int64_t G) {
    return ((row >> 7) * G + g) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

// Scale byte of a block whose largest magnitude has the bit pattern `amax`
// (fp32, sign cleared): floor(log2 a) - 2 + 127, at least 0 (subnormal and
// tiny blocks), 255 for a NaN or an infinity.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
    const uint32_t f = amax >> 23;
    return f == 255u ? 255u : (f > 2u ? f - 2u : 0u);
}

// 2^(127 - E) for E <= 253.
__device__ __forceinline__ float mx_inverse(uint32_t E) { return __uint_as_float((254u - E) << 23); }

// 2^(E - 127), NaN for E = 255.
__device__ __forceinline__ float mx_value(uint32_t E) {
    return E == 0u ? __uint_as_float(0x00400000u) : E == 255u ? __uint_as_float(0x7FC00000u)
                                                              : __uint_as_float(E << 23);
}

// Eight numbers, already divided by their scale, to eight codes (nearest,
// ties to even, above 6 to 6), the first in the lowest bits.
__device__ __forceinline__ uint32_t mx_codes8(const float (&u)[8]) {
    uint32_t r;
    asm("{\n .reg .b8 a, b, c, d;\n"
        " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
        " cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        " mov.b32 %0, {a, b, c, d};\n}"
        : "=r"(r)
        : "f"(u[0]), "f"(u[1]), "f"(u[2]), "f"(u[3]), "f"(u[4]), "f"(u[5]), "f"(u[6]), "f"(u[7]));
    return r;
}

// Eight codes to the numbers they stand for before scaling, two a register.
// Each byte is moved down by itself: taking the word apart with one
// mov.b32 {a, b, c, d} loses the upper bytes when the word was put together
// the same way just before (nvcc 12.9).
__device__ __forceinline__ void mx_halves8(uint32_t codes, __half2 (&h)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t r;
        asm("{\n .reg .b8 a;\n cvt.u8.u32 a, %1;\n cvt.rn.f16x2.e2m1x2 %0, a;\n}" : "=r"(r) : "r"(codes >> (8 * i)));
        h[i] = *reinterpret_cast<const __half2 *>(&r);
    }
}
__device__ __forceinline__ void mx_units8(uint32_t codes, float (&u)[8]) {
    __half2 h[4];
    mx_halves8(codes, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(h[i]);
        u[2 * i] = f.x;
        u[2 * i + 1] = f.y;
    }
}

// ---- bf16 rows as sums of MXFP4 rows.  With a = max |x| of a
// block, slice 0 has the least unit 2^e0 with a <= 7 * 2^e0: rounding to the
// grid leaves at most 1 unit (up to 5 by half a step, above 5 to 6).  In units
// a quarter as large that rest is at most 4, where the grid's half step is
// 1/2; in units an eighth as large again at most 4, and so on.  After S slices
// the rest is at most 2^(e0 - 3 (S - 1)): below 2^-22 a with eight (a > 3.5 * 2^e0).
// Always eight, whatever the output's type: how much of an element must stay is
// not for the output's last bit to say, since a block's largest element may meet
// weights of zero and leave the output to elements a thousandth its size.  Six
// slices, 2^-16 a, kept only six bits of those (256 x 14336 x 4096: 35 us with
// six, 43 with eight).
constexpr int kMxSlices = 8;

__device__ __forceinline__ uint32_t mx_slice0_byte(uint32_t amax) {
    const uint32_t f = (amax >> 23) + ((amax & 0x7FFFFFu) > 0x600000u ? 1u : 0u);   // a > 1.75 * 2^k
    return (amax >> 23) == 255u ? 255u : (f > 2u ? f - 2u : 0u);
}
// Scale byte of slice j from that of slice 0 (at least 0; 255 stays).
__device__ __forceinline__ uint32_t mx_slice_byte(uint32_t E, int j) {
    const uint32_t d = j == 0 ? 0u : 3u * (uint32_t)j - 1u;
    return E == 255u ? 255u : (E > d ? E - d : 0u);
}
// Eight numbers, already divided by slice 0's unit (at most 7), as the start of
// the slices.  fp16 holds them: a bf16 number's 8 bits down to 2^-14 of the unit,
// and below that what it cuts off, at most 2^-25, is less than eight slices leave.
__device__ __forceinline__ void mx_slice_start(const float (&x)[8], float inv, __half2 (&u)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __floats2half2_rn(x[2 * i] * inv, x[2 * i + 1] * inv);
}
// Codes of one slice of eight numbers u (in the slice's unit); u becomes the
// rest in the next slice's unit, 2^-step times as large.  Both steps are exact:
// the rest has no bit below the number's own last one and is smaller.
__device__ __forceinline__ uint32_t mx_slice_codes(__half2 (&u)[4], uint32_t step) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = __half22float2(u[i]);
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
    const uint32_t c = mx_codes8(f);
    __half2 q[4];
    mx_halves8(c, q);
    const __half2 m = __half2half2(__ushort_as_half((unsigned short)((15u + step) << 10)));   // 2^step
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __hmul2(__hsub2(u[i], q[i]), m);
    return c;
}

}  // namespace mq
