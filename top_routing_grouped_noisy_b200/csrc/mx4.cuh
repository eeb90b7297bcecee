// mx4.cuh -- the microscaled 4-bit format of the mx4 calls (OCP Microscaling Formats
// (MX) Specification v1.0, MXFP4): e2m1 elements, one e8m0 scale per 32 columns.
//
// Every step of a block's quantisation is exact or a hardware rounding of the value
// itself, so codes and scales are the formula's, bit for bit: the maximum is taken on
// the f32 bit patterns, the scale exponent is a field of that pattern, 2^-s is a power
// of two (its product with the value is exact unless it falls below 2^-126, far under
// the smallest code), and the conversion rounds to nearest, ties to even, saturating.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {

constexpr int kMx4Block = 32;      // columns that share a scale
constexpr int kMx4Tile = 512;      // bytes of a scale tile: 128 rows x 4 blocks

// Scale byte (s + 127) of a block whose largest magnitude has the bit pattern `amax`;
// 255 for a NaN or an infinity.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax)
{
    const uint32_t e = amax >> 23;
    return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}

// 2^-s of a scale byte <= 252 (what mx4_scale_byte gives for finite blocks)
__device__ __forceinline__ float mx4_inverse(uint32_t byte)
{
    return __uint_as_float((254u - byte) << 23);
}

// 2^s of any scale byte; 255 is NaN
__device__ __forceinline__ float mx4_scale(uint32_t byte)
{
    if (byte == 255u)
        return __uint_as_float(0x7fc00000u);
    return __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
}

// 8 values, already multiplied by 2^-s, as 8 codes (value 0 in the low bits)
__device__ __forceinline__ uint32_t mx4_codes8(const float (&v)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// 8 codes as four f16 pairs (exact): h[i] holds codes 2i (low half) and 2i + 1
__device__ __forceinline__ void mx4_halves8(uint32_t codes, uint32_t (&h)[4])
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
}

// Byte of row r (of its matrix or expert) and block b in a matrix whose tile rows hold
// `tk` tiles, the matrix starting at tile row `tile0`.
__host__ __device__ inline int64_t mx4_scale_at(int64_t tile0, int tk, int r, int b)
{
    return ((tile0 + r / 128) * tk + b / 4) * kMx4Tile + (r % 32) * 16 + (r % 128) / 32 * 4 + b % 4;
}

// First tile row of expert e's rows (they start at row `off`): an expert's tiles end
// before the next one's, since off/128 + e + ceil(n/128) <= (off + n)/128 + e + 1.
__host__ __device__ inline int64_t mx4_expert_tile(int off, int e) { return off / 128 + e; }

// Tile rows that T*k rows of E experts can take.
__host__ __device__ inline int64_t mx4_row_tiles(int64_t rows, int E) { return rows / 128 + E + 1; }

__host__ __device__ inline int mx4_k32(int K) { return (K + 31) / 32 * 32; }

}  // namespace moe
