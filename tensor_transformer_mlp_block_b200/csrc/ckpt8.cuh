// The 8-bit checkpoint of a pre-activation: blocks of 32 columns of a row, one
// power of two per block, 8-bit integers (the format is stated in
// include/tpmlp.h). Used by the GEMM epilogues and by the element-wise
// kernels, so both round alike. In the epilogues a lane's row of a chunk is one
// block, so neither the scale nor the rounding needs other lanes. Forward and
// backward of 6144 × 1024 → 4096 → 1024 in bf16 (fp32 weight gradients, captured)
// take 312 µs on B200, 298 with H and Y kept in bf16: the backward's epilogue
// rebuilds Y beside dH.
//
// Block scale. For top = max |x| = m·2^k, m in [1, 2), the integers of the
// scale 2^(k-6) reach rint(64·m) <= 128, and 128 only for 64·m >= 127.5 (the
// tie rounds to even), where the scale is doubled. m >= 127.5/64 is a fraction
// field >= 0x7F0000, so adding 0x10000 to the float's bits carries into the
// exponent exactly there, and the biased exponent of the scale is the sum's
// exponent field less 6 (at least 0: 2^-127).
#pragma once

#include <cstdint>

namespace tpmlp {

constexpr int kC8Block = 32;      // columns per scale
constexpr uint32_t kC8NaN = 255;  // scale byte of a block that reads as NaN

// max that keeps a NaN (fmaxf drops it)
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Scale byte of a block whose largest magnitude is top (NaN if it holds one).
// The carry reaches the exponent of infinities from 127.5·2^121 up: there the
// scale would be 2^122 and 64 of it 2^128, no float, so such a block is marked
// like one with an infinity.
__device__ __forceinline__ uint32_t c8_scale_byte(float top) {
    const uint32_t carried = (__float_as_uint(top) & 0x7fffffffu) + 0x10000u;
    if (carried >= 0x7f800000u) return kC8NaN;
    const uint32_t field = carried >> 23;
    return field > 6u ? field - 6u : 0u;
}

// 2^(127 - s): what x is multiplied by to be rounded. s <= 248 otherwise.
__device__ __forceinline__ float c8_inverse(uint32_t s) {
    return s == kC8NaN ? 0.0f : __uint_as_float((254u - s) << 23);
}

// The scale 2^(s - 127) itself (2^-127 is a subnormal); NaN for kC8NaN.
__device__ __forceinline__ float c8_scale(uint32_t s) {
    if (s == kC8NaN) return __uint_as_float(0x7fffffffu);
    return __uint_as_float(s == 0u ? 0x00400000u : s << 23);
}

// Rounding: x·inv + 1.5·2^23 is rounded once, to an integer (ties to even), whose
// low byte is the two's complement wanted. (A block marked NaN stores zeros.)
constexpr float kC8Round = 12582912.0f;

__device__ __forceinline__ uint32_t c8_gather4(float t0, float t1, float t2, float t3) {
    return __byte_perm(__byte_perm(__float_as_uint(t0), __float_as_uint(t1), 0x0040),
                       __byte_perm(__float_as_uint(t2), __float_as_uint(t3), 0x0040), 0x5410);
}

__device__ __forceinline__ uint32_t c8_pack4(float x0, float x1, float x2, float x3, float inv) {
    return c8_gather4(__fmaf_rn(x0, inv, kC8Round), __fmaf_rn(x1, inv, kC8Round), __fmaf_rn(x2, inv, kC8Round),
                      __fmaf_rn(x3, inv, kC8Round));
}

// The integers of four int8 as floats (exact): byte + 128 in the low mantissa
// bits of 2^23, less 2^23 + 128.
__device__ __forceinline__ void c8_unpack4(uint32_t w, float scale, float* x) {
    const uint32_t u = w ^ 0x80808080u;
    constexpr float kBias = 8388736.0f;
    x[0] = (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440)) - kBias) * scale;
    x[1] = (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441)) - kBias) * scale;
    x[2] = (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7442)) - kBias) * scale;
    x[3] = (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7443)) - kBias) * scale;
}

}  // namespace tpmlp
