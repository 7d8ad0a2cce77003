// MXFP4 quantisation of one 32-element block (OCP Microscaling v1.0, E2M1 elements, E8M0 scale),
// shared by the quantiser and the product's SwiGLU epilogue, and the launchers of both.
//
//   m = max|v|,  e = max(floor(log2 m) - 2, -127)   (e = 0 for a block of zeros)
//   code = E2M1(v * 2^-e), round to nearest even, saturating at 6;  scale byte = e + 127
//
// v * 2^-e is exact (a power of two, and the result is in the normal range whenever it is 0.25
// or more), so the only rounding is the one to E2M1.  A block that holds a NaN or an infinity gets
// the scale byte 0xFF (NaN) and zero codes: every value of it reads as NaN.
#pragma once
#include "kernels.h"

namespace ftmoe {

// bits: max over the block of the elements' float bit patterns without the sign (an unsigned
// maximum, so a NaN wins over everything).  Returns the scale byte and the multiplier 2^-e.
__device__ __forceinline__ uint32_t mx4_scale_of(uint32_t bits, float& mul) {
    if (bits >= 0x7F800000u) { mul = 0.f; return 255u; }
    if (bits == 0u) { mul = 1.f; return 127u; }
    const uint32_t f = bits >> 23;                   // floor(log2 m) + 127; 0 for subnormals, which clamp anyway
    const uint32_t s = f > 2u ? f - 2u : 0u;
    mul = __uint_as_float((254u - s) << 23);         // 2^(127 - s), a normal float for s in 0..252
    return s;
}
// 2^(s - 127); s = 0 is a subnormal float, 255 a NaN
__device__ __forceinline__ float e8m0_float(uint32_t s) {
    return __uint_as_float(s == 0u ? 0x00400000u : s == 255u ? 0x7FFFFFFFu : s << 23);
}
// eight scaled floats -> four code bytes, element 0 in the low nibble of the lowest byte
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r) : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}
// eight codes -> the values they stand for, times scale (exact in fp32)
__device__ __forceinline__ void e2m1x8_values(uint32_t w, float scale, float (&o)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 p = *reinterpret_cast<const __half2*>(&h[i]);
        o[2 * i] = __low2float(p) * scale;
        o[2 * i + 1] = __high2float(p) * scale;
    }
}

// ------------------------------------------------------------------ launchers
cudaError_t launch_mx4_quantize(int64_t rows, int cols, int dtype, const void* x, int64_t x_stride, uint8_t* codes,
                                uint8_t* scales, void* values, cudaStream_t st);
// bf16 rows x [T, H] quantised once and written to their sorted places (inv_pos) of codes / scales
cudaError_t launch_mx4_sorted_tokens(int T, int H, int k, int S, const uint16_t* x, const int32_t* inv_pos,
                                     uint8_t* codes, uint8_t* scales, cudaStream_t st);

struct Mx4Launch {
    int swiglu;                 // 1: gate/up pairs -> silu(gate) * up -> MXFP4 h; 0: bf16 rows
    int G, E, R, N, K;          // groups, routed groups (group E.. takes the shared weights), rows, output columns, contraction
    const int32_t* offsets;     // [G + 1]
    const uint8_t* a;           // activation codes [R, K/2], scales [R, K/32]
    const uint8_t* as;
    const uint8_t* w;           // weight codes [E, rows, K/2], scales [E, rows, K/32]; rows = N, or 2N with swiglu
    const uint8_t* ws;
    const uint8_t* sw;          // the shared group's weights (G > E)
    const uint8_t* sws;
    uint16_t* out;              // swiglu == 0: [R, N] bf16
    uint8_t* hq;                // swiglu == 1: [R, N/2] codes, [R, N/32] scales
    uint8_t* hs;
    uint32_t* err;
    int early;                  // the kernel launched before on the stream is the token quantiser or this product, with
                                // offsets and weights from before it: they may be read ahead of the wait for it
};
// 0 ok, 1 tensor-map failure, 2 launch failure
int launch_mx4_product(const Mx4Launch& L, cudaStream_t st);

}  // namespace ftmoe
