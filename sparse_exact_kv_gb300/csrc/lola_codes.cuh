// Shared by the kernels that read a quantised cache: e4m3 numbers and powers of two as a byte (biased by 127).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace lola {

// four e4m3 numbers as float16 numbers
__device__ __forceinline__ void widen(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ uint32_t half2_of(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

constexpr float kUpBits = 15.f;           // the weights' factor: 2^15
// Parts of softmaxes are left against 2^20 times the largest score's weight: sums of that many values of float32's largest
// size stay in its range, and means of rows of the smallest powers, 2^-100, nearly all their bits.
constexpr float kRoom = 20.f;

}  // namespace lola
